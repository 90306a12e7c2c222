// dense_instantiate.hip -- defines the drivers of norm.hpp and linear.hpp (and so
// instantiates their kernels). Compiled with -DSWIGLU_INST_DTYPE=0|1|2 (bf16,
// fp16, fp32) and -DSWIGLU_INST_PART=0 (norms), 1 (linear layer) or, for 16-bit
// types, 2 .. 6 (the ring kernel of activation 0 .. 4, with 0
// that of a tile's parts).
#include "linear.hpp"

#if !defined(SWIGLU_INST_DTYPE) || !defined(SWIGLU_INST_PART)
#error "compile with -DSWIGLU_INST_DTYPE=<0|1|2> -DSWIGLU_INST_PART=<0..6>"
#endif

namespace swiglu {
#if SWIGLU_INST_DTYPE == 0
using InstE = Bf16;
#elif SWIGLU_INST_DTYPE == 1
using InstE = Fp16;
#else
using InstE = Fp32;
#endif

#if SWIGLU_INST_PART == 0
namespace norm {
template int run_fwd<InstE>(const Args&, bool, hipStream_t);
template int run_bwd<InstE>(const Args&, bool, void*, void*, hipStream_t);
}  // namespace norm
#elif SWIGLU_INST_PART == 1
namespace lin {
#if SWIGLU_INST_DTYPE != 2
SWIGLU_LIN_RING_DECL(extern, InstE)
#endif
template int run_fwd<InstE>(const Fwd&);
template int run_bwd<InstE>(const Bwd&);
}  // namespace lin
#else
namespace lin {
template int launch_lin_ring<InstE, SWIGLU_INST_PART - 2>(const KArgs&, hipStream_t);
#if SWIGLU_INST_PART == 2
template int launch_lin_ring_parts<InstE>(const KArgs&, hipStream_t);
#endif
}  // namespace lin
#endif
}  // namespace swiglu
