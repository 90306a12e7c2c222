// few_instantiate.hip -- defines the few-token drivers of few.hpp and route.hpp
// for one storage type and weight format. Compiled once per combination with
// -DSWIGLU_INST_DTYPE=0|1|2 (bf16, fp16, fp32) and -DSWIGLU_INST_FMT=0 (rows)
// or 32|64|128 (4 bits, that group size; 16-bit storage only).
#include "route.hpp"

#if !defined(SWIGLU_INST_DTYPE) || !defined(SWIGLU_INST_FMT)
#error "compile with -DSWIGLU_INST_DTYPE=<0|1|2> -DSWIGLU_INST_FMT=<0|32|64|128>"
#endif

namespace swiglu {
#if SWIGLU_INST_DTYPE == 0
using InstE = Bf16;
#elif SWIGLU_INST_DTYPE == 1
using InstE = Fp16;
#else
using InstE = Fp32;
#endif

namespace few {
template int run_block<InstE, SWIGLU_INST_FMT>(const Call&);
#if SWIGLU_INST_FMT != 0
template int run_linear<InstE, SWIGLU_INST_FMT>(const Call&);
#endif
}  // namespace few
#if SWIGLU_INST_FMT == 0
namespace route {
template int run_route<InstE>(Args, hipStream_t);
}
#endif
}  // namespace swiglu
