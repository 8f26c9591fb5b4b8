// attn_many_fp16.hip -- attn_many.h's kernels for fp16 (a source each: they take long to compile).
#include "attn_many.h"

namespace hca {
hipError_t launch_many_fp16(const AttendArgs& a, hipStream_t s) { return run_many<true>(a, s); }
}  // namespace hca
