// attn_many_bf16.hip -- attn_many.h's kernels for bf16 (a source each: they take long to compile).
#include "attn_many.h"

namespace hca {
hipError_t launch_many_bf16(const AttendArgs& a, hipStream_t s) { return run_many<false>(a, s); }
}  // namespace hca
