// zo_internal.h -- launchers between the C ABI of the training operators
// (zo_abi.hip) and their kernels.  Arguments arrive validated; launchers pick
// the template instance and the grid.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zero_ops.h"

namespace zo {

hipError_t launch_qk_norm_rope_fwd(const zero_qk_norm_rope_args& a, hipStream_t s);
hipError_t launch_qk_norm_rope_bwd(const zero_qk_norm_rope_args& a, hipStream_t s);
size_t qk_norm_rope_workspace(int64_t T, int D);

hipError_t launch_attn_fwd(const zero_attn_args& a, hipStream_t s);
hipError_t launch_attn_bwd(const zero_attn_args& a, hipStream_t s);
hipError_t launch_attn_ranges(const int32_t* doc, const int32_t* prefix, int B, int T, int causal,
                              int32_t* ranges, hipStream_t s);
size_t attn_fwd_workspace(int B, int Tq, int Tk, int Hq, int Hk, int D);
size_t attn_bwd_workspace(int B, int Tq, int Tk, int Hq, int Hk, int D, int n_buckets);

hipError_t launch_distill(const zero_distill_args& a, bool forward, hipStream_t s);

}  // namespace zo
