// Between the attention's entry points (attn.hip) and its kernels, which are
// compiled once per cache type (attn_typed.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "attn.hpp"

namespace gqk {
void launch_attn_f16(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
void launch_attn_bf16(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
void launch_attn_q8_0(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
// Several new tokens per sequence.
void launch_attn_rows_f16(const AttnRowsArgs& a, dim3 grid, hipStream_t stream);
void launch_attn_rows_bf16(const AttnRowsArgs& a, dim3 grid, hipStream_t stream);
void launch_attn_rows_q8_0(const AttnRowsArgs& a, dim3 grid, hipStream_t stream);
}  // namespace gqk
