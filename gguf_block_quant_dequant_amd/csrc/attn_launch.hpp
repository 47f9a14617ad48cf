// Between the attention's entry points (attn.hip) and its kernels, which are
// compiled once per cache type (attn_typed.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "attn.hpp"

namespace gqk {
void launch_attn_f16(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
void launch_attn_bf16(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
void launch_attn_q8_0(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
// Several new tokens per sequence; columns of a block, 16 or 32: up to head dim 128, where
// registers hold two tiles of them (Q8_0: one wave per SIMD then, 57 us against 51 for 8 x 5
// drafted tokens).
constexpr int attn_most_columns(bool q8, int dim) { return dim <= 128 && !q8 ? 32 : 16; }
void launch_attn_rows_f16(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream);
void launch_attn_rows_bf16(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream);
void launch_attn_rows_q8_0(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream);
}  // namespace gqk
