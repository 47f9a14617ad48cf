// Between the attention's entry points (attn.hip) and its kernels, which are
// compiled once per cache type (attn_typed.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "attn.hpp"

namespace gqk {
void launch_attn_f16(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
void launch_attn_bf16(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
void launch_attn_q8_0(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream);
// Several new tokens per sequence; columns of a block, 16 or 32 (Q8_0: with two tiles one
// wave per SIMD at head dim 128, 57 us against 48 for 8 x 5 drafted tokens behind 8000 slots;
// at 64 27 against 31, but 30 against 22 for 64 x 5 behind 1000).
constexpr int attn_most_columns(bool q8) { return q8 ? 16 : 32; }
void launch_attn_rows_f16(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream);
void launch_attn_rows_bf16(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream);
void launch_attn_rows_q8_0(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream);
}  // namespace gqk
