// Between the entry points of the attention of several new tokens (attn_extend.hip)
// and the kernels for many of them (attn_prompt_typed.hip, once per cache type).
#pragma once

#include <hip/hip_runtime.h>

#include "attn_prompt.hpp"

namespace gqk {
// groups: of four waves per block, 1 or (up to head dim 128) 2.
void launch_prompt_f16(const AttnPromptArgs& a, int groups, dim3 grid, hipStream_t stream);
void launch_prompt_bf16(const AttnPromptArgs& a, int groups, dim3 grid, hipStream_t stream);
void launch_prompt_q8_0(const AttnPromptArgs& a, int groups, dim3 grid, hipStream_t stream);
}  // namespace gqk
