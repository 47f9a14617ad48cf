// The kernels of the attention of many new tokens, of one cache type: GQK_KV_KIND 0
// F16, 1 BF16, 2 Q8_0.
#include "attn_prompt_launch.hpp"

namespace gqk {

template <int NB>
static void launch_dim(const AttnPromptArgs& a, int groups, dim3 grid, hipStream_t stream) {
  if constexpr (prompt_groups(GQK_KV_KIND == 2, NB * 32) == 2) {
    if (groups == 2) {
      hipLaunchKernelGGL((attn_prompt_kernel<GQK_KV_KIND, NB, 2>), grid, dim3(2 * kPromptThreads), 0, stream, a);
      return;
    }
  }
  hipLaunchKernelGGL((attn_prompt_kernel<GQK_KV_KIND, NB, 1>), grid, dim3(kPromptThreads), 0, stream, a);
}

#if GQK_KV_KIND == 0
void launch_prompt_f16(const AttnPromptArgs& a, int groups, dim3 grid, hipStream_t stream) {
#elif GQK_KV_KIND == 1
void launch_prompt_bf16(const AttnPromptArgs& a, int groups, dim3 grid, hipStream_t stream) {
#else
void launch_prompt_q8_0(const AttnPromptArgs& a, int groups, dim3 grid, hipStream_t stream) {
#endif
  switch (a.c.dim) {
    case 64: return launch_dim<2>(a, groups, grid, stream);
    case 96: return launch_dim<3>(a, groups, grid, stream);
    case 128: return launch_dim<4>(a, groups, grid, stream);
    case 192: return launch_dim<6>(a, groups, grid, stream);
    default: return launch_dim<8>(a, groups, grid, stream);
  }
}

}  // namespace gqk
