// The attention kernels of one cache type: GQK_KV_KIND 0 F16, 1 BF16, 2 Q8_0.
#include "attn_launch.hpp"

namespace gqk {

template <int NB>
static void launch_dim(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream) {
  if (track)
    hipLaunchKernelGGL((attn_decode_kernel<GQK_KV_KIND, NB, true>), grid, dim3(kAttnThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((attn_decode_kernel<GQK_KV_KIND, NB, false>), grid, dim3(kAttnThreads), 0, stream, a);
}

template <int NB>
static void launch_dim(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream) {
  if constexpr (attn_most_columns(GQK_KV_KIND == 2) == 32) {
    if (columns == 32) {
      hipLaunchKernelGGL((attn_decode_kernel<GQK_KV_KIND, NB, false, AttnRowsArgs, 2>), grid, dim3(kAttnThreads), 0,
                         stream, a);
      return;
    }
  }
  hipLaunchKernelGGL((attn_decode_kernel<GQK_KV_KIND, NB, false, AttnRowsArgs>), grid, dim3(kAttnThreads), 0, stream, a);
}

#if GQK_KV_KIND == 0
void launch_attn_f16(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream) {
#elif GQK_KV_KIND == 1
void launch_attn_bf16(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream) {
#else
void launch_attn_q8_0(const AttnArgs& a, bool track, dim3 grid, hipStream_t stream) {
#endif
  switch (a.c.dim) {
    case 64: return launch_dim<2>(a, track, grid, stream);
    case 96: return launch_dim<3>(a, track, grid, stream);
    case 128: return launch_dim<4>(a, track, grid, stream);
    case 192: return launch_dim<6>(a, track, grid, stream);
    default: return launch_dim<8>(a, track, grid, stream);
  }
}

#if GQK_KV_KIND == 0
void launch_attn_rows_f16(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream) {
#elif GQK_KV_KIND == 1
void launch_attn_rows_bf16(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream) {
#else
void launch_attn_rows_q8_0(const AttnRowsArgs& a, int columns, dim3 grid, hipStream_t stream) {
#endif
  switch (a.c.dim) {
    case 64: return launch_dim<2>(a, columns, grid, stream);
    case 96: return launch_dim<3>(a, columns, grid, stream);
    case 128: return launch_dim<4>(a, columns, grid, stream);
    case 192: return launch_dim<6>(a, columns, grid, stream);
    default: return launch_dim<8>(a, columns, grid, stream);
  }
}

}  // namespace gqk
