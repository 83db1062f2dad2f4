// Attention kernels over a MXFP4 cache.
#include "ft_attn_chunk.cuh"
#include "ft_attn_rows.cuh"

namespace ft {
namespace kv {
cudaError_t attn_rows_mxfp4(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s) {
  return rows::launch_type<FT_KV_MXFP4>(p, D, rows, n_sm, s);
}
cudaError_t attn_chunk_mxfp4(const AttnParams& p, int D, int, int n_sm, cudaStream_t s) {
  return chunk::launch_type<FT_KV_MXFP4>(p, D, n_sm, s);
}
}  // namespace kv
}  // namespace ft
