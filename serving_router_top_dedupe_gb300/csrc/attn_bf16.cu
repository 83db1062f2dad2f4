// Attention kernels over a BF16 cache.
#include "ft_attn_chunk.cuh"
#include "ft_attn_rows.cuh"

namespace ft {
namespace kv {
cudaError_t attn_rows_bf16(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s) {
  return rows::launch_type<FT_KV_BF16>(p, D, rows, n_sm, s);
}
cudaError_t attn_chunk_bf16(const AttnParams& p, int D, int, int n_sm, cudaStream_t s) {
  return chunk::launch_type<FT_KV_BF16>(p, D, n_sm, s);
}
}  // namespace kv
}  // namespace ft
