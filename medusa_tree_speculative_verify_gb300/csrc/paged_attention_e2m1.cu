// Attention of one new token for each sequence over a paged cache of 4-bit rows: the kernel of paged_attn.cuh for them.
#include "paged_attn.cuh"

mv_status launch_paged_attention_e2m1(const AttnArgs& a, bool big, bool wide, cudaStream_t stream) {
  if (big) return wide ? launch<128, kE2M1, 2>(a, stream) : launch<128, kE2M1, 1>(a, stream);
  return wide ? launch<64, kE2M1, 2>(a, stream) : launch<64, kE2M1, 1>(a, stream);
}
