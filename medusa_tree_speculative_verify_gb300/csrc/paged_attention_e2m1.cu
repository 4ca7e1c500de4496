// Attention of one new token for each sequence over a paged cache of 4-bit rows: the kernel of paged_attn.cuh for them.
#include "paged_attn.cuh"

namespace {

template <int kDim, bool kWhole>
mv_status launch_dims(const AttnArgs& a, bool wide, cudaStream_t stream) {
  return wide ? launch<kDim, kE2M1, 2, kWhole>(a, stream) : launch<kDim, kE2M1, 1, kWhole>(a, stream);
}

}  // namespace

mv_status launch_paged_attention_e2m1(const AttnArgs& a, bool wide, cudaStream_t stream) {
  switch (a.c.dim) {
    case 128: return launch_dims<128, true>(a, wide, stream);
    case 96: return launch_dims<128, false>(a, wide, stream);
    case 64: return launch_dims<64, true>(a, wide, stream);
    default: return launch_dims<64, false>(a, wide, stream);
  }
}
