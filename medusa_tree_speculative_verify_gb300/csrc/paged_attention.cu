// Attention of one new token for each sequence over a paged cache: the entry points (the kernel: paged_attn.cuh).
#include "paged_attn.cuh"

namespace {

// Keys of a step of all warps.
template <PagedFormat kFormat>
int step_keys(bool big, bool wide) {
  if (big) return wide ? Layout<128, kFormat, 2>::kStepKeys : Layout<128, kFormat, 1>::kStepKeys;
  return wide ? Layout<64, kFormat, 2>::kStepKeys : Layout<64, kFormat, 1>::kStepKeys;
}

}  // namespace

extern "C" mv_status paged_attention_workspace(int32_t n_seq, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                               size_t* bytes) {
  if (!bytes || n_seq < 0) return MV_ERR_INVALID_ARG;
  if (n_seq > kPagedMaxSeq || n_kv_heads < 1 || n_heads < n_kv_heads || n_heads > kPagedMaxHeads ||
      n_heads % n_kv_heads || head_dim < 16 || head_dim > kPagedMaxDim || head_dim % 16)
    return MV_ERR_SHAPE;
  // counters, and two partial results of 16 heads for each CTA
  *bytes = kMaxCtas * sizeof(uint32_t) + (size_t)kMaxCtas * 2 * Layout<128, kBf16, 2>::kPart * sizeof(float);
  return MV_OK;
}

extern "C" mv_status paged_attention(mv_rows q, int32_t n_heads, const mv_paged_kv* cache, const int32_t* block_table,
                                     int32_t ld_table, int32_t max_pages, const int32_t* seq_lens, int32_t n_seq,
                                     float scale, mv_rows out, void* workspace, size_t ws_bytes, mv_stream stream) {
  if (n_seq < 0) return MV_ERR_INVALID_ARG;
  if (n_seq == 0) return MV_OK;
  AttnArgs a;
  mv_status s = mv_paged_check(cache, block_table, ld_table, max_pages, seq_lens, n_seq, &a.c);
  if (s != MV_OK) return s;
  size_t need = 0;
  s = paged_attention_workspace(n_seq, n_heads, a.c.heads, a.c.dim, &need);
  if (s != MV_OK) return s;
  if (!mv_rows_ok(q, n_seq, n_heads, a.c.dim) || !mv_out_rows_ok(out, n_seq, n_heads, a.c.dim)) return MV_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) || !(scale >= 0.0f && scale * kLog2E < INFINITY))
    return MV_ERR_INVALID_ARG;
  if (ws_bytes < need) return MV_ERR_CAPACITY;
  a.group = n_heads / a.c.heads;
  const bool wide = a.group > 8;  // 16 heads a unit: their second tile of 8 shares the copies
  a.parts = wide ? (a.group + 15) / 16 : 1;
  a.scale_log2 = scale * kLog2E;
  a.count = static_cast<unsigned int*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kMaxCtas * sizeof(uint32_t));
  a.err = mv_error_word();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->dtype == MV_DTYPE_E4M3, e2m1 = cache->dtype == MV_DTYPE_E2M1, big = a.c.dim > 64;
  const int step = e2m1 ? step_keys<kE2M1>(big, wide) : e4m3 ? step_keys<kE4M3>(big, wide) : step_keys<kBf16>(big, wide);
  // sequences of a launch: no more than have places in 31 bits, whatever their lengths
  const int chunk = (int)std::min<int64_t>(kChunkSeq, 0x7fffffff / most_places(a, step));
  if (chunk < 1) return MV_ERR_SHAPE;
  for (int first = 0; first < n_seq; first += chunk) {
    a.c.n_seq = std::min(chunk, n_seq - first);
    a.c.table = block_table + (int64_t)first * ld_table;
    a.c.seq_lens = seq_lens + first;
    a.q = {static_cast<uint16_t*>(q.ptr) + first * q.token_stride, q.token_stride, q.head_stride};
    a.out = {static_cast<uint16_t*>(out.ptr) + first * out.token_stride, out.token_stride, out.head_stride};
    if (e2m1)
      s = launch_paged_attention_e2m1(a, wide, st);
    else if (big)
      s = e4m3 ? (wide ? launch<128, kE4M3, 2>(a, st) : launch<128, kE4M3, 1>(a, st))
               : (wide ? launch<128, kBf16, 2>(a, st) : launch<128, kBf16, 1>(a, st));
    else
      s = e4m3 ? (wide ? launch<64, kE4M3, 2>(a, st) : launch<64, kE4M3, 1>(a, st))
               : (wide ? launch<64, kBf16, 2>(a, st) : launch<64, kBf16, 1>(a, st));
    if (s != MV_OK) return s;
  }
  return MV_OK;
}
