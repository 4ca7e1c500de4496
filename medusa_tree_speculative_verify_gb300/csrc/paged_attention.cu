// Attention of one new token for each sequence over a paged cache (bf16, or e4m3 with an exponent for each row).
//
// A warp computes one (sequence, query head): a lane holds four of the dim values, the warp goes over the keys with
// the running maximum and sum of the softmax.
#include "kernels.cuh"
#include "paged.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kCounters = 1024;

struct AttnArgs {
  PagedArgs c;
  RowsArgs q, out;
  int n_heads;
  float scale_log2;
  unsigned int* err;
};

template <bool kE4M3>
MV_DEV float4 load4(const uint8_t* pages, const uint8_t* exps, int64_t row, int D, int d0) {
  if (kE4M3) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(pages + row * D + d0);
    const float s = exp_byte_scale(exps[row]);
    const float2 a = half2_to_float2(e4m3x2_to_half2((uint16_t)w)), b = half2_to_float2(e4m3x2_to_half2((uint16_t)(w >> 16)));
    return make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
  }
  const uint2 w = *reinterpret_cast<const uint2*>(pages + (row * D + d0) * 2);
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

template <bool kE4M3>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_kernel(const AttnArgs a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, u = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (u >= a.c.n_seq * a.n_heads) return;
  const int b = u / a.n_heads, h = u % a.n_heads, kh = h / (a.n_heads / a.c.heads);
  const int D = a.c.dim, P = a.c.page_size, d0 = lane * 4;
  const bool on = d0 < D;
  const int len = __ldcg(a.c.seq_lens + b);
  if (len < 0 || len > a.c.max_pages * P) {
    if (lane == 0) mv_set_error_detail(a.err, kPagedAttnSite, MV_DEVERR_INDEX, (uint32_t)b);
    return;
  }
  float4 q = make_float4(0.f, 0.f, 0.f, 0.f), o = q;
  const int64_t qat = (int64_t)b * a.q.ts + (int64_t)h * a.q.hs + d0;
  if (on) {
    const uint2 w = *reinterpret_cast<const uint2*>(a.q.p + qat);
    q = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = 0; j < len; ++j) {
    const int page = __ldcg(a.c.table + (int64_t)b * a.c.ld_table + j / P);
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) mv_set_error_detail(a.err, kPagedAttnSite, MV_DEVERR_INDEX, (uint32_t)page);
      return;
    }
    const int64_t row = ((int64_t)page * a.c.heads + kh) * P + j % P;
    float x = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      const float4 k = load4<kE4M3>(a.c.k, a.c.k_exp, row, D, d0);
      v = load4<kE4M3>(a.c.v, a.c.v_exp, row, D, d0);
      x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
    }
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    x *= a.scale_log2;
    const float mn = fmaxf(m, x), f = m == mn ? 1.0f : exp2f(m - mn), p = exp2f(x - mn);
    m = mn;
    l = l * f + p;
    o = make_float4(o.x * f + p * v.x, o.y * f + p * v.y, o.z * f + p * v.z, o.w * f + p * v.w);
  }
  const float inv = len > 0 ? 1.0f / l : 0.0f;
  if (on)
    *reinterpret_cast<uint2*>(a.out.p + (int64_t)b * a.out.ts + (int64_t)h * a.out.hs + d0) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

}  // namespace

extern "C" mv_status paged_attention_workspace(int32_t n_seq, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                               size_t* bytes) {
  if (!bytes || n_seq < 0) return MV_ERR_INVALID_ARG;
  if (n_seq > kPagedMaxSeq || n_kv_heads < 1 || n_heads < n_kv_heads || n_heads > kPagedMaxHeads ||
      n_heads % n_kv_heads || head_dim < 16 || head_dim > kPagedMaxDim || head_dim % 16)
    return MV_ERR_SHAPE;
  *bytes = kCounters * sizeof(uint32_t);
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
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) || !(scale >= 0.0f && scale < INFINITY))
    return MV_ERR_INVALID_ARG;
  if (ws_bytes < need) return MV_ERR_CAPACITY;
  a.q = {static_cast<uint16_t*>(q.ptr), q.token_stride, q.head_stride};
  a.out = {static_cast<uint16_t*>(out.ptr), out.token_stride, out.head_stride};
  a.n_heads = n_heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.err = mv_error_word();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid((n_seq * n_heads + kWarps - 1) / kWarps);
  const cudaError_t e = cache->dtype == MV_DTYPE_E4M3
                            ? mv_launch(paged_attn_kernel<true>, grid, dim3(kWarps * 32), 0, st, a)
                            : mv_launch(paged_attn_kernel<false>, grid, dim3(kWarps * 32), 0, st, a);
  return e == cudaSuccess ? mv_last_launch("paged_attention") : MV_ERR_CUDA;
}
