// Rows of keys and values written into a paged cache, and read back.
//
// A row is one token's head_dim values of one kv head. A group of kLanes threads moves one row, 8 elements a thread
// (16 bytes of bf16, 8 of e4m3). Writing e4m3: the group's largest |x| gives the exponent e, the smallest with max|x| <=
// 448 * 2^e: with max|x| = 1.m * 2^(E-127), 448 = 1.75 * 2^8, that is e = E - 135, one more when 1.m > 1.75. The
// product with 2^-e is exact (short of underflow), so the row is rounded once, by the conversion, and what it stands
// for is exact in bf16 again.
//
// Bound by memory: 2 * dim bytes read (written) and dim + 1 or 2 * dim written (read) for each row, K and V.
#include "kernels.cuh"
#include "paged.cuh"

namespace {

constexpr int kThreads = 256;

struct MoveArgs {
  PagedArgs c;
  RowsArgs k, v;
  const int32_t* cu;
  int n_rows, tokens;  // tokens: rows of a CTA
  unsigned int* err;
};

// Where row token t of the packed rows lies: page * page_size + slot, -1 for a row behind the last sequence, -2 when
// the table, the lengths or cu are out of range.
MV_DEV int64_t place_of(const MoveArgs& a, int t) {
  if (t >= __ldcg(a.cu + a.c.n_seq)) return -1;
  int lo = 0, hi = a.c.n_seq;  // the last b with cu[b] <= t (cu[0] = 0), found whatever cu holds
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(a.cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int c0 = __ldcg(a.cu + lo), c1 = __ldcg(a.cu + lo + 1);
  if (c0 < 0 || t < c0 || t >= c1) return -2;
  const int len = __ldcg(a.c.seq_lens + lo);
  const int64_t pos = (int64_t)len - c1 + t;
  if (len < c1 - c0 || pos < 0 || pos >= (int64_t)a.c.max_pages * a.c.page_size) return -2;
  const int page = __ldcg(a.c.table + (int64_t)lo * a.c.ld_table + (int)pos / a.c.page_size);
  if (page < 0 || page >= a.c.n_pages) return -2;
  return (int64_t)page * a.c.page_size + (int)pos % a.c.page_size;
}

template <bool kE4M3, bool kWrite>
__global__ void __launch_bounds__(kThreads) paged_rows_kernel(const MoveArgs a, int lanes) {
  __shared__ int64_t s_place[32];
  pdl_trigger();
  pdl_wait();
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.n_rows - t0);
  if ((int)threadIdx.x < nt) {
    const int64_t at = place_of(a, t0 + threadIdx.x);
    if (at == -2) mv_set_error_detail(a.err, kPagedRowsSite, MV_DEVERR_INDEX, (uint32_t)(t0 + threadIdx.x));
    s_place[threadIdx.x] = at;
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.c.n_seq; b += kThreads) {
      const int c0 = __ldcg(a.cu + b), c1 = __ldcg(a.cu + b + 1);
      if ((b == 0 && c0 != 0) || c1 < c0 || c1 > a.n_rows)
        mv_set_error_detail(a.err, kPagedRowsSite, MV_DEVERR_INDEX, (uint32_t)b);
    }
  __syncthreads();
  const int ln = threadIdx.x & (lanes - 1), d0 = ln * 8;  // this thread's elements d0 .. d0 + 7 of its row
  const int H = a.c.heads, D = a.c.dim, P = a.c.page_size;
  const int rows = nt * 2 * H;  // (token, K or V, head), heads fastest
  // whole groups of lanes leave the loop together: rows is the same for all of a group
  for (int r = threadIdx.x / lanes; r < rows; r += kThreads / lanes) {
    const int h = r % H, tv = r / H, tok = tv >> 1;
    const int64_t at = s_place[tok];
    const bool is_v = tv & 1, live = at >= 0 && d0 < D;
    const RowsArgs& x = is_v ? a.v : a.k;
    uint16_t* row = x.p + (int64_t)(t0 + tok) * x.ts + (int64_t)h * x.hs + d0;
    const int64_t prow = at < 0 ? 0 : (at / P * H + h) * P + at % P;
    uint8_t* pages = is_v ? a.c.v : a.c.k;
    if (!kE4M3) {
      uint4* held = reinterpret_cast<uint4*>(pages + (prow * D + d0) * 2);
      if (live) {
        if (kWrite) *held = *reinterpret_cast<const uint4*>(row);
        else *reinterpret_cast<uint4*>(row) = *held;
      }
    } else {
      uint8_t* exps = is_v ? a.c.v_exp : a.c.k_exp;
      uint2* held = reinterpret_cast<uint2*>(pages + prow * D + d0);
      if (kWrite) {
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (live) raw = *reinterpret_cast<const uint4*>(row);
        float f[8];
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf16lo(w[i]);
          f[2 * i + 1] = bf16hi(w[i]);
          top = fmaxf(top, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));  // a NaN does not count
        }
        const uint32_t mask = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
        for (int o = lanes >> 1; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
        const uint32_t b = __float_as_uint(top);
        const int e = max(-100, min(120, (int)(b >> 23) - 135 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0)));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint16_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = float2_to_e4m3x2(f[2 * i] * inv, f[2 * i + 1] * inv);
        if (live) {
          *held = make_uint2((uint32_t)q[0] | ((uint32_t)q[1] << 16), (uint32_t)q[2] | ((uint32_t)q[3] << 16));
          if (ln == 0) exps[prow] = (uint8_t)(e + 127);
        }
      } else if (live) {
        const float s = exp_byte_scale(exps[prow]);
        const uint2 w = *held;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = half2_to_float2(e4m3x2_to_half2((uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1)))));
          o[i] = pack_bf16x2(f.x * s, f.y * s);
        }
        *reinterpret_cast<uint4*>(row) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <bool kWrite>
mv_status move_rows(const mv_rows& k, const mv_rows& v, int32_t n_rows, const int32_t* cu, const mv_paged_kv* cache,
                    const int32_t* table, int32_t ld_table, int32_t max_pages, const int32_t* seq_lens, int32_t n_seq,
                    mv_stream stream) {
  if (n_rows < 0 || n_seq < 0) return MV_ERR_INVALID_ARG;
  if (n_rows == 0 || n_seq == 0) return MV_OK;
  MoveArgs a;
  const mv_status s = mv_paged_check(cache, table, ld_table, max_pages, seq_lens, n_seq, &a.c);
  if (s != MV_OK) return s;
  bool (*rows_ok)(const mv_rows&, int64_t, int, int) = kWrite ? mv_rows_ok : mv_out_rows_ok;
  if (!cu || !rows_ok(k, n_rows, a.c.heads, a.c.dim) || !rows_ok(v, n_rows, a.c.heads, a.c.dim))
    return MV_ERR_INVALID_ARG;
  a.k = {static_cast<uint16_t*>(k.ptr), k.token_stride, k.head_stride};
  a.v = {static_cast<uint16_t*>(v.ptr), v.token_stride, v.head_stride};
  a.cu = cu;
  a.n_rows = n_rows;
  a.tokens = 1;
  a.err = mv_error_word();
  int lanes = 2;
  while (lanes * 8 < a.c.dim) lanes *= 2;
  const dim3 grid((n_rows + a.tokens - 1) / a.tokens);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == MV_DTYPE_E4M3
                            ? mv_launch(paged_rows_kernel<true, kWrite>, grid, dim3(kThreads), 0, st, a, lanes)
                            : mv_launch(paged_rows_kernel<false, kWrite>, grid, dim3(kThreads), 0, st, a, lanes);
  return e == cudaSuccess ? mv_last_launch("paged_rows") : MV_ERR_CUDA;
}

}  // namespace

extern "C" mv_status paged_kv_append(mv_rows k, mv_rows v, int32_t n_rows, const int32_t* cu_rows,
                                     const mv_paged_kv* cache, const int32_t* block_table, int32_t ld_table,
                                     int32_t max_pages, const int32_t* seq_lens, int32_t n_seq, mv_stream stream) {
  return move_rows<true>(k, v, n_rows, cu_rows, cache, block_table, ld_table, max_pages, seq_lens, n_seq, stream);
}

extern "C" mv_status paged_kv_read(const mv_paged_kv* cache, const int32_t* block_table, int32_t ld_table,
                                   int32_t max_pages, const int32_t* seq_lens, int32_t n_seq, const int32_t* cu_rows,
                                   int32_t n_rows, mv_rows k, mv_rows v, mv_stream stream) {
  return move_rows<false>(k, v, n_rows, cu_rows, cache, block_table, ld_table, max_pages, seq_lens, n_seq, stream);
}
