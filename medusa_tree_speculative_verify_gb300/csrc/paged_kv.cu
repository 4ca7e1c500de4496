// Rows of keys and values written into a paged cache, and read back.
//
// A row is one token's head_dim values of one kv head. A group of kLanes threads moves one row, 16 elements a thread.
//
// Writing e4m3: the group's largest |x| gives the exponent e, the smallest with max|x| <= 448 * 2^e: with max|x| =
// 1.m * 2^(E-127), 448 = 1.75 * 2^8, that is e = E - 135, one more when 1.m > 1.75. The product with 2^-e is exact (short of
// underflow), so the row is rounded once, by the conversion, and what it stands for is exact in bf16 again.
//
// Writing e2m1: a thread's 16 elements are a group. Its scale s is the one nearest to max|x| / 6 and each element goes to the
// value nearest to x / s. A border between two values (0.25, 0.75, 1.25 .. 5) times s has at most 7 significant bits and x has
// 8, so x / s is a border or at least 2^-8 of itself from one. x times the rounded 1 / s, rounded to a multiple of 2^-11 by
// adding 6144 and taking it off again, is a border just where x / s is one, and on the same side of it elsewhere.
//
// Bound by memory: 2 * dim bytes read (written) and dim + 1, 9 / 16 * dim or 2 * dim written (read) for each row, K and V. A
// CTA takes up to 64 consecutive tokens, all heads, K and V: their places are looked up once, in shared memory where all
// sequences fit there (8294 e4m3 tokens x 8 heads written and read back 26.6 -> 20.1 us, 38 k read 40.7 -> 37.6), else by 16
// to 4 lanes a token; what a thread computes of an address serves a row of K and one of V. 4-bit rows: a thread has two pairs
// of rows on their way when it writes, four when it reads (8294 tokens written and read back 19.2 us, one pair and lookups
// as for many sequences 28.4).
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace {

constexpr int kThreads = 256;

constexpr int kTokens = 64;   // of a CTA, at most
constexpr int kResident = 4;  // CTAs of an SM
struct MoveArgs {
  PagedArgs c;
  RowsArgs k, v;
  const int32_t* cu;
  int n_rows, tokens, look_lanes;  // tokens of a CTA, threads that look one of them up
  bool wide;                       // all bf16 rows start on a multiple of 32 bytes
  unsigned int* err;
};

// 32 bytes at once where they start on a multiple of 32: whole sectors, which two halves in turn ask for twice (e4m3 rows of
// 38 k tokens x 8 heads read 46.8 -> 41.0 us, 8294 tokens written and read back 27.6 -> 24.5)
MV_DEV void load32(const uint8_t* p, uint32_t (&x)[8], bool wide) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                 : "l"(p));
    return;
  }
  const uint4 lo = reinterpret_cast<const uint4*>(p)[0], hi = reinterpret_cast<const uint4*>(p)[1];
  const uint32_t both[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = both[j];
}
MV_DEV void store32(uint8_t* p, const uint32_t (&x)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "l"(p)
                 : "memory");
    return;
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
}

// The page and slot of position `pos` of sequence b, page -2 for one outside the pool
MV_DEV int2 slot_of(const MoveArgs& a, int b, int pos) {
  const int nth = pos / a.c.page_size, page = __ldcg(a.c.table + (int64_t)b * a.c.ld_table + nth);
  return page < 0 || page >= a.c.n_pages ? make_int2(-2, 0) : make_int2(page, pos - nth * a.c.page_size);
}

// Where token t of the packed rows lies: page and slot; page -1 for a row behind the last sequence, -2 when the table,
// the lengths or cu are out of range. By n = 2^k consecutive lanes, which narrow the sequences down to an n-th at a time.
MV_DEV int2 place_of(const MoveArgs& a, int t, int n) {
  const int lane = threadIdx.x & (n - 1), first = threadIdx.x & 31 & ~(n - 1), n_seq = a.c.n_seq;
  const unsigned int mask = ((1u << n) - 1u) << first;  // n <= 16
  const int end = __ldcg(a.cu + n_seq);
  int lo = 0, hi = n_seq;  // the last b in [lo, hi) with cu[b] <= t, where cu does not decrease
  while (hi - lo > 1) {
    const int step = (hi - lo + n - 1) / n, at = lo + lane * step;
    const bool le = at < hi && __ldcg(a.cu + at) <= t;
    const unsigned int all = __ballot_sync(mask, le) & mask;
    if (all) lo += (31 - __clz(all) - first) * step;
    hi = all ? min(hi, lo + step) : lo + 1;
  }
  const int c0 = __ldcg(a.cu + lo), c1 = __ldcg(a.cu + lo + 1), len = __ldcg(a.c.seq_lens + lo);
  if (t >= end) return make_int2(-1, 0);
  if (c0 < 0 || t < c0 || t >= c1) return make_int2(-2, 0);
  const int64_t pos = (int64_t)len - c1 + t;
  // a length over the table's is refused with all its rows, those too that would have a place
  if (len < c1 - c0 || pos < 0 || len > a.c.max_pages * a.c.page_size) return make_int2(-2, 0);
  return slot_of(a, lo, (int)pos);
}

// The same with cu and the lengths in shared memory
MV_DEV int2 place_in(const MoveArgs& a, int t, const int* cu, const int* lens) {
  const int n_seq = a.c.n_seq;
  int lo = 0, hi = n_seq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int c0 = cu[lo], c1 = cu[lo + 1], len = lens[lo];
  if (t >= cu[n_seq]) return make_int2(-1, 0);
  const int64_t pos = (int64_t)len - c1 + t;
  if (c0 < 0 || t < c0 || t >= c1 || len < c1 - c0 || pos < 0 || len > a.c.max_pages * a.c.page_size) return make_int2(-2, 0);
  return slot_of(a, lo, (int)pos);
}

// A group's 16 bf16 as 4-bit values and their scale byte
MV_DEV uint2 quantise(const uint32_t (&x)[8], uint32_t& byte) {
  uint32_t top = 0u;  // without the sign, bf16 bits are ordered as their values are, NaN above infinity
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, x[j] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  const bool finite = top < 0x7f80u;
  byte = finite ? scale_byte(__fdiv_rn(bf16lo(top), 6.0f)) : kNanScale;
  const float inv = byte && finite ? __fdiv_rn(1.0f, scale_value(byte)) : 0.0f;
  auto quotient = [&](float f) { return __fsub_rn(__fmaf_rn(f, inv, 6144.0f), 6144.0f); };
  uint32_t q[2] = {0u, 0u};
  if (finite)  // (an infinity or a NaN times zero would be no number)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j >> 1] |= float4_to_e2m1x4(quotient(bf16lo(x[2 * j])), quotient(bf16hi(x[2 * j])), quotient(bf16lo(x[2 * j + 1])),
                                    quotient(bf16hi(x[2 * j + 1]))) << (16 * (j & 1));
  return make_uint2(q[0], q[1]);
}
// and back
MV_DEV void dequantise(uint2 q, uint32_t byte, uint32_t (&x)[8]) {
  const float s = scale_value(byte);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t h[4];
    e2m1x8_to_half2(j ? q.y : q.x, h);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = half2_to_float2(h[k]);
      x[4 * j + k] = pack_bf16x2(f.x * s, f.y * s);
    }
  }
}

// The rows of nt tokens over a 4-bit pool: a thread has a group of 16 elements of a row of K and of V, of several rows at once.
template <bool kWrite, int kLanes>
MV_DEV void move_e2m1(const MoveArgs& a, const int2* s_place, int t0, int nt) {
  constexpr int kAhead = kWrite ? 2 : 4;  // pairs of rows
  constexpr int kGroups = kThreads / kLanes;
  const int ln = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int H = a.c.heads, D = a.c.dim, P = a.c.page_size, pairs = nt * H, per_row = D / kGroup;
  const int n_fast = kWrite ? H : nt, add_slow = kGroups / n_fast, add_fast = kGroups % n_fast;
  int slow = group / n_fast, fast = group - slow * n_fast;
  for (int r0 = group; r0 < pairs; r0 += kAhead * kGroups) {
    int64_t held[kAhead];  // the group's number in the pool, -1: nothing to move
    int tok[kAhead], head[kAhead];
    uint32_t x[kAhead][2][kWrite ? 8 : 2], byte[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      tok[i] = kWrite ? slow : fast;
      head[i] = kWrite ? fast : slow;
      held[i] = -1;
      const int2 at = r0 + i * kGroups < pairs ? s_place[tok[i]] : make_int2(-1, 0);
      if (at.x >= 0 && ln < per_row) {
        held[i] = (((int64_t)at.x * H + head[i]) * P + at.y) * per_row + ln;
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
          if constexpr (kWrite) {
            const RowsArgs& p = is_v ? a.v : a.k;
            load32(reinterpret_cast<const uint8_t*>(p.p + (int64_t)(t0 + tok[i]) * p.ts + (int64_t)head[i] * p.hs + ln * kGroup),
                   x[i][is_v], a.wide);
          } else {
            const uint2 w = __ldcg(reinterpret_cast<const uint2*>((is_v ? a.c.v : a.c.k) + held[i] * 8));
            x[i][is_v][0] = w.x;
            x[i][is_v][1] = w.y;
            byte[i][is_v] = (is_v ? a.c.v_exp : a.c.k_exp)[held[i]];
          }
        }
      }
      slow += add_slow;
      fast += add_fast;
      if (fast >= n_fast) {
        fast -= n_fast;
        ++slow;
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (held[i] < 0) continue;
#pragma unroll
      for (int is_v = 0; is_v < 2; ++is_v) {
        if constexpr (kWrite) {
          uint32_t b;
          *reinterpret_cast<uint2*>((is_v ? a.c.v : a.c.k) + held[i] * 8) = quantise(x[i][is_v], b);
          (is_v ? a.c.v_exp : a.c.k_exp)[held[i]] = (uint8_t)b;
        } else {
          const RowsArgs& p = is_v ? a.v : a.k;
          uint32_t o[8];
          dequantise(make_uint2(x[i][is_v][0], x[i][is_v][1]), byte[i][is_v], o);
          store32(reinterpret_cast<uint8_t*>(p.p + (int64_t)(t0 + tok[i]) * p.ts + (int64_t)head[i] * p.hs + ln * kGroup), o,
                  a.wide);
        }
      }
    }
  }
}

// kLanes threads a row, the power of two from dim / kEl up
template <PagedFormat kFormat, bool kWrite, int kLanes>
__global__ void __launch_bounds__(kThreads, kResident) paged_rows_kernel(const MoveArgs a) {
  constexpr int kEl = 16;  // elements of a thread
  // Rows on their way, K and V in turn: as many as a thread's registers hold (8294 tokens x 8 heads written and read back:
  // bf16 with two 35 us, with four 26; e4m3 written with four 26.8, with two 24.9; 38 k e4m3 tokens read with two 43, with four 41)
  constexpr int kAhead = kFormat != kBf16 && kWrite ? 2 : 4;
  constexpr int kWords = kWrite || kFormat == kBf16 ? 8 : 4;
  __shared__ int2 s_place[kTokens];
  pdl_trigger();
  pdl_wait();
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.n_rows - t0);
  const bool few = a.c.n_seq < kThreads;
  __shared__ int s_cu[kThreads], s_lens[kThreads];
  if (few) {  // all sequences at once: two loads one after the other, with the table's, in place of four and more
    if ((int)threadIdx.x <= a.c.n_seq) s_cu[threadIdx.x] = __ldcg(a.cu + threadIdx.x);
    if ((int)threadIdx.x < a.c.n_seq) s_lens[threadIdx.x] = __ldcg(a.c.seq_lens + threadIdx.x);
    __syncthreads();
    if ((int)threadIdx.x < nt) {
      const int2 at = place_in(a, t0 + threadIdx.x, s_cu, s_lens);
      if (at.x == -2) mv_set_error_detail(a.err, kPagedRowsSite, MV_DEVERR_INDEX, (uint32_t)(t0 + threadIdx.x));
      s_place[threadIdx.x] = at;
    }
  } else {
    const int i = threadIdx.x / a.look_lanes;
    if (i < nt) {
      const int2 at = place_of(a, t0 + i, a.look_lanes);
      if ((threadIdx.x & (a.look_lanes - 1)) == 0) {
        if (at.x == -2) mv_set_error_detail(a.err, kPagedRowsSite, MV_DEVERR_INDEX, (uint32_t)(t0 + i));
        s_place[i] = at;
      }
    }
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.c.n_seq; b += kThreads) {
      const int c0 = __ldcg(a.cu + b), c1 = __ldcg(a.cu + b + 1);
      if ((b == 0 && c0 != 0) || c1 < c0 || c1 > a.n_rows)
        mv_set_error_detail(a.err, kPagedRowsSite, MV_DEVERR_INDEX, (uint32_t)b);
    }
  __syncthreads();
  constexpr int kGroups = kThreads / kLanes;                           // rows at a time
  const int ln = threadIdx.x % kLanes, group = threadIdx.x / kLanes, d0 = ln * kEl;  // elements d0 .. of a row
  const int H = a.c.heads, D = a.c.dim, P = a.c.page_size;
  const int pairs = nt * H;  // a row of K and one of V, which lie at the same place of the two pools
  if constexpr (kFormat == kE2M1) {
    move_e2m1<kWrite, kLanes>(a, s_place, t0, nt);
    return;
  }
  // The order of the rows is the source's: heads, then tokens of the caller's; tokens, then heads of the pool's
  const int n_fast = kWrite ? H : nt, add_slow = kGroups / n_fast, add_fast = kGroups % n_fast;
  int slow = group / n_fast, fast = group - slow * n_fast;
  for (int r0 = group; r0 < pairs; r0 += kAhead / 2 * kGroups) {  // the lanes of a group stay together
    uint8_t *to[kAhead], *exp[kAhead];                            // null: nothing to move
    uint32_t x[kAhead][kWords], byte[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i += 2) {
      to[i] = to[i + 1] = nullptr;
#pragma unroll
      for (int j = 0; j < kWords; ++j) x[i][j] = x[i + 1][j] = 0u;
      const int tok = kWrite ? slow : fast, h = kWrite ? fast : slow;
      const int2 at = r0 + i / 2 * kGroups < pairs ? s_place[tok] : make_int2(-1, 0);
      if (at.x >= 0 && d0 < D) {
        const int64_t prow = ((int64_t)at.x * H + h) * P + at.y;
        const int64_t held_at = (prow * D + d0) * (kFormat == kE4M3 ? 1 : 2);
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
          const RowsArgs& p = is_v ? a.v : a.k;
          uint8_t* row = reinterpret_cast<uint8_t*>(p.p + (int64_t)(t0 + tok) * p.ts + (int64_t)h * p.hs + d0);
          uint8_t* held = (is_v ? a.c.v : a.c.k) + held_at;
          to[i + is_v] = kWrite ? held : row;
          if (kFormat != kBf16) exp[i + is_v] = (is_v ? a.c.v_exp : a.c.k_exp) + prow;
          const uint8_t* from = kWrite ? row : held;
          if constexpr (kWords == 8) {
            load32(from, x[i + is_v], a.wide);
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(from);
            x[i + is_v][0] = w.x;
            x[i + is_v][1] = w.y;
            x[i + is_v][2] = w.z;
            x[i + is_v][3] = w.w;
          }
          if (kFormat != kBf16 && !kWrite) byte[i + is_v] = *exp[i + is_v];
        }
      }
      slow += add_slow;
      fast += add_fast;
      if (fast >= n_fast) {
        fast -= n_fast;
        ++slow;
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if constexpr (kFormat == kBf16) {
        if (to[i]) store32(to[i], x[i], a.wide);
      } else if constexpr (kWrite) {
        float f[16], top = 0.0f;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          f[(2 * j) & 15] = bf16lo(x[i][j]);
          f[(2 * j + 1) & 15] = bf16hi(x[i][j]);
          top = fmaxf(top, fmaxf(fabsf(f[(2 * j) & 15]), fabsf(f[(2 * j + 1) & 15])));  // a NaN does not count
        }
        // groups of one warp may have left the loop: a mask of this group's lanes
        const unsigned int mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
#pragma unroll
        for (int o = kLanes >> 1; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
        const uint32_t b = __float_as_uint(top);
        const int e = max(-100, min(120, (int)(b >> 23) - 135 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0)));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          q[j] = float2_to_e4m3x2(f[4 * j] * inv, f[4 * j + 1] * inv) |
                 ((uint32_t)float2_to_e4m3x2(f[4 * j + 2] * inv, f[4 * j + 3] * inv) << 16);
        if (to[i]) {
          *reinterpret_cast<uint4*>(to[i]) = make_uint4(q[0], q[1], q[2], q[3]);
          if (ln == 0) *exp[i] = (uint8_t)(e + 127);
        }
      } else if (to[i]) {
        const float s = exp_byte_scale(byte[i]);
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 f = half2_to_float2(e4m3x2_to_half2((uint16_t)(x[i][j >> 1] >> (16 * (j & 1)))));
          o[j] = pack_bf16x2(f.x * s, f.y * s);
        }
        store32(to[i], o, a.wide);
      }
    }
  }
}

template <PagedFormat kFormat, bool kWrite>
cudaError_t launch_rows(const MoveArgs& a, dim3 grid, cudaStream_t st) {
  constexpr int kMost = 8;
  if (a.c.dim > 64) return mv_launch(paged_rows_kernel<kFormat, kWrite, kMost>, grid, dim3(kThreads), 0, st, a);
  if (a.c.dim > 32) return mv_launch(paged_rows_kernel<kFormat, kWrite, kMost / 2>, grid, dim3(kThreads), 0, st, a);
  return mv_launch(paged_rows_kernel<kFormat, kWrite, kMost / 4>, grid, dim3(kThreads), 0, st, a);
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
  const auto whole = [](const mv_rows& r) {
    return !((reinterpret_cast<uintptr_t>(r.ptr) | (uint64_t)r.token_stride * 2 | (uint64_t)r.head_stride * 2) & 31);
  };
  a.wide = whole(k) && whole(v) &&
           (cache->dtype != MV_DTYPE_BF16 ||
            !((reinterpret_cast<uintptr_t>(cache->k) | reinterpret_cast<uintptr_t>(cache->v)) & 31));
  a.n_rows = n_rows;
  // Whole waves of CTAs with as many tokens each as share one round of lookups, which nothing hides. Reads do better with
  // more and smaller CTAs (38 k tokens x 8 heads of 128: 41 us with up to 16, 43 with up to 32; x 32 heads: 142 with up to 8,
  // 147 with up to 16), down to two rounds of copies for each thread (23 k tokens x 4 heads of 64: 10 us with up to 64, 20
  // with up to 16). Writes do not (120 prompts 78 us with up to 64, 83 with up to 16).
  const int groups = kThreads / (a.c.dim > 64 ? 8 : a.c.dim > 32 ? 4 : 2);
  const int64_t ctas = kResident * mv_sm_count();
  const int64_t most = kWrite ? kTokens : std::max(8, std::min(kTokens, 4 * groups / a.c.heads));
  const int64_t waves = (n_rows + ctas * most - 1) / (ctas * most);
  a.tokens = (int)((n_rows + ctas * waves - 1) / (ctas * waves));
  a.look_lanes = 16;
  while (a.look_lanes * a.tokens > kThreads) a.look_lanes /= 2;
  a.err = mv_error_word();
  const dim3 grid((n_rows + a.tokens - 1) / a.tokens);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == MV_DTYPE_E4M3   ? launch_rows<kE4M3, kWrite>(a, grid, st)
                        : cache->dtype == MV_DTYPE_E2M1 ? launch_rows<kE2M1, kWrite>(a, grid, st)
                                                        : launch_rows<kBf16, kWrite>(a, grid, st);
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
