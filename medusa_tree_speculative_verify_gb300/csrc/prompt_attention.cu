// Causal attention over whole prompts packed in one call, and the plan that lays out its work.
//
// S = Q K^T and O += P V run as tcgen05.mma with S, P and O in tensor memory, 128 query rows by 128 keys at a time. A CTA
// takes two sub-tiles (128 tokens of one head each) of one prompt and kv head: with grouped heads two heads of the
// same tokens, else two neighbouring row blocks, so one copy of a K and V tile serves both and the products of one run
// while the other's softmax works. One thread owns one row: it reads the row of S, updates the running maximum, writes
// the weights as bf16 for the second product and sums them in fp32. The reference of the exponentials moves only when
// the row maximum has grown by more than 2^8; then the thread rescales its row of O in place. Weights are rounded to bf16
// since both operands of a product have one type; the sums stay in fp32.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "kernels.cuh"
#include "paged.cuh"
#include "tc.cuh"

struct mv_prompt_plan {
  int32_t n_seq, group, n_tokens;
  std::vector<int32_t> items;  // [n_items][4], see mv_prompt_plan_desc
  int32_t* d_items;
  int device;  // -1: made without a device
};

namespace {

constexpr int kRows = 128;  // query rows of a sub-tile, keys of a key tile
constexpr int kMaxItems = 1 << 22;
constexpr uint32_t kSite = 42;  // device error site

struct PromptArgs {
  RowsArgs q, k, v, out;
  const int4* items;
  int group, kv_heads, dim, head_outer;  // head_outer: bit 0, 1, 2: q, k, v have the head as the outermost dimension
  float scale_log2;
  unsigned int* err;
};

// Nonzero where one of the two bf16 of w is a NaN or an infinity (its exponent bits all set).
MV_DEV uint32_t special2(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// w with those replaced by zeros
MV_DEV uint32_t finite2(uint32_t w) {
  const uint32_t s = special2(w);
  return w & ~(((s >> 15) & 0x00010001u) * 0xffffu);
}

// Adds to o (elements d0 .. d0 + 31 of query row i) the NaNs and infinities of V that the row sees in the last key
// tiles of the CTA's two sub-tiles. Added once more they change nothing, so it does not matter which of them the
// products have met already.
MV_DEV void add_specials(const PromptArgs& a, float (&o)[32], int d0, int t0, int i, int kh, const int (&block)[2]) {
  for (int s = 0; s < 2; ++s)
    for (int j = block[s] * kRows; j < (block[s] + 1) * kRows && j <= i; ++j) {
      const uint16_t* v = a.v.p + (int64_t)(t0 + j) * a.v.ts + (int64_t)kh * a.v.hs + d0;
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        if (d0 + e >= a.dim) continue;
        const uint4 w = *reinterpret_cast<const uint4*>(v + e);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t sp = special2(u[h]);
          if (sp & 0x8000u) o[e + 2 * h] += bf16lo(u[h]);
          if (sp & 0x80000000u) o[e + 2 * h + 1] += bf16hi(u[h]);
        }
      }
    }
}

// Warps 0-15: softmax, of sub-tile warp / 8 and of keys 64 (warp / 4 % 2) .. of a tile, for the rows of TMEM's lanes
// 32 (warp % 4) ..; warp 16: products, warp 17: copies, warp 18 tells when both operands are there (19 fills up
// the warpgroup, whose registers go to the softmax)
constexpr int kSoftmaxWarps = 16, kThreads = 640;
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;  // 4 * 104 + 64 <= 5 * 96, what a block of 640 threads starts with
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleLog2 = 8.0f;  // move the exponent reference when the row maximum grows by more than this

// kDim: head_dim rounded up to 64 or 128 (the copies fill the rest with zeros). Shared memory from a 1024-byte aligned
// base: Q of both sub-tiles, then a ring of kRing tiles of 128 keys, K and V of a tile in turn; each as kDim / 64
// regions of [128 rows][64] bf16 with the 128-byte swizzle.
template <int kDim>
struct Layout {
  static constexpr int kHalves = kDim / 64;
  static constexpr int kRegion = kRows * 128;
  static constexpr int kTile = kHalves * kRegion;
  static constexpr int kRing = kDim == 128 ? 5 : 10;
  static constexpr int kKV = 2 * kTile;
  static constexpr int kRest = kKV + kRing * kTile;
  // Tensor memory: S of the two sub-tiles, their O, and P (bf16, two keys a column). With 128-wide heads all 512
  // columns are taken and P lies over the S that it is computed from.
  static constexpr uint32_t kColS = 0, kColO = 256;
  static constexpr uint32_t kColP = kDim == 128 ? 0 : 384, kPStep = kDim == 128 ? 128 : 64;
  // 64-wide heads: P has its own place, so S of the next tile may be computed as soon as this one's has been read
  static constexpr bool kEarly = kDim == 64;
  // 128-wide heads: P is handed over in two parts (keys 0-31 and 64-95 of a tile, then the rest), so that its product
  // starts while the second exponentials are taken: 345 -> 341 us for 8192 tokens; for 64-wide ones 259 -> 282
  static constexpr int kParts = kDim == 128 ? 2 : 1;
};

// What follows the tiles in shared memory.
struct Rest {
  uint64_t qfull, full[10], freed[8], sfull[2], sread[2], pfull[2][2], ofull[2], drain;
  uint32_t tmem;
  volatile int abort, special;
  float half[2][2][kRows];  // [sub-tile][half]: what the two threads of a row tell each other
};

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const PromptArgs a) {
  using Ly = Layout<kDim>;
  constexpr uint32_t kIdS = tc_idesc(kRows, false), kIdO = tc_idesc(kDim, true);
  // All of the shared memory is this array, which starts on a multiple of 1024 bytes then: there is no room to round up
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + Ly::kKV;
  Rest& sh = *reinterpret_cast<Rest*>(smem + Ly::kRest);
  uint64_t &qfull = sh.qfull, (&full)[10] = sh.full, (&freed)[8] = sh.freed, (&sfull)[2] = sh.sfull,
           (&sread)[2] = sh.sread, (&pfull)[2][2] = sh.pfull, (&ofull)[2] = sh.ofull, &drain = sh.drain;
  volatile int &s_abort = sh.abort, &s_special = sh.special;
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) mv_set_error(a.err, kSite, MV_DEVERR_INDEX);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  pdl_trigger();
  if (warp == kSoftmaxWarps + 1 && lane == 0) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  const int4 item = a.items[blockIdx.x / a.kv_heads];
  const int kh = blockIdx.x % a.kv_heads, t0 = item.x, len = item.y;
  int block[2], head[2], tiles[2];  // row block of 128 tokens, query head, key tiles (0: no such sub-tile)
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    block[s] = (item.z + s) / a.group;
    head[s] = kh * a.group + (item.z + s) % a.group;
    tiles[s] = block[s] * kRows < len ? block[s] + 1 : 0;
  }
  const int n_tiles = max(tiles[0], tiles[1]);

  auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head_outer, int h, int row) {
#pragma unroll
    for (int hb = 0; hb < Ly::kHalves; ++hb)
      tma_load_3d(dst + hb * Ly::kRegion, map, bar, hb * 64, head_outer ? row : h, head_outer ? h : row);
  };
  auto load_tile = [&](int n, int st) {  // K(0), V(0), K(1), V(1), ...
    mbar_arrive_expect_tx(&full[st], (uint32_t)Ly::kTile);
    load(ring + st * Ly::kTile, n & 1 ? &vmap : &kmap, &full[st], a.head_outer & (n & 1 ? 4 : 2), kh,
         t0 + (n >> 1) * kRows);
  };
  if (warp == kSoftmaxWarps + 1) {
    // the copies start while the rest of the CTA is being set up: Q, and as many tiles as there are places
    if (lane == 0) {
      mbar_init(&qfull, 1);
      for (int i = 0; i < Ly::kRing; ++i) mbar_init(&full[i], 1);
      mbar_fence_init();
      pdl_wait();
      mbar_arrive_expect_tx(&qfull, (uint32_t)((tiles[1] ? 2 : 1) * Ly::kTile));
      load(smem, &qmap, &qfull, a.head_outer & 1, head[0], t0 + block[0] * kRows);
      load_tile(0, 0);
      if (tiles[1]) load(smem + Ly::kTile, &qmap, &qfull, a.head_outer & 1, head[1], t0 + block[1] * kRows);
      for (int n = 1; n < min(Ly::kRing, 2 * n_tiles); ++n) load_tile(n, n);
    }
    __syncwarp();
  } else if (warp == kSoftmaxWarps) {
    tc_alloc(&sh.tmem, kTmemCols);
    tc_relinquish();
  } else if (tid == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(&freed[i], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sread[s], kSoftmaxWarps / 2 + 1);
      mbar_init(&pfull[s][0], kSoftmaxWarps / 2 + 1);
      mbar_init(&pfull[s][1], kSoftmaxWarps / 2);
      mbar_init(&ofull[s], 1);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    s_special = 0;
    mbar_fence_init();
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();

  // a bounded wait that also gives up once any other wait of this CTA has
  auto wait = [&](uint64_t* bar, int phase) {
    if (mbar_try_wait(bar, (uint32_t)(phase & 1))) return true;
    const uint64_t t_start = mv_globaltimer();
    while (!s_abort) {
      if (mbar_try_wait(bar, (uint32_t)(phase & 1))) return true;
      if (mv_globaltimer() - t_start > MV_WAIT_LIMIT_NS) s_abort = 1;
    }
    return false;
  };

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSoftmaxWarps + 1 && lane == 0) {
      // ---------------------------------------------------------------- copies (one thread)
      int n = min(Ly::kRing, 2 * n_tiles);  // those are on their way
      for (int st = 0; n < 2 * n_tiles; ++n, st = st + 1 == Ly::kRing ? 0 : st + 1) {
        // what was there: K(i) or V(i - 1), freed as the i-th (at most five are outstanding: eight barriers in turn)
        const int i = (n - Ly::kRing + 1) >> 1;
        if (!wait(&freed[i & 7], i >> 3)) break;
        load_tile(n, st);
      }
      // every copy has landed before the CTA may leave (they have, unless a wait gave up)
      if (s_abort) mbar_wait(&qfull, 0u);
      for (int i = max(0, n - Ly::kRing); i < n; ++i)
        if (!mbar_wait(&full[i % Ly::kRing], (uint32_t)((i / Ly::kRing) & 1))) break;
    } else if (warp == kSoftmaxWarps) {
      // ---------------------------------------------------------------- products (one warp, an elected lane issues)
      // S_s(j) = Q_s K(j)^T, O_s += P_s(j) V(j). S of the next tile goes right behind the P V that frees its place; the
      // products of one sub-tile run while the other one's softmax works. The tensor cores take only one or two products
      // ahead, so what this warp spends between them is lost: one wait for each sub-tile and tile (pfull: P is written and
      // K and V have come), nothing divided, no flag carried along. (A warp for each sub-tile interleaves the two chains
      // product by product: 550 us in place of 446 for 8192 tokens.)
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int n0 = __shfl_sync(0xffffffffu, tiles[0], 0), n1 = __shfl_sync(0xffffffffu, tiles[1], 0);
      const int n_all = max(n0, n1);
      const uint64_t q_desc = desc_kmajor(smem_u32(smem)), k_desc = desc_kmajor(smem_u32(ring)),
                     v_desc = desc_mnmajor(smem_u32(ring), (uint32_t)Ly::kRegion);
      auto mma_s = [&](int s, int at) {
        const uint64_t q = q_desc + (uint64_t)(s * (Ly::kTile >> 4)), k = k_desc + (uint64_t)(at * (Ly::kTile >> 4));
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kDim / 16; ++i)
            tc_mma_f16(tm + Ly::kColS + 128 * s, q + (uint64_t)(i / 4 * (Ly::kRegion >> 4) + i % 4 * 2),
                       k + (uint64_t)(i / 4 * (Ly::kRegion >> 4) + i % 4 * 2), kIdS, i ? 1u : 0u);
          tc_commit_to(&sfull[s]);
        }
      };
      auto mma_o = [&](int s, int at, bool first, int part) {
        const uint64_t v = v_desc + (uint64_t)(at * (Ly::kTile >> 4));
        if (elect_one()) {
#pragma unroll
          for (int e = 0; e < 8 / Ly::kParts; ++e) {  // 16 keys each
            const int i = Ly::kParts == 1 ? e : (e & 1) + 4 * (e >> 1) + 2 * part;
            tc_mma_f16_ta(tm + Ly::kColO + kDim * s, tm + Ly::kColP + Ly::kPStep * s + 8 * i,
                          v + (uint64_t)(i * (16 * 128 >> 4)), kIdO, first && i == 0 ? 0u : 1u);
          }
        }
      };
      wait(&qfull, 0);
      wait(&full[0], 0);
      __syncwarp();
      tc_after();
      if (n0) mma_s(0, 0);
      if (n1) mma_s(1, 0);
      if (elect_one()) tc_commit_to(&freed[0]);
      int v_at = 1, k_at = 2;  // places in the ring of V(j) and K(j + 1)
      for (int j = 0; j < n_all; ++j) {
        if (Ly::kEarly) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (j + 1 >= (s ? n1 : n0)) continue;
            wait(&sread[s], j);
            __syncwarp();
            tc_after();
            mma_s(s, k_at);
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int n = s ? n1 : n0;
          if (j >= n) continue;
#pragma unroll
          for (int part = 0; part < Ly::kParts; ++part) {
            wait(&pfull[s][part], j);
            __syncwarp();
            tc_after();
            mma_o(s, v_at, j == 0, part);
          }
          if (Ly::kEarly || j + 1 == n) {
            if (elect_one()) tc_commit_to(&ofull[s]);
          } else {
            mma_s(s, k_at);
          }
        }
        if (j + 1 < n_all && elect_one()) tc_commit_to(&freed[(j + 1) & 7]);
        v_at = v_at + 2 >= Ly::kRing ? v_at + 2 - Ly::kRing : v_at + 2;
        k_at = k_at + 2 >= Ly::kRing ? k_at + 2 - Ly::kRing : k_at + 2;
      }
      if (__any_sync(0xffffffffu, s_abort)) {  // every product issued finishes before the CTA's memory is let go
        if (elect_one()) tc_commit_to(&drain);
        mbar_wait(&drain, 0u);
      }
    } else if (warp == kSoftmaxWarps + 2 && lane == 0) {
      // ---------------------------------------------------------------- V(j) and K(j + 1) have come: the last arrival at pfull (sread)
      int st = 0, phase = 0;
      auto next = [&]() {
        if (++st == Ly::kRing) {
          st = 0;
          phase ^= 1;
        }
      };
      for (int j = 0; j < n_tiles; ++j) {
        next();
        wait(&full[st], phase);
        if (j + 1 < n_tiles) {
          next();
          wait(&full[st], phase);
        }
        for (int s = 0; s < 2; ++s) {
          if (j >= tiles[s]) continue;
          if (Ly::kEarly) {
            if (j > 0) wait(&sread[s], j - 1);  // not twice in one phase
            mbar_arrive(&sread[s]);
          }
          if (j > 0) wait(&pfull[s][0], j - 1);
          mbar_arrive(&pfull[s][0]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax: two threads for each query row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int s = warp >> 3, half = (warp >> 2) & 1, r = tid & (kRows - 1), n = tiles[s], i = block[s] * kRows + r;
    const int pair = 1 + (warp & 3) + 4 * s;  // named barrier of the two warps that share rows
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t at_s = lane_base + Ly::kColS + 128 * s + 64 * half;
    const uint32_t at_p = lane_base + Ly::kColP + Ly::kPStep * s + 32 * half;
    const uint32_t at_o = lane_base + Ly::kColO + kDim * s + kDim / 2 * half;  // this thread's half of the row's output
    // what both threads of a row put in, in either's hand
    // (the place is free again for the next tile: S of that comes after every warp's P of this)
    auto exchange = [&](float mine) {
      sh.half[s][half][r] = mine;
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
      return sh.half[s][half ^ 1][r];
    };
    float m_ref = -INFINITY, l = 0.0f;  // exponent reference (log2 domain, the same in both threads) and this half's sum
    for (int j = 0; j < n; ++j) {
      if (j == n - 1) {
        // The last tile holds keys after this row. Their weights are zero, but zero times a NaN or an infinity in V
        // is a NaN, so such elements become zeros here (usually there is none) and reach the rows that see them at
        // the end. A tile is looked through by each sub-tile that ends with it; what one of them has cleared the
        // other does not find, so the mark is the CTA's.
        wait(&full[(2 * j + 1) % Ly::kRing], (2 * j + 1) / Ly::kRing);
        uint4* v = reinterpret_cast<uint4*>(ring + (2 * j + 1) % Ly::kRing * Ly::kTile);
        uint32_t any = 0;
#pragma unroll 4
        for (int e = tid & (2 * kRows - 1); e < Ly::kTile / 16; e += 2 * kRows) {
          const uint4 w = v[e];
          any |= special2(w.x) | special2(w.y) | special2(w.z) | special2(w.w);
        }
        if (any) {
          s_special = 1;
          __threadfence_block();
          for (int e = tid & (2 * kRows - 1); e < Ly::kTile / 16; e += 2 * kRows) {
            const uint4 w = v[e];
            v[e] = make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      }
      wait(&sfull[s], j);
      __syncwarp();
      tc_after();
      float x[64];
      tc_ld64(at_s, x);
      if (Ly::kEarly) {
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sread[s]);
      }
      // the last tile: keys after the row's own are masked (warps whose rows see all of their 64 keys have nothing to do)
      if (j == n - 1 && 64 * half + 63 > (r & ~31)) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (64 * half + c > r) x[c] = -INFINITY;
      }
      float tops[4] = {x[0], x[1], x[2], x[3]};  // chains short enough to issue without waiting
#pragma unroll
      for (int c = 4; c < 64; c += 2) tops[(c >> 1) & 3] = fmaxf(tops[(c >> 1) & 3], fmaxf(x[c], x[c + 1]));
      float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      top = fmaxf(top, exchange(top));  // both have read their S: P may be written over it
      const float m_new = fmaxf(m_ref, top * a.scale_log2);
      const bool move = m_new > m_ref + kRescaleLog2 || (m_ref == -INFINITY && m_new > -INFINITY);
      // O of this sub-tile has to be at rest, and P be read: the last P V came before the S that was waited for, or is
      // waited for itself
      if (Ly::kEarly && j > 0) {
        wait(&ofull[s], j - 1);
        __syncwarp();
        tc_after();
      }
      if (j > 0 && __any_sync(0xffffffffu, move)) {
        const float f = move ? fast_exp2(m_ref - m_new) : 1.0f;
        l *= f;
#pragma unroll 1
        for (int c = 0; c < kDim / 2; c += 16) {  // seldom: a few registers at a time, the row of S stays in its own
          uint32_t o[16];
          tc_ld16u(at_o + c, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tc_st16u(at_o + c, o);
        }
      }
      if (move) m_ref = m_new;
      const float base = m_ref == -INFINITY ? 0.0f : m_ref;
      const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), base2 = pack2(-base, -base);
      uint64_t sums[4] = {};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 y = unpack2(fma2(pack2(x[32 * q + 2 * e], x[32 * q + 2 * e + 1]), scale2, base2));
          const float p0 = fast_exp2(y.x), p1 = fast_exp2(y.y);
          sums[e & 3] = add2(sums[e & 3], pack2(p0, p1));
          p[e] = pack_bf16x2(p0, p1);
        }
        tc_st16u(at_p + 16 * q, p);
        if (Ly::kParts == 2 || q == 1) {
          tc_wait_st();
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[s][Ly::kParts == 2 ? q : 0]);
        }
      }
      const float2 sum = unpack2(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])));
      l += sum.x + sum.y;
    }
    if (n > 0) {
      wait(&ofull[s], Ly::kEarly ? n - 1 : 0);
      l += exchange(l);
      __syncwarp();
      tc_after();
      // The row, normalised, through the sub-tile's Q (every product with it is done) so that whole rows are stored by
      // neighbouring lanes: pieces of 16 bytes, their place within eight turned by the row.
      constexpr int kRowBytes = 2 * kDim, kPieces = kRowBytes / 16;
      uint8_t* stage = smem + s * Ly::kTile;
      const float inv = 1.0f / l;
      const bool special = s_special;
#pragma unroll
      for (int c = 0; c < kDim / 64; ++c) {
        const int d0 = kDim / 2 * half + 32 * c;
        float o[32];
        tc_ld32(at_o + 32 * c, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
        if (special && i < len) add_specials(a, o, d0, t0, i, kh, block);
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4*>(stage + r * kRowBytes + ((((d0 + e) >> 3) ^ (r & 7)) << 4)) =
              make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]), pack_bf16x2(o[e + 4], o[e + 5]),
                         pack_bf16x2(o[e + 6], o[e + 7]));
        __syncwarp();
      }
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");  // both halves of the 32 rows are there
      uint16_t* out = a.out.p + (int64_t)(t0 + block[s] * kRows) * a.out.ts + (int64_t)head[s] * a.out.hs;
      const int piece = lane & (kPieces - 1), rows_left = len - block[s] * kRows;
#pragma unroll
      for (int e = 0; e < 16; e += 32 / kPieces) {  // 16 of them by each warp
        const int row = (r & ~31) + 16 * half + e + lane / kPieces;
        const uint4 w = *reinterpret_cast<const uint4*>(stage + row * kRowBytes + ((piece ^ (row & 7)) << 4));
        if (row < rows_left && 8 * piece < a.dim) *reinterpret_cast<uint4*>(out + (int64_t)row * a.out.ts + 8 * piece) = w;
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (s_abort && tid == 0) mv_set_error(a.err, kSite, MV_DEVERR_TIMEOUT);
  if (warp == kSoftmaxWarps) tc_dealloc(tmem, kTmemCols);
}

template <int kDim>
mv_status launch(const CUtensorMap (&maps)[3], const PromptArgs& a, int64_t grid, cudaStream_t stream) {
  constexpr int kBytes = Layout<kDim>::kRest + (int)sizeof(Rest);
  static_assert(kBytes <= 227 * 1024 && Layout<kDim>::kRing <= 10, "shared memory of one CTA");
  static int flags[64] = {};
  if (!mv_set_smem_once((const void*)prompt_attn_kernel<kDim>, kBytes, flags)) return MV_ERR_CUDA;
  // the warpgroups' shares come out of the registers that the block starts with: never launch with fewer
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, prompt_attn_kernel<kDim>) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs * kThreads < 128 * (kSoftmaxWarps / 4 * kSoftmaxRegs + kOtherRegs)) return MV_ERR_UNSUPPORTED;
  const cudaError_t e = mv_launch(prompt_attn_kernel<kDim>, dim3((unsigned)grid), dim3(kThreads), kBytes,
                                  stream, maps[0], maps[1], maps[2], a);
  return e == cudaSuccess ? mv_last_launch("prompt_attention") : MV_ERR_CUDA;
}

// bf16 rows as boxes of 64 elements x one head x 128 tokens; the dimension with the larger stride is the outer one.
bool rows_map(CUtensorMap* map, const mv_rows& r, int64_t tokens, int heads, int dim, bool* head_major) {
  const uint64_t least = (uint64_t)dim * 2;  // the stride of a dimension of one
  const uint64_t ts = tokens > 1 ? (uint64_t)r.token_stride * 2 : least;
  const uint64_t hs = heads > 1 ? (uint64_t)r.head_stride * 2 : least;
  *head_major = hs > ts;
  const uint64_t dims[3] = {(uint64_t)dim, (uint64_t)(*head_major ? tokens : heads),
                            (uint64_t)(*head_major ? heads : tokens)};
  const uint64_t strides[2] = {*head_major ? ts : hs, *head_major ? hs : ts};
  const uint32_t box[3] = {64, *head_major ? (uint32_t)kRows : 1u, *head_major ? 1u : (uint32_t)kRows};
  return mv_encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

extern "C" mv_status mv_prompt_plan_create(const int32_t* lens, int32_t n_seq, int32_t group, mv_prompt_plan** out) {
  if (!out) return MV_ERR_INVALID_ARG;
  *out = nullptr;
  if (n_seq < 0 || (n_seq > 0 && !lens) || group < 1) return MV_ERR_INVALID_ARG;
  if (group > kPagedMaxHeads) return MV_ERR_SHAPE;
  int64_t tokens = 0, n_items = 0;
  for (int32_t b = 0; b < n_seq; ++b) {
    if (lens[b] < 0) return MV_ERR_INVALID_ARG;
    tokens += lens[b];
    n_items += (((int64_t)lens[b] + kRows - 1) / kRows * group + 1) / 2;
    if (tokens > 0x7fffffff - kRows || n_items > kMaxItems) return MV_ERR_SHAPE;
  }
  mv_prompt_plan* p = new (std::nothrow) mv_prompt_plan();
  if (!p) return MV_ERR_CAPACITY;
  p->n_seq = n_seq;
  p->group = group;
  p->n_tokens = (int32_t)tokens;
  p->d_items = nullptr;
  p->device = -1;
  try {
    struct Item {
      int32_t start, len, tile, keys;
    };
    std::vector<Item> v;
    v.reserve((size_t)n_items);
    int32_t start = 0;
    for (int32_t b = 0; b < n_seq; ++b) {
      const int64_t tiles = ((int64_t)lens[b] + kRows - 1) / kRows * group;
      for (int64_t t = 0; t < tiles; t += 2)  // the key tiles of the later one of the two: its row block and before
        v.push_back({start, lens[b], (int32_t)t, (int32_t)(std::min(t + 1, tiles - 1) / group) + 1});
      start += lens[b];
    }
    // longest first: the short items fill the gaps at the end
    std::stable_sort(v.begin(), v.end(), [](const Item& x, const Item& y) { return x.keys > y.keys; });
    p->items.reserve(v.size() * 4);
    for (const Item& i : v) p->items.insert(p->items.end(), {i.start, i.len, i.tile, i.keys});
  } catch (const std::bad_alloc&) {
    delete p;
    return MV_ERR_CAPACITY;
  }
  int n_dev = 0;
  if (cudaGetDeviceCount(&n_dev) != cudaSuccess || n_dev == 0) {
    cudaGetLastError();
    *out = p;
    return MV_OK;
  }
  mv_status s = MV_OK;
  if (cudaGetDevice(&p->device) != cudaSuccess) s = MV_ERR_CUDA;
  if (s == MV_OK && !p->items.empty()) {
    const size_t bytes = p->items.size() * sizeof(int32_t);
    const cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&p->d_items), bytes);
    if (e != cudaSuccess) {
      cudaGetLastError();
      s = e == cudaErrorMemoryAllocation ? MV_ERR_CAPACITY : MV_ERR_CUDA;
    } else if (cudaMemcpy(p->d_items, p->items.data(), bytes, cudaMemcpyHostToDevice) != cudaSuccess) {
      cudaGetLastError();
      s = MV_ERR_CUDA;
    }
  }
  if (s != MV_OK) {
    mv_prompt_plan_destroy(p);
    return s;
  }
  *out = p;
  return MV_OK;
}

extern "C" mv_status mv_prompt_plan_describe(const mv_prompt_plan* p, mv_prompt_plan_desc* d) {
  if (!p || !d) return MV_ERR_INVALID_ARG;
  d->n_seq = p->n_seq;
  d->group = p->group;
  d->n_tokens = p->n_tokens;
  d->n_items = (int32_t)(p->items.size() / 4);
  d->items = p->items.data();
  return MV_OK;
}

extern "C" void mv_prompt_plan_destroy(mv_prompt_plan* p) {
  if (!p) return;
  cudaFree(p->d_items);
  delete p;
}

extern "C" mv_status prompt_attention(mv_rows q, mv_rows k, mv_rows v, int32_t n_heads, int32_t n_kv_heads,
                                      int32_t head_dim, const mv_prompt_plan* plan, float scale, mv_rows out,
                                      mv_stream stream) {
  if (!plan || !(scale >= 0.0f && scale < INFINITY)) return MV_ERR_INVALID_ARG;
  if (n_kv_heads < 1 || n_heads < 1 || n_heads > kPagedMaxHeads || (int64_t)n_kv_heads * plan->group != n_heads)
    return MV_ERR_SHAPE;
  if (head_dim < 8 || head_dim > kPagedMaxDim || head_dim % 8) return MV_ERR_SHAPE;
  if (plan->n_tokens == 0) return MV_OK;
  const int64_t T = plan->n_tokens;
  if (!mv_rows_ok(q, T, n_heads, head_dim) || !mv_rows_ok(k, T, n_kv_heads, head_dim) ||
      !mv_rows_ok(v, T, n_kv_heads, head_dim) || !mv_out_rows_ok(out, T, n_heads, head_dim))
    return MV_ERR_INVALID_ARG;
  if (plan->device < 0) return MV_ERR_CUDA;
  if (plan->device != mv_device()) return MV_ERR_INVALID_ARG;
  PromptArgs a;
  a.q = {static_cast<uint16_t*>(q.ptr), q.token_stride, q.head_stride};
  a.k = {static_cast<uint16_t*>(k.ptr), k.token_stride, k.head_stride};
  a.v = {static_cast<uint16_t*>(v.ptr), v.token_stride, v.head_stride};
  a.out = {static_cast<uint16_t*>(out.ptr), out.token_stride, out.head_stride};
  a.items = reinterpret_cast<const int4*>(plan->d_items);
  a.group = plan->group;
  a.kv_heads = n_kv_heads;
  a.dim = head_dim;
  // a masked score is -inf: with a scale of zero the smallest weight in the exponent keeps -inf * scale what it is
  a.scale_log2 = fmaxf(scale * 1.4426950408889634f, 1e-30f);
  a.err = mv_error_word();
  const int64_t grid = (int64_t)(plan->items.size() / 4) * n_kv_heads;  // at most 2^22 * 2^8
  CUtensorMap maps[3];
  bool hm[3];
  if (!rows_map(&maps[0], q, T, n_heads, head_dim, &hm[0]) || !rows_map(&maps[1], k, T, n_kv_heads, head_dim, &hm[1]) ||
      !rows_map(&maps[2], v, T, n_kv_heads, head_dim, &hm[2]))
    return MV_ERR_CUDA;
  a.head_outer = (hm[0] ? 1 : 0) | (hm[1] ? 2 : 0) | (hm[2] ? 4 : 0);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return head_dim <= 64 ? launch<64>(maps, a, grid, st) : launch<128>(maps, a, grid, st);
}
