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
  int group, kv_heads, dim, head_major;
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

constexpr int kThreads = 320;  // warps 0-3 and 4-7: softmax of sub-tile 0 and 1; warp 8: products; warp 9: copies
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
  static constexpr int kBytes = kKV + kRing * kTile + 1024;
  static_assert(kBytes <= 230 * 1024, "shared memory of one CTA");
  // Tensor memory: S of the two sub-tiles, their O, and P (bf16, two keys a column). With 128-wide heads all 512
  // columns are taken and P lies over the S that it is computed from.
  static constexpr uint32_t kColS = 0, kColO = 256;
  static constexpr uint32_t kColP = kDim == 128 ? 0 : 384, kPStep = kDim == 128 ? 128 : 64;
};

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const PromptArgs a) {
  using Ly = Layout<kDim>;
  constexpr uint32_t kIdS = tc_idesc(kRows, false), kIdO = tc_idesc(kDim, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + Ly::kKV;
  __shared__ __align__(8) uint64_t qfull, full[Ly::kRing], empty[Ly::kRing], sfull[2], pfull[2], ofull[2], drain;
  __shared__ uint32_t tmem_sh;
  __shared__ volatile int s_abort, s_special;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

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

  if (tid == 0) {
    mbar_init(&qfull, 1);
    for (int i = 0; i < Ly::kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[s], kRows);
      mbar_init(&ofull[s], 1);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    s_special = 0;
    mbar_fence_init();
  }
  if (warp == 8) {
    tc_alloc(&tmem_sh, kTmemCols);
    tc_relinquish();
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_sh;
  pdl_trigger();
  pdl_wait();

  // a bounded wait that gives up at once after any other wait of this CTA gave up
  auto wait = [&](uint64_t* bar, int phase) {
    if (s_abort) return false;
    if (mbar_wait(bar, (uint32_t)(phase & 1))) return true;
    s_abort = 1;
    return false;
  };

  if (warp == 9) {
    // ------------------------------------------------------------------ copies (one thread)
    if (lane == 0) {
      const int c1 = a.head_major;  // bit 0, 1, 2: q, k, v have the head as the outermost dimension
      auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int hm, int h, int row) {
#pragma unroll
        for (int hb = 0; hb < Ly::kHalves; ++hb)
          tma_load_3d(dst + hb * Ly::kRegion, map, bar, hb * 64, hm ? row : h, hm ? h : row);
      };
      mbar_arrive_expect_tx(&qfull, (uint32_t)((tiles[1] ? 2 : 1) * Ly::kTile));
      load(smem, &qmap, &qfull, c1 & 1, head[0], t0 + block[0] * kRows);
      if (tiles[1]) load(smem + Ly::kTile, &qmap, &qfull, c1 & 1, head[1], t0 + block[1] * kRows);
      int n = 0;
      for (; n < 2 * n_tiles; ++n) {  // K of tile 0, V of tile 0, K of tile 1, ...
        const int st = n % Ly::kRing;
        if (n >= Ly::kRing && !wait(&empty[st], n / Ly::kRing - 1)) break;
        mbar_arrive_expect_tx(&full[st], (uint32_t)Ly::kTile);
        load(ring + st * Ly::kTile, n & 1 ? &vmap : &kmap, &full[st], n & 1 ? c1 & 4 : c1 & 2, kh, t0 + (n >> 1) * kRows);
      }
      // every copy has landed before the CTA may leave (they have, unless a wait gave up)
      if (s_abort) mbar_wait(&qfull, 0u);
      for (int i = max(0, n - Ly::kRing); i < n; ++i)
        if (!mbar_wait(&full[i % Ly::kRing], (uint32_t)((i / Ly::kRing) & 1))) break;
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ products (one thread)
    // S_s(j) = Q_s K(j)^T, O_s += P_s(j) V(j). S of the next tile goes right behind the P V that frees its place; the
    // products of one sub-tile run while the other one's softmax works.
    if (lane == 0) {
      auto mma_s = [&](int s, int j) {
        const uint32_t qb = smem_u32(smem) + s * Ly::kTile, kb = smem_u32(ring) + 2 * j % Ly::kRing * Ly::kTile;
#pragma unroll
        for (int hb = 0; hb < Ly::kHalves; ++hb)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_f16(tmem + Ly::kColS + 128 * s, desc_kmajor(qb + hb * Ly::kRegion) + (uint64_t)(2 * k),
                       desc_kmajor(kb + hb * Ly::kRegion) + (uint64_t)(2 * k), kIdS, (hb | k) ? 1u : 0u);
        tc_commit_to(&sfull[s]);
      };
      auto mma_o = [&](int s, int j) {
        const uint32_t vb = smem_u32(ring) + (2 * j + 1) % Ly::kRing * Ly::kTile;
#pragma unroll
        for (int k = 0; k < 8; ++k)  // 16 keys each
          tc_mma_f16_ta(tmem + Ly::kColO + kDim * s, tmem + Ly::kColP + Ly::kPStep * s + 8 * k,
                        desc_mnmajor(vb + (uint32_t)(16 * k * 128), (uint32_t)Ly::kRegion), kIdO,
                        (j > 0 || k > 0) ? 1u : 0u);
      };
      auto tile_in = [&](int n) { return wait(&full[n % Ly::kRing], n / Ly::kRing); };
      bool ok = wait(&qfull, 0) && tile_in(0);
      tc_after();
      if (ok)
        for (int s = 0; s < 2; ++s)
          if (tiles[s]) mma_s(s, 0);
      tc_commit_to(&empty[0]);
      for (int j = 0; ok && j < n_tiles; ++j) {
        ok = tile_in(2 * j + 1) && (j + 1 == n_tiles || tile_in(2 * j + 2));
        for (int s = 0; ok && s < 2; ++s) {
          if (j >= tiles[s]) continue;
          if (!(ok = wait(&pfull[s], j))) break;
          tc_after();
          mma_o(s, j);
          if (j + 1 < tiles[s]) mma_s(s, j + 1);
          else tc_commit_to(&ofull[s]);
        }
        if (!ok) break;
        tc_commit_to(&empty[(2 * j + 1) % Ly::kRing]);
        if (j + 1 < n_tiles) tc_commit_to(&empty[(2 * j + 2) % Ly::kRing]);
      }
      if (!ok) {  // every product issued finishes before the CTA's memory is let go
        mv_set_error(a.err, kSite, MV_DEVERR_TIMEOUT);
        tc_commit_to(&drain);
        mbar_wait(&drain, 0u);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax: one thread for each query row
    const int s = warp >> 2, r = tid & (kRows - 1), n = tiles[s], i = block[s] * kRows + r;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t at_s = lane_base + Ly::kColS + 128 * s, at_p = lane_base + Ly::kColP + Ly::kPStep * s,
                   at_o = lane_base + Ly::kColO + kDim * s;
    float m_ref = -INFINITY, l = 0.0f;  // exponent reference (log2 domain) and sum
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
        for (int e = r; e < Ly::kTile / 16; e += kRows) {
          const uint4 w = v[e];
          any |= special2(w.x) | special2(w.y) | special2(w.z) | special2(w.w);
        }
        if (any) {
          s_special = 1;
          __threadfence_block();
          for (int e = r; e < Ly::kTile / 16; e += kRows) {
            const uint4 w = v[e];
            v[e] = make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      }
      wait(&sfull[s], j);
      __syncwarp();
      tc_after();
      float x[kRows];
      tc_ld128(at_s, x);
      if (j == n - 1) {
#pragma unroll
        for (int c = 0; c < kRows; ++c)
          if (c > r) x[c] = -INFINITY;
      }
      float top = x[0];
#pragma unroll
      for (int c = 1; c < kRows; ++c) top = fmaxf(top, x[c]);
      const float m_new = fmaxf(m_ref, top * a.scale_log2);
      const bool move = m_new > m_ref + kRescaleLog2 || (m_ref == -INFINITY && m_new > -INFINITY);
      // O of this sub-tile is at rest: its last P V came before the S that was waited for
      if (j > 0 && __any_sync(0xffffffffu, move)) {
        const float f = move ? fast_exp2(m_ref - m_new) : 1.0f;
        l *= f;
#pragma unroll
        for (int c = 0; c < kDim / 32; ++c) {
          float o[32];
          tc_ld32(at_o + 32 * c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          tc_st32(at_o + 32 * c, o);
        }
      }
      if (move) m_ref = m_new;
      const float base = m_ref == -INFINITY ? 0.0f : m_ref;
      float sum = 0.0f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float p0 = fast_exp2(fmaf(x[64 * half + 2 * e], a.scale_log2, -base));
          const float p1 = fast_exp2(fmaf(x[64 * half + 2 * e + 1], a.scale_log2, -base));
          sum += p0 + p1;
          p[e] = pack_bf16x2(p0, p1);
        }
        tc_st32u(at_p + 32 * half, p);
      }
      l += sum;
      tc_wait_st();
      tc_before();
      mbar_arrive(&pfull[s]);
    }
    if (n > 0) {
      const bool live = wait(&ofull[s], 0) && i < len;
      __syncwarp();
      tc_after();
      const float inv = 1.0f / l;
      uint16_t* row = a.out.p + (int64_t)(t0 + i) * a.out.ts + (int64_t)head[s] * a.out.hs;
      const bool special = s_special;
#pragma unroll
      for (int c = 0; c < kDim / 32; ++c) {
        float o[32];
        tc_ld32(at_o + 32 * c, o);
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          if (special) add_specials(a, o, 32 * c, t0, i, kh, block);
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            if (32 * c + e < a.dim)
              *reinterpret_cast<uint4*>(row + 32 * c + e) =
                  make_uint4(pack_bf16x2(o[e], o[e + 1]), pack_bf16x2(o[e + 2], o[e + 3]),
                             pack_bf16x2(o[e + 4], o[e + 5]), pack_bf16x2(o[e + 6], o[e + 7]));
        }
        __syncwarp();
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (s_abort && tid == 0) mv_set_error(a.err, kSite, MV_DEVERR_TIMEOUT);
  if (warp == 8) tc_dealloc(tmem, kTmemCols);
}

template <int kDim>
mv_status launch(const CUtensorMap (&maps)[3], const PromptArgs& a, int64_t grid, cudaStream_t stream) {
  static int flags[64] = {};
  if (!mv_set_smem_once((const void*)prompt_attn_kernel<kDim>, Layout<kDim>::kBytes, flags)) return MV_ERR_CUDA;
  const cudaError_t e = mv_launch(prompt_attn_kernel<kDim>, dim3((unsigned)grid), dim3(kThreads), Layout<kDim>::kBytes,
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
  a.head_major = (hm[0] ? 1 : 0) | (hm[1] ? 2 : 0) | (hm[2] ? 4 : 0);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return head_dim <= 64 ? launch<64>(maps, a, grid, st) : launch<128>(maps, a, grid, st);
}
