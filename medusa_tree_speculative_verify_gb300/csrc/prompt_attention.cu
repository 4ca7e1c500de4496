// Causal attention over whole prompts packed in one call, and the plan that lays out its work.
//
// S = Q K^T and O += P V run as tcgen05.mma with S, P and O in tensor memory, 128 query rows by 128 keys at a time. A CTA
// takes two sub-tiles (128 tokens of one head each) of one prompt and kv head: with grouped heads two heads of the
// same tokens, else two neighbouring row blocks, so one copy of a K and V tile serves both and the products of one run
// while the other's softmax works. Two threads own a row, 64 keys of a tile each: they read S, update the running maximum
// together, write the weights as bf16 for the second product and sum them in fp32. The reference of the exponentials moves
// only when the row maximum has grown by more than 2^8; then they rescale their row of O in place. Weights are rounded to
// bf16 since both operands of a product have one type; the sums stay in fp32.
//
// 8192 tokens of 32 heads of 128 over 8: 312 us, 1.76 PFLOP/s, in a burst (344 us once the power cap acts); of 64: 245 us, 1.12
// PFLOP/s. With 128-wide heads the products, their issue and the softmax's chain (read S, maximum, exponentials, write P) bound
// it alike. With 64-wide ones nothing is near full (tensor cores 41 % of the cycles, exponentials' pipe 42 %, issue 61 %): it is
// that chain's latency, with a barrier between the two threads of a row, and its six instructions a score, for half the
// products. Short prompts (24 of up to 300 tokens, 32 heads: 19 us) are bound by the chain too, two or three tiles in a row an item.
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
// tiles of the item's two sub-tiles. Added once more they change nothing, so it does not matter which of them the
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
// 32 (warp % 4) ..; warp 16: products, warp 17: copies, warp 18 tells when both operands are there, and looks
// through V (19 fills up the warpgroup, whose registers go to the softmax)
constexpr int kSoftmaxWarps = 16, kThreads = 640;
constexpr int kSoftmaxRegs = 104, kOtherRegs = 64;  // 4 * 104 + 64 <= 5 * 96, what a block of 640 threads starts with
constexpr uint32_t kTmemCols = 512;

// The descriptor d with its address moved on, in units of 16 bytes, within the field: one 32-bit addition (8192 tokens of
// 64-wide heads 250 -> 238 us when it came; what the issuing warp computes between products is lost)
MV_DEV uint64_t desc_plus(uint64_t d, uint32_t by) { return (d & 0xffffffff00000000ull) | (uint32_t)((uint32_t)d + by); }

constexpr float kRescaleLog2 = 8.0f;  // move the exponent reference when the row maximum grows by more than this
// From here on the reference's rounding is half an exponent and more: a row's scores are rounded like it before it is taken
// off, and brought back to what the multiplication below makes the difference of.
constexpr float kLargeLog2 = 0x1p22f;

// kDim: head_dim rounded up to 64 or 128 (the copies fill the rest with zeros). Shared memory from a 1024-byte aligned
// base: Q of both sub-tiles, then a ring of kRing tiles of 128 keys, K and V of a tile in turn; each as kDim / 64
// regions of [128 rows][64] bf16 with the 128-byte swizzle. Then 2 KB for each softmax warp, through which its output goes.
template <int kDim>
struct Layout {
  static constexpr int kHalves = kDim / 64;
  static constexpr int kRegion = kRows * 128;
  static constexpr int kTile = kHalves * kRegion;
  static constexpr int kRing = kDim == 128 ? 4 : 8;
  static constexpr int kKV = 2 * kTile;
  static constexpr int kStage = kKV + kRing * kTile, kRest = kStage + kSoftmaxWarps * 2048;
  // Tensor memory: S of the two sub-tiles, their O, and P (bf16, two keys a column). With 128-wide heads all 512
  // columns are taken and P lies over the S that it is computed from.
  static constexpr uint32_t kColS = 0, kColO = 256;
  static constexpr uint32_t kColP = kDim == 128 ? 0 : 384, kPStep = kDim == 128 ? 128 : 64;
  // 64-wide heads: P has its own place, so S of the next tile may be computed as soon as this one's has been read
  static constexpr bool kEarly = kDim == 64;
  // 128-wide heads: P is handed over in two parts (keys 0-31 and 64-95 of a tile, then the rest), so that its product
  // starts while the second exponentials are taken: 345 -> 341 us for 8192 tokens; for 64-wide ones 259 -> 282
  static constexpr int kParts = kDim == 128 ? 2 : 1;
  static constexpr int kSlots = kEarly ? 2 : 1;  // see exchange
};

// Cluster launch control: asks for a block of this grid that has not started yet, which then will not start; the answer
// (16 bytes, counted on `bar`) names it or says that there is none. After a "none" nothing more may be asked.
MV_DEV void clc_request(uint4* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// blockIdx.x of the block taken over, -1 for none
MV_DEV int clc_block(const uint4* answer) {
  uint32_t any, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\tld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(any), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // read before the next answer is written
  return any ? (int)x : -1;
}

// A work item of one kv head: two sub-tiles of a prompt.
struct Work {
  int t0, len, kh;                  // the prompt's first token and length, kv head
  int block[2], head[2], tiles[2];  // row block of 128 tokens, query head, key tiles (0: no such sub-tile)
  int n;                            // key tiles of the longer one; 0: there is no more work
};

// What follows the tiles in shared memory. kSlots: places for what the two threads of a row tell each other, used in turn.
template <int kSlots>
struct Rest {
  uint64_t qfull, qfree, full[8], freed[16], sfull[2], sread[2], pfull[2][2], ofull[2], drain;
  uint64_t wfull[2], wempty[2], cfull;
  uint4 cancel;   // the answer to a request for another block's work
  Work work[2];   // the CTA's items in turn
  int used[8];    // the event that frees each place of the ring
  uint32_t tmem;
  volatile int abort, special;
  float half[kSlots][2][2][kRows];  // [.][sub-tile][half]
};

// A block for each item, longest first; but a CTA that has an item's copies under way takes over the next block that has
// not started (cluster launch control), so that the SMs stay evenly loaded and no item waits for a CTA to be set up. The
// copying thread deals the items out; each role goes through them on its own, counting the barriers' phases on from item to
// item: while the softmax warps write an item's output, the next one's Q, K and V come and its first S is computed.
// With a CTA set up for each item 8192 tokens took 336 us (320 so), 12 prompts of up to 2048 tokens 57 (50), 24 of up to
// 300 28 (21).
template <int kDim>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const PromptArgs a) {
  using Ly = Layout<kDim>;
  constexpr uint32_t kIdS = tc_idesc(kRows, false), kIdO = tc_idesc(kDim, true);
  // All of the shared memory is this array, which starts on a multiple of 1024 bytes then: there is no room to round up
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + Ly::kKV;
  auto& sh = *reinterpret_cast<Rest<Ly::kSlots>*>(smem + Ly::kRest);
  volatile int &s_abort = sh.abort, &s_special = sh.special;
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) mv_set_error(a.err, kSite, MV_DEVERR_INDEX);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  pdl_trigger();
  if (warp == kSoftmaxWarps) {
    tc_alloc(&sh.tmem, kTmemCols);
    tc_relinquish();
  } else if (tid == 0) {
    mbar_init(&sh.qfull, 1);
    mbar_init(&sh.qfree, 1);
    for (int i = 0; i < Ly::kRing; ++i) mbar_init(&sh.full[i], 1);
    for (int i = 0; i < 16; ++i) mbar_init(&sh.freed[i], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.sfull[s], 1);
      mbar_init(&sh.sread[s], kSoftmaxWarps / 2 + 1);
      mbar_init(&sh.pfull[s][0], kSoftmaxWarps / 2 + 1);
      mbar_init(&sh.pfull[s][1], kSoftmaxWarps / 2);
      mbar_init(&sh.ofull[s], 1);
      mbar_init(&sh.wfull[s], 1);
      mbar_init(&sh.wempty[s], kSoftmaxWarps + 2);
    }
    mbar_init(&sh.drain, 1);
    mbar_init(&sh.cfull, 1);
    s_abort = 0;
    s_special = 0;
    mbar_fence_init();
  } else if (warp == kSoftmaxWarps + 1 && lane == 0) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
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
  // The r-th item, or that there is none. The copying thread always ends the list, whatever was given up on, and within a few
  // time limits: all roles have to see the same items (the two warps of a row meet at barriers), so this waits on
  // regardless of the others, and counts attempts, which a CTA that is not running does not use up.
  auto work_in = [&](int r) -> const Work* {
    for (unsigned int i = 0; i < 1u << 30; ++i)
      if (mbar_try_wait(&sh.wfull[r & 1], (uint32_t)((r >> 1) & 1))) return sh.work[r & 1].n ? &sh.work[r & 1] : nullptr;
    s_abort = 1;
    return nullptr;
  };

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kSoftmaxWarps + 1 && lane == 0) {
      // ---------------------------------------------------------------- items and copies (one thread)
      // Tile g of the CTA (K(0), V(0), K(1), .. of its first item, then of the next) has place g % kRing of the ring. An item
      // frees its tiles in n + 1 events: K(0); V(j) and K(j + 1); V(n - 1). Event e is phase e / 16 of barrier e % 16: never
      // more than the ring's tiles are outstanding.
      int g = 0, event = 0, r = 0, q = 0;  // tiles, events, items, copies of Q so far
      for (int next = (int)blockIdx.x;; ++r) {
        Work w = {};
        if (next >= 0) {
          const int4 item = a.items[next / a.kv_heads];
          w.kh = next % a.kv_heads;
          w.t0 = item.x;
          w.len = item.y;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            w.block[s] = (item.z + s) / a.group;
            w.head[s] = w.kh * a.group + (item.z + s) % a.group;
            w.tiles[s] = w.block[s] * kRows < w.len ? w.block[s] + 1 : 0;
          }
          w.n = max(w.tiles[0], w.tiles[1]);
        }
        if (r >= 2) mbar_wait(&sh.wempty[r & 1], (uint32_t)(((r - 2) >> 1) & 1), 4 * MV_WAIT_LIMIT_NS);
        sh.work[r & 1] = w;
        mbar_arrive(&sh.wfull[r & 1]);
        if (next < 0) break;
        auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head_outer, int h, int row) {
#pragma unroll
          for (int hb = 0; hb < Ly::kHalves; ++hb)
            tma_load_3d(dst + hb * Ly::kRegion, map, bar, hb * 64, head_outer ? row : h, head_outer ? h : row);
        };
        next = -1;
        if (r > 0 && !wait(&sh.qfree, r - 1)) continue;
        ++q;
        mbar_arrive_expect_tx(&sh.qfull, (uint32_t)((w.tiles[1] ? 2 : 1) * Ly::kTile));
        load(smem, &qmap, &sh.qfull, a.head_outer & 1, w.head[0], w.t0 + w.block[0] * kRows);
        if (w.tiles[1]) load(smem + Ly::kTile, &qmap, &sh.qfull, a.head_outer & 1, w.head[1], w.t0 + w.block[1] * kRows);
        bool ok = true;
        for (int m = 0; m < 2 * w.n; ++m, ++g) {
          const int st = g & (Ly::kRing - 1);
          if (g >= Ly::kRing && !(ok = wait(&sh.freed[sh.used[st] & 15], sh.used[st] >> 4))) break;
          sh.used[st] = event + ((m + 1) >> 1);
          mbar_arrive_expect_tx(&sh.full[st], (uint32_t)Ly::kTile);
          load(ring + st * Ly::kTile, m & 1 ? &vmap : &kmap, &sh.full[st], a.head_outer & (m & 1 ? 4 : 2), w.kh,
               w.t0 + (m >> 1) * kRows);
        }
        event += w.n + 1;
        if (!ok) continue;
        mbar_arrive_expect_tx(&sh.cfull, 16);
        clc_request(&sh.cancel, &sh.cfull);
        if (mbar_wait(&sh.cfull, (uint32_t)(r & 1)))
          next = clc_block(&sh.cancel);
        else
          s_abort = 1;
      }
      if (s_abort) {  // every copy has landed before the CTA may leave (else they have)
        for (int i = max(0, g - Ly::kRing); i < g; ++i)
          if (!mbar_wait(&sh.full[i & (Ly::kRing - 1)], (uint32_t)((i / Ly::kRing) & 1))) break;
        if (q > 0) mbar_wait(&sh.qfull, (uint32_t)((q - 1) & 1));
      }
    } else if (warp == kSoftmaxWarps) {
      // ---------------------------------------------------------------- products (one warp, an elected lane issues)
      // S_s(j) = Q_s K(j)^T, O_s += P_s(j) V(j). S of the next tile goes right behind the P V that frees its place; the
      // products of one sub-tile run while the other one's softmax works. The tensor cores take only one or two products
      // ahead, so what this warp spends between them is lost: few waits (pfull: P is written and K and V have come),
      // nothing divided, no flag carried along. (A warp for each sub-tile interleaves the two chains product by product:
      // 550 us in place of 446 for 8192 tokens.) elect_one is for whole warps: only under conditions that all lanes share.
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = desc_kmajor(smem_u32(smem)), k_desc = desc_kmajor(smem_u32(ring)),
                     v_desc = desc_mnmajor(smem_u32(ring), (uint32_t)Ly::kRegion);
      auto mma_s = [&](int s, int at) {
        const uint64_t q = desc_plus(q_desc, s * (Ly::kTile >> 4)), k = desc_plus(k_desc, at * (Ly::kTile >> 4));
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kDim / 16; ++i)
            tc_mma_f16(tm + Ly::kColS + 128 * s, desc_plus(q, i / 4 * (Ly::kRegion >> 4) + i % 4 * 2),
                       desc_plus(k, i / 4 * (Ly::kRegion >> 4) + i % 4 * 2), kIdS, i ? 1u : 0u);
          tc_commit_to(&sh.sfull[s]);
        }
      };
      auto mma_o = [&](int s, int at, bool first, int part) {
        uint32_t col = tm;
        asm volatile("" : "+r"(col));  // taken anew each time: hoisted out of the loops these operands would spill
        const uint64_t v = desc_plus(v_desc, at * (Ly::kTile >> 4));
        if (elect_one()) {
#pragma unroll
          for (int e = 0; e < 8 / Ly::kParts; ++e) {  // 16 keys each
            const int i = Ly::kParts == 1 ? e : (e & 1) + 4 * (e >> 1) + 2 * part;
            tc_mma_f16_ta(col + Ly::kColO + kDim * s, col + Ly::kColP + Ly::kPStep * s + 8 * i,
                          desc_plus(v, i * (16 * 128 >> 4)), kIdO, first && i == 0 ? 0u : 1u);
          }
        }
      };
      auto wait_for = [&](uint64_t* bar, int phase) {
        wait(bar, phase);
        __syncwarp();
        tc_after();
      };
      int event = 0, tile = 0, c0 = 0, c1 = 0;  // next event and tile, tiles of each sub-tile in the items before
      for (int r = 0;; ++r) {
        const Work* w = work_in(r);
        if (!__any_sync(0xffffffffu, w != nullptr)) break;
        const int n0 = __shfl_sync(0xffffffffu, w->tiles[0], 0), n1 = __shfl_sync(0xffffffffu, w->tiles[1], 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.wempty[r & 1]);
        const int n_all = max(n0, n1);
        wait(&sh.qfull, r);
        wait_for(&sh.full[tile & (Ly::kRing - 1)], tile / Ly::kRing);
        mma_s(0, tile & (Ly::kRing - 1));
        if (n1) mma_s(1, tile & (Ly::kRing - 1));
        if (elect_one()) {
          tc_commit_to(&sh.freed[event & 15]);
          if (n_all == 1) tc_commit_to(&sh.qfree);
        }
        for (int j = 0; j < n_all; ++j) {
          const int v_at = (tile + 1) & (Ly::kRing - 1), k_at = (tile + 2) & (Ly::kRing - 1);
          tile += 2;
          ++event;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int n = s ? n1 : n0;
            if (j >= n) continue;
            if (Ly::kEarly && j + 1 < n) {
              wait_for(&sh.sread[s], (s ? c1 : c0) + j);
              mma_s(s, k_at);
            }
#pragma unroll
            for (int part = 0; part < Ly::kParts; ++part) {
              wait_for(&sh.pfull[s][part], (s ? c1 : c0) + j);
              mma_o(s, v_at, j == 0, part);
            }
            if (Ly::kEarly || j + 1 == n) {
              if (elect_one()) tc_commit_to(&sh.ofull[s]);
            } else {
              mma_s(s, k_at);
            }
          }
          if (elect_one()) {
            tc_commit_to(&sh.freed[event & 15]);
            if (j + 2 == n_all) tc_commit_to(&sh.qfree);  // the item's last S has been issued
          }
        }
        ++event;
        c0 += n0;
        c1 += n1;
      }
      // Every product issued, and with them the last commits' arrivals, are over before the CTA's memory is let go
      if (elect_one()) tc_commit_to(&sh.drain);
      mbar_wait(&sh.drain, 0u);
    } else if (warp == kSoftmaxWarps + 2) {
      // ---------------------------------------------------------------- V(j) and K(j + 1) have come: the last arrival at pfull (sread)
      // The last tile of a sub-tile holds keys after its rows. Their weights are zero, but zero times a NaN or an infinity
      // in V is a NaN, so such elements become zeros here (usually there is none), before any product of that tile, and
      // reach the rows that see them at the end. (One look for both sub-tiles, while their S is computed: by the softmax
      // warps themselves, behind the wait for S, 12 prompts of up to 2048 tokens take 51 us, 47 so.)
      int tile = 0, c[2] = {0, 0};
      for (int r = 0;; ++r) {
        const Work* w = work_in(r);
        if (!__any_sync(0xffffffffu, w != nullptr)) break;
        const int n[2] = {__shfl_sync(0xffffffffu, w->tiles[0], 0), __shfl_sync(0xffffffffu, w->tiles[1], 0)};
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.wempty[r & 1]);
        const int n_all = max(n[0], n[1]);
        for (int j = 0; j < n_all; ++j) {
          // the phases before are over: one arrival in each, and all of K that came before has been waited for
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (j >= n[s] || c[s] == 0) continue;
            if (Ly::kEarly) wait(&sh.sread[s], c[s] - 1);
            wait(&sh.pfull[s][0], c[s] - 1);
          }
          const int at = tile + 1;
          tile += 2;
          wait(&sh.full[at & (Ly::kRing - 1)], at / Ly::kRing);
          if (j + 1 == n[0] || j + 1 == n[1]) {
            uint4* v = reinterpret_cast<uint4*>(ring + (at & (Ly::kRing - 1)) * Ly::kTile);
            uint32_t any = 0;
#pragma unroll 8
            for (int e = lane; e < Ly::kTile / 16; e += 32) {
              const uint4 x = v[e];
              any |= special2(x.x) | special2(x.y) | special2(x.z) | special2(x.w);
            }
            if (any) {
              s_special = 1;
              for (int e = lane; e < Ly::kTile / 16; e += 32) {
                const uint4 x = v[e];
                v[e] = make_uint4(finite2(x.x), finite2(x.y), finite2(x.z), finite2(x.w));
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
          }
          if (j + 1 < n_all) wait(&sh.full[tile & (Ly::kRing - 1)], tile / Ly::kRing);
          __syncwarp();
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (j >= n[s]) continue;
            if (Ly::kEarly && lane == 0) mbar_arrive(&sh.sread[s]);
            if (lane == 0) mbar_arrive(&sh.pfull[s][0]);
            ++c[s];
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax: two threads for each query row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int s = warp >> 3, half = (warp >> 2) & 1, r = tid & (kRows - 1);
    const int pair = 1 + (warp & 3) + 4 * s;  // named barrier of the two warps that share rows
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t at_s = lane_base + Ly::kColS + 128 * s + 64 * half;
    const uint32_t at_p = lane_base + Ly::kColP + Ly::kPStep * s + 32 * half;
    const uint32_t at_o = lane_base + Ly::kColO + kDim * s + kDim / 2 * half;  // this thread's half of the row's output
    int c = 0, o_phase = 0;  // tiles and items of this sub-tile so far
    // What the other thread of the row puts in. With one place for it, it is free again for the next tile because S of
    // that comes after every warp's P of this. Where S comes as soon as this one has been read (kEarly), the partner may
    // still be on its way from the barrier to its load when this thread writes for the next tile: the places take turns, and
    // the barrier of the tile in between keeps a load and the next write of the same place apart. The sum at an item's
    // end goes in turn like a tile's maximum, with a barrier of its own behind it.
    auto exchange = [&](float mine) {
      float(&place)[2][kRows] = sh.half[Ly::kSlots == 2 ? c & 1 : 0][s];
      place[half][r] = mine;
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
      return place[half ^ 1][r];
    };
    for (int round = 0;; ++round) {
      const Work* w = work_in(round);
      if (!__any_sync(0xffffffffu, w != nullptr)) break;
      const int n = __shfl_sync(0xffffffffu, w->tiles[s], 0);
      float m_ref = -INFINITY, l = 0.0f;  // exponent reference (log2 domain, the same in both threads) and this half's sum
      for (int left = n; left > 0; --left, ++c) {
        wait(&sh.sfull[s], c);
        __syncwarp();
        tc_after();
        float x[64];
        tc_ld64(at_s, x);
        if (Ly::kEarly) {
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.sread[s]);
        }
        // the last tile: keys after the row's own are masked (warps whose rows see all of their 64 keys have nothing to do)
        if (left == 1 && 64 * half + 63 > (r & ~31)) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (64 * half + e > r) x[e] = -INFINITY;
        }
        float tops[4] = {x[0], x[1], x[2], x[3]};  // chains short enough to issue without waiting
#pragma unroll
        for (int e = 4; e < 64; e += 2) tops[(e >> 1) & 3] = fmaxf(tops[(e >> 1) & 3], fmaxf(x[e], x[e + 1]));
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        top = fmaxf(top, exchange(top));  // both have read their S: P may be written over it
        const float m_new = fmaxf(m_ref, top * a.scale_log2);
        const bool move = m_new > m_ref + kRescaleLog2 || (m_ref == -INFINITY && m_new > -INFINITY);
        // O of this sub-tile has to be at rest, and P be read: the last P V came before the S that was waited for, or is
        // waited for itself
        if (Ly::kEarly && c > 0) {
          wait(&sh.ofull[s], c - 1);
          __syncwarp();
          tc_after();
        }
        float base = move ? m_new : m_ref;
        if (__any_sync(0xffffffffu, (move && m_ref > -INFINITY) || fabsf(m_new) >= kLargeLog2)) {
          if (__any_sync(0xffffffffu, move && m_ref > -INFINITY)) {
            const float f = move ? fast_exp2(m_ref - m_new) : 1.0f;
            l *= f;
#pragma unroll 1
            for (int e0 = 0; e0 < kDim / 2; e0 += 16) {  // seldom: a few registers at a time, the row of S stays in its own
              uint32_t o[16];
              tc_ld16u(at_o + e0, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tc_st16u(at_o + e0, o);
            }
          }
          m_ref = base;
          if (fabsf(m_new) >= kLargeLog2 && fabsf(m_new) < INFINITY) {  // the score is finite: scale is 2^-106 at least
            const float back = 1.0f / a.scale_log2;
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e] = __fsub_rn(__fmul_rn(x[e], a.scale_log2), base) * back;
            base = 0.0f;
          }
        } else {
          m_ref = base;
        }
        if (base == -INFINITY) base = 0.0f;
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
            if (lane == 0) mbar_arrive(&sh.pfull[s][Ly::kParts == 2 ? q : 0]);
          }
        }
        const float2 sum = unpack2(add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])));
        l += sum.x + sum.y;
      }
      if (n > 0) {
        wait(&sh.ofull[s], Ly::kEarly ? c - 1 : o_phase);
        ++o_phase;
        l += exchange(l);
        asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");  // the other has it: free for the next item
        tc_after();
        // The row, normalised, in 32 columns at a time through the warp's own 2 KB, so that whole sectors are stored by
        // neighbouring lanes: pieces of 16 bytes, their place within four turned by the row.
        uint8_t* stage = smem + Ly::kStage + warp * 2048;
        const float inv = 1.0f / l;
        const int block = w->block[s], i = block * kRows + r, len = w->len;
        const int row0 = block * kRows + (r & ~31) + (lane >> 2), piece = lane & 3;
        uint16_t* out = a.out.p + (int64_t)(w->t0 + row0) * a.out.ts + (int64_t)w->head[s] * a.out.hs;
        const bool special = s_special;
#pragma unroll
        for (int e0 = 0; e0 < kDim / 2; e0 += 32) {
          const int d0 = kDim / 2 * half + e0;
          float o[32];
          tc_ld32(at_o + e0, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          if (special && i < len) add_specials(a, o, d0, w->t0, i, w->kh, w->block);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                           pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            const int row = e + (lane >> 2);
            const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
            if (row0 + e < len && d0 + 8 * piece < a.dim)
              *reinterpret_cast<uint4*>(out + (int64_t)e * a.out.ts + d0 + 8 * piece) = x;
          }
          __syncwarp();
        }
        tc_before();  // before the next item's first P, and with it the product that writes O anew
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.wempty[round & 1]);
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
  constexpr int kBytes = Layout<kDim>::kRest + (int)sizeof(Rest<Layout<kDim>::kSlots>);
  static_assert(kBytes <= 227 * 1024 && Layout<kDim>::kRing <= 8, "shared memory of one CTA");
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
    } else if (cudaMemcpy(p->d_items, p->items.data(), bytes, cudaMemcpyHostToDevice) != cudaSuccess ||
               // a copy from pageable memory may still be under way, on a stream that the plan's first call does not wait for
               cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess) {
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
  if (!plan || !(scale >= 0.0f && scale * kLog2E < INFINITY)) return MV_ERR_INVALID_ARG;
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
  // a masked score is -inf, and 0 * -inf would be a NaN: the smallest scale in place of zero, with which no score is anything
  a.scale_log2 = fmaxf(scale * kLog2E, 1.4e-45f);
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
