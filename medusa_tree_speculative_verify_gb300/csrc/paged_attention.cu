// Attention of one new token for each sequence over a paged cache (bf16, or e4m3 with an exponent for each row).
//
// Bound by the cache's bytes: every row is read once for up to 16 query heads of a kv head (once for each 16 of more). What
// they share is read for all of them together, 8 (or 16) heads a work unit, on the tensor cores with the keys as the rows of the products (mma.sync
// m16n8k16): S^T = K Q^T and O^T += V^T P^T. At 8 heads a unit the products cost 16 to 24 instructions for each 16 keys'
// 4 to 8 KB, far below what the copies take, and keys as rows waste nothing on padding the heads.
//
// Copies: by TMA, 16 rows of a page's head at a time, a queue of kStages steps of 8 KB for each warp, which waits for
// nobody else. The order of the dim in a dot product, and of the dim as output rows, is free, so that each lane's operands
// are whole 16-byte pieces of rows, read from shared memory without shuffles; the 128-byte swizzle of the copy keeps the
// value reads free of bank conflicts and the key reads at two a bank.
//   K: lane (g, t) = (lane / 4, lane % 4) reads rows g and g + 8 of 16 keys, pieces t, t + 4, ..; the words of a piece
//      are consecutive dim pairs, a product's k index 2 t, 2 t + 1, 2 t + 8, 2 t + 9. Q is read in the same order.
//   V: rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9, piece g: pairs of rows are interleaved byte-wise (prmt) to operands.
// P goes from the layout of S^T to that of P^T by a transposing movmatrix.
//
// A column may have nothing in the rows of the largest weights, so small weights need their bits as much as large ones. In
// bf16 they are split in two (16 bits), one more product each.
//
// e4m3: K and V convert exactly to fp16. Q is brought to fp16 with a power of two for each head (largest element in
// [2^14, 2^15), so what fp16 loses lies 2^-38 below it). A key row's scale multiplies its score; a value row's scale 2^e
// goes into the weight's exponent, and the weight in fp16 (11 bits) into one product. Where one of a step's weights is below
// fp16's normal range, the step is done as for bf16, with rows of V that are multiplied by their scale in bf16. The sums are
// in units of 2^unit, -24 <= unit <= 0, which only follows the largest e (unit >= e - 7, so weights of up to 2^8 stay within
// fp16's 2^15): however far rows' scales and weights lie apart, the sums have fp32's range. (Every step in bf16: 16 x
// 24576 keys of 32/8 heads 151 us, 133 so; 64 ragged sequences 46, 39.5. With a unit that follows the largest scaled weight,
// and nothing else, a row 2^25 below it was lost. Scores so far apart that all steps are done in bf16: 175 and 53.)
//
// Split. The work is a line of steps, kWarps tiles of keys each, over all units (sequence, kv head, 8 or 16 of its
// heads); every CTA takes an equal piece of the line, whatever the lengths are. A unit's start and end (its Q, putting the
// warps' results together) cost about kUnitCost steps, which have their places on the line too, so that a piece of many
// short sequences takes no longer than one of a long one. A unit within one CTA is done there; one that crosses pieces
// leaves partial results (reference, sum, output in fp32) in the workspace, and the CTA that adds the last one joins all of
// them in the order of the line, so the result does not depend on who comes last.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.cuh"
#include "paged.cuh"

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kStages = 3;       // steps of a warp's queue
constexpr int kUnitCost = 2;     // what a unit costs beside its steps, in steps (128 sequences of up to 2000 keys: 30 us, with 1: 35)
constexpr int kShortSteps = 16;  // steps of one warp up to which a sequence may go a unit to each warp
constexpr unsigned int kEvenMost = 20;  // places of a piece up to which all have one length
constexpr int kMaxCtas = 160;    // counters at the start of the workspace; CTAs of a launch
constexpr int kChunkSeq = 1024;  // sequences of one launch, at most
constexpr int kClusterMost = 16;
constexpr int kUnitLeast = -24;  // log2 of the sums' unit: from here to 0

struct AttnArgs {
  PagedArgs c;
  RowsArgs q, out;
  int group, parts;  // query heads of a kv head, units of a kv head
  int cluster;       // CTAs of a cluster
  int short_keys;    // sequences of at most so many keys go a unit to each warp
  int box_tiles;     // 16-key tiles of a copy: 1, 2 or 4, never over a page's end
  // divisions by a page's 16-key tiles, done once on the host: of a tile number n by n * page_inv >> 36; pages and tiles in
  // them from a step to the next of all warps and of one (a division takes a hundred cycles and more of a call's start)
  uint64_t page_inv;
  int page_add, tile_add, page_one, tile_one, groups_log2;  // 2^groups_log2 copies for K or V's tiles of a step
  float scale_log2;
  unsigned int* count;  // [kMaxCtas]
  float* part;          // [CTAs][2] partial results
  unsigned int* err;
};

template <int kDim, bool kE4M3, int kNT>
struct Layout {
  static constexpr int kRow = kE4M3 ? kDim : 2 * kDim;   // bytes of a row in shared memory
  static constexpr int kBox = kRow < 128 ? kRow : 128;   // bytes of a row that a copy takes, and of the swizzle
  static constexpr int kBoxes = kRow / kBox;             // copies for 16 rows
  static constexpr int kRegion = 16 * kBox;              // bytes of one
  static constexpr int kSub = 256 / kRow;                // 16-key tiles of a warp's step: 8 KB
  static constexpr int kKeys = 16 * kSub;                // keys of a warp's step
  // a step: for each box of the row the regions of its kSub tiles, K, then the same of V
  static constexpr int kV = kBoxes * kSub * kRegion, kStage = 2 * kV;
  static constexpr int kExps = kE4M3 ? 32 * kSub : 0;    // bytes of their exponents
  static constexpr int kVPiece = kRow / 8 < 16 ? 8 : 16; // bytes a lane reads of a value row at once
  static constexpr int kMT = kDim / 16;                  // 16-row tiles of O^T
  static constexpr int kHeads = 8 * kNT;
  static constexpr int kSlot = kMT * 4 * 32;             // floats of one warp's O^T of 8 heads
  static constexpr int kPart = kHeads * (kDim + 4);      // floats of a partial result
  static constexpr int kQueue = kWarps * kStages * kStage;
  // the join of a unit's parts: their weights for 8 heads, a partial sum of 8 values for each thread
  static constexpr int kJoin = (8 * kMaxCtas + 8 * kThreads) * 4;
  static constexpr int kMerge = 4 * kSlot * 4 > kJoin ? 4 * kSlot * 4 : kJoin;
  static constexpr int kExpsAt = kQueue, kMergeAt = kExpsAt + kWarps * kStages * kExps, kPreAt = kMergeAt + kMerge;
  static_assert(kWarps * kKeys == (kE4M3 ? (kDim > 64 ? 256 : 512) : (kDim > 64 ? 128 : 256)), "paged_attention's chunks");
  static_assert(kStage == 8192 && kSub * 2 * kBoxes <= 16 && 2 * kSub <= 16 && kMergeAt % 16 == 0, "");
  static int bytes(int n_seq) { return 1024 + kPreAt + (2 * n_seq + 1) * 4; }
};

MV_DEV uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
MV_DEV uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
MV_DEV uint32_t lds_byte(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
// 16 bytes of global memory to shared memory by this thread
MV_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// arrives at `bar` once this thread's cp_async16 so far have come
MV_DEV void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
template <bool kF16>
MV_DEV void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
MV_DEV uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
MV_DEV uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
MV_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two e4m3 values of two rows as bf16, times the rows' scales (bf16, powers of two): rounded only below the normal range.
MV_DEV uint32_t scaled_bf16x2(uint16_t x, uint32_t scales) {
  const float2 f = half2_to_float2(e4m3x2_to_half2(x));
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632)), "r"(scales));
  return r;
}
// Two weights each split in two bf16, transposed
MV_DEV void split_weights(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  const uint32_t h = pack_bf16x2(p0, p1);
  hi = transpose8x8(h);
  lo = transpose8x8(pack_bf16x2(p0 - bf16lo(h), p1 - bf16hi(h)));
}
// 2^(a - b) where both may be -inf (then the weight of nothing: 0)
MV_DEV float weight(float a, float b) { return a == -INFINITY ? 0.0f : exp2f(a - b); }

// kCluster: one sequence, a cluster of CTAs for each unit (see launch).
template <int kDim, bool kE4M3, int kNT, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttnArgs a) {
  using Ly = Layout<kDim, kE4M3, kNT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t s_full[kWarps][kStages];
  __shared__ float s_ml[kWarps][2][8];  // reference, sum
  __shared__ float s_fin[4][8];         // all warps': factor of the output, reference, sum, bad
  __shared__ float s_unit[kWarps];      // unit of the sums
  __shared__ bool s_bad[kWarps];
  __shared__ int s_scan[kWarps];
  struct Split {
    int b, head0, n_heads, u0, n;  // u0, n: first place and steps of the unit; n = 0: none
  };
  __shared__ Split s_split[2];  // the units of which this CTA holds a part
  __shared__ bool s_last[2];
  float* s_merge = reinterpret_cast<float*>(smem + Ly::kMergeAt);
  int* s_pre = reinterpret_cast<int*>(smem + Ly::kPreAt);  // [n_seq + 1] first place of each sequence
  int* s_len = s_pre + a.c.n_seq + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int n_seq = a.c.n_seq, units = a.c.heads * a.parts, groups = (units + kWarps - 1) / kWarps;  // of a sequence
  constexpr int kStepKeys = kWarps * Ly::kKeys;
  pdl_trigger();
  if (tid == 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], kE4M3 ? 33 : 1);  // the copies' bytes, and each lane's exponents
    mbar_fence_init();
  }
  pdl_wait();

  int total = 0;
  if (kCluster) {
    if (tid == 0) {
      const int len = __ldcg(a.c.seq_lens);
      const bool bad = len < 0 || len > a.c.max_pages * a.c.page_size;
      if (bad && blockIdx.x == 0) mv_set_error_detail(a.err, kPagedAttnSite, MV_DEVERR_INDEX, 0u);
      s_len[0] = bad ? -1 : len;
    }
    __syncthreads();
    if (s_len[0] < 0) return;  // the whole grid
  } else {
    // ---- the line: for every unit kUnitCost places that stand for its start and end, then its steps (one for an empty
    // sequence: its zeros are written). A sequence of a bad length has none.
    int carry = 0;
    for (int base = 0; base < n_seq; base += kThreads) {
      const int b = base + tid;
      int steps = 0;
      if (b < n_seq) {
        int len = __ldcg(a.c.seq_lens + b);
        const bool bad = len < 0 || len > a.c.max_pages * a.c.page_size;
        if (bad && blockIdx.x == 0) mv_set_error_detail(a.err, kPagedAttnSite, MV_DEVERR_INDEX, (uint32_t)b);
        const bool one = len <= a.short_keys;
        steps = bad ? 0
                    : (kUnitCost + max(1, one ? (len + Ly::kKeys - 1) / Ly::kKeys : (len + kStepKeys - 1) / kStepKeys)) *
                          (one ? groups : units);
        s_len[b] = bad ? 0 : len;
      }
      int incl = steps;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      int before = carry, all = carry;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_scan[w];
        all += s_scan[w];
      }
      if (b < n_seq) s_pre[b] = before + incl - steps;
      carry = all;
      __syncthreads();
    }
    if (tid == 0) s_pre[n_seq] = carry;
    if (tid < 2) s_split[tid].n = 0;
    __syncthreads();
    total = carry;
  }
  // Pieces of one length, the least that the grid can do them in: with the places spread over all CTAs none would be done
  // sooner, and units would have more parts (12 sequences of up to 38 k keys, 16 heads of one kv head: 17 us, spread 21; 4 of
  // 2000, 8 kv heads: 12 and 14.5). Long pieces are spread, the first `rest` of them one longer: there the last few SMs count
  // for their bandwidth (64 sequences of up to 8191 keys, 33 places a piece: 38.7 us, of one length 39.9).
  const unsigned int all = (unsigned)total, least = (all + gridDim.x - 1) / gridDim.x;
  const bool even = least <= kEvenMost;
  const int each = kCluster ? 1 : max(1, (int)(even ? least : all / gridDim.x)), rest = even ? 0 : total - each * (int)gridDim.x;
  const int ctas = kCluster ? 1 : even ? (int)((all + each - 1) / (unsigned)each) : (int)gridDim.x, cta = blockIdx.x;
  if (!kCluster && cta >= ctas) return;
  auto piece = [&](int c) { return (int)min((unsigned)c * (unsigned)each + min(c, rest), all); };
  const int s_first = kCluster ? 0 : piece(cta);
  int s_end = kCluster ? 0 : piece(cta + 1);
  // A place on the line: step `step` of the `n` of an entry, which is unit `idx` of sequence b for all warps (a step is
  // kWarps tiles in turn) or, `one`, units kWarps * idx .. of a short sequence, one for each warp.
  struct Place {
    int b, idx, step, n, len;
    bool one;
  };
  auto enter = [&](Place& p, int b) {
    p.b = b;
    p.len = s_len[b];
    p.one = !kCluster && p.len <= a.short_keys;
    p.n = max(1, p.one ? (p.len + Ly::kKeys - 1) / Ly::kKeys : (p.len + kStepKeys - 1) / kStepKeys);
  };
  // to the next entry, whose first place is s < total
  auto next_entry = [&](Place& p, int s) {
    p.step = 0;
    if (++p.idx < (p.one ? groups : units)) return;
    p.idx = 0;
    int b = p.b;
    do ++b;
    while (s_pre[b + 1] <= s);
    enter(p, b);
  };
  Place ahead;
  int s_begin;  // the first step at or after s_first that this CTA does
  const int c_rank = kCluster ? (int)cluster_rank() : 0, c_size = kCluster ? a.cluster : 1;
  if (kCluster) {  // an equal share of the unit's steps, possibly none; places counted from 0
    enter(ahead, 0);
    ahead.idx = cta / c_size;
    ahead.step = (int)((int64_t)ahead.n * c_rank / c_size);
    s_begin = 0;
    s_end = (int)((int64_t)ahead.n * (c_rank + 1) / c_size) - ahead.step;
  } else {
    int lo = 0, hi = n_seq;  // the last b with pre[b] <= s_first: one with places
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] <= s_first) lo = mid;
      else hi = mid;
    }
    enter(ahead, lo);
    const int in_b = s_first - s_pre[lo], width = kUnitCost + ahead.n;
    ahead.idx = (unsigned)in_b / (unsigned)width;
    const int at = in_b - ahead.idx * width;
    ahead.step = max(0, at - kUnitCost);
    s_begin = s_first - at + kUnitCost + ahead.step;
    if (ahead.one && ahead.step > 0) {  // belongs to the CTA that holds its first step, as a whole
      s_begin = s_first - at + width + kUnitCost;
      if (s_begin < s_end) next_entry(ahead, s_begin - kUnitCost);
    }
  }
  if (!kCluster && s_begin >= s_end) return;
  Place here = ahead;
  auto head_of = [&](int unit) { return a.parts == 1 ? unit : (int)((unsigned)unit / (unsigned)a.parts); };

  // ---- this warp's queue. A lane is there for one of a step's copies (its tiles from my_u on, a box of K or V; from lane
  // 16 on: the exponents of one tile's K or V). Page and tile in it are carried along: a step is kWarps * kSub tiles after
  // the one before. The table's entries are asked for two steps before their copies.
  const uint32_t queue = smem_u32(smem) + warp * kStages * Ly::kStage;
  const uint32_t exps = smem_u32(smem) + Ly::kExpsAt + warp * kStages * Ly::kExps;
  const int page16 = a.c.page_size >> 4, box_groups = 1 << a.groups_log2;
  const bool my_exp = lane >= 16;
  const int my_u = my_exp ? (lane - 16) >> 1 : (lane & (box_groups - 1)) * a.box_tiles;
  const int my_op = my_exp ? lane & 1 : lane >> a.groups_log2;  // K boxes, then V boxes
  const bool my_v = my_exp ? my_op : my_op >= Ly::kBoxes;
  const bool mine_any = my_exp ? kE4M3 && my_u < Ly::kSub : my_op < 2 * Ly::kBoxes;
  int s_ahead = s_begin, page, tile;  // of the step that is looked up next
  int key_ahead, h_ahead;             // its first key here (past the end: nothing to do) and kv head
  bool more = s_begin < s_end;
  auto enter_copy = [&]() {
    const int first = (ahead.one ? ahead.step : ahead.step * kWarps + warp) * Ly::kSub;
    const int unit = ahead.one ? ahead.idx * kWarps + warp : ahead.idx;
    key_ahead = unit < units ? 16 * first : ahead.len;
    h_ahead = head_of(unit);
    page = (int)((uint64_t)(first + my_u) * a.page_inv >> 36);
    tile = first + my_u - page * page16;
  };
  enter_copy();
  struct Next {
    int entry, row;  // this lane's page and first row in it
    bool has, valid;
  };
  auto look_up = [&]() {
    Next x = {0, 0, false, more};
    if (more) {
      x.has = mine_any && key_ahead + 16 * my_u < ahead.len;
      x.row = h_ahead * a.c.page_size + tile * 16;
      if (x.has) x.entry = __ldcg(a.c.table + (int64_t)ahead.b * a.c.ld_table + page);
      ++s_ahead;
      if (++ahead.step < ahead.n) {
        more = ahead.one || s_ahead < s_end;
        key_ahead = key_ahead < ahead.len ? key_ahead + (ahead.one ? Ly::kKeys : kStepKeys) : ahead.len;
        page += ahead.one ? a.page_one : a.page_add;
        tile += ahead.one ? a.tile_one : a.tile_add;
        if (tile >= page16) {
          tile -= page16;
          ++page;
        }
      } else {
        s_ahead += kUnitCost;
        more = s_ahead < s_end;
        if (more) {
          next_entry(ahead, s_ahead - kUnitCost);
          enter_copy();
        }
      }
    }
    return x;
  };
  Next next = look_up(), then = look_up();
  // A page outside the pool is not copied. What the step's place holds then is of no sequence, so a unit with such a step, in
  // whichever warp or CTA, is bad: its rows of out stay as they were.
  constexpr uint32_t kBad = 1u << 16;  // a lane's bad page in the sum of a step's bytes, which are fewer
  static_assert(Ly::kStage < (int)kBad, "");
  uint32_t bad_slots = 0;
  int copied = 0, used = 0;  // steps
  auto copy_step = [&](int slot) {
    if (next.valid) {
      const bool bad = next.has && (next.entry < 0 || next.entry >= a.c.n_pages);
      if (bad) mv_set_error_detail(a.err, kPagedAttnSite, MV_DEVERR_INDEX, (uint32_t)next.entry);
      const bool go = next.has && !bad;
      const uint32_t bytes = go && !my_exp ? (uint32_t)(a.box_tiles * Ly::kRegion) : 0u;
      const uint32_t sum = __reduce_add_sync(0xffffffffu, bytes + (bad ? kBad : 0u));  // also: every lane is done with the slot
      bad_slots = (bad_slots & ~(1u << slot)) | (sum >= kBad ? 1u << slot : 0u);
      uint64_t* bar = &s_full[warp][slot];
      if (lane == 0) mbar_arrive_expect_tx(bar, sum & (kBad - 1));
      if (bytes) {
        const int box = my_v ? my_op - Ly::kBoxes : my_op;
        uint8_t* dst = smem + (warp * kStages + slot) * Ly::kStage + (my_op * Ly::kSub + my_u) * Ly::kRegion;
        tma_load_3d(dst, my_v ? &vmap : &kmap, bar, box * (kE4M3 ? Ly::kBox : Ly::kBox / 2), next.row, next.entry);
      }
      if (kE4M3) {
        if (go && my_exp)
          cp_async16(exps + slot * Ly::kExps + (lane - 16) * 16,
                     (my_v ? a.c.v_exp : a.c.k_exp) + (int64_t)next.entry * a.c.heads * a.c.page_size + next.row);
        cp_async_arrive(bar);
      }
      ++copied;
    }
    next = then;
    then = look_up();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy_step(i);
  // where this lane reads in a 16-row region: its piece of key row g (row g + 8: + 8 rows), of value row 2 t and 2 t + 1
  uint32_t k_off, v_off[2];
  if (Ly::kBox == 128) {
    k_off = g * 128 + ((t ^ g) << 4);  // piece t; piece t + 4: ^ 64
    v_off[0] = 2 * t * 128 + ((g ^ (2 * t)) << 4);
    v_off[1] = (2 * t + 1) * 128 + ((g ^ (2 * t + 1)) << 4);
  } else {
    k_off = g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
    v_off[0] = 2 * t * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
    v_off[1] = v_off[0] + 64;
  }

  // the words of Q of a unit: head g of each tile of 8, the pieces as of K
  uint32_t q_raw[kNT][kDim / 8];
  auto load_q = [&](const Place& p) {
    constexpr int kWords = kE4M3 ? 8 : 4;  // words of Q for a piece of K
    const int unit = p.one ? p.idx * kWarps + warp : p.idx, kh = head_of(unit);
    const int head0 = kh * a.group + (unit - kh * a.parts) * Ly::kHeads;
    const int n_heads = unit < units ? min(Ly::kHeads, (kh + 1) * a.group - head0) : 0;
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const int h = 8 * n + g;
      const uint16_t* row = a.q.p + (int64_t)p.b * a.q.ts + (int64_t)(h < n_heads ? head0 + h : 0) * a.q.hs;
#pragma unroll
      for (int i = 0; i < Ly::kRow / 64; ++i) {
        const int d = 2 * kWords * (t + 4 * i);
#pragma unroll
        for (int j = 0; j < kWords; j += 4) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (h < n_heads && d + 2 * j < a.c.dim) v = *reinterpret_cast<const uint4*>(row + d + 2 * j);
          q_raw[n][i * kWords + j] = v.x;
          q_raw[n][i * kWords + j + 1] = v.y;
          q_raw[n][i * kWords + j + 2] = v.z;
          q_raw[n][i * kWords + j + 3] = v.w;
        }
      }
    }
  };

  // ---- unit after unit
  int s = s_begin, slot = 0, phase = 0;
  bool once = kCluster;  // a CTA of a cluster puts its results together even where it has no step
  load_q(here);
  while (s < s_end || once) {
    once = false;
    const int b = here.b, len = here.len, nb = here.n, step0 = here.step;
    const bool one = here.one;
    const int steps = one ? nb : min(nb - step0, s_end - s);  // of this entry, here
    const int unit = one ? here.idx * kWarps + warp : here.idx, kh = head_of(unit);
    const int head0 = kh * a.group + (unit - kh * a.parts) * Ly::kHeads;
    const int n_heads = unit < units ? min(Ly::kHeads, (kh + 1) * a.group - head0) : 0;
    // this warp's first key, and from step to step
    int key0 = one ? 0 : step0 * kStepKeys + warp * Ly::kKeys;
    const int key_add = one ? Ly::kKeys : kStepKeys, key_end = n_heads > 0 ? len : 0;

    // Q as the second operand: head g (of each tile of 8), the dim in the order of the K pieces
    uint32_t qf[kNT][kDim / 16][2];
    float mult[kNT][2];  // score of head 2 t (+ 1) into the exponent
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const uint32_t(&w)[kDim / 8] = q_raw[n];
      if (kE4M3) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kDim / 8; ++i) top = fmaxf(top, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t e = max(15u, __float_as_uint(top) >> 23);
        const float up = __uint_as_float((268u - e) << 23), back = __uint_as_float((e - 14u) << 23);
#pragma unroll
        for (int i = 0; i < kDim / 8; ++i) qf[n][i >> 1][i & 1] = pack_f16x2(bf16lo(w[i]) * up, bf16hi(w[i]) * up);
        mult[n][0] = __shfl_sync(0xffffffffu, back, 8 * t) * a.scale_log2;
        mult[n][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4) * a.scale_log2;
      } else {
#pragma unroll
        for (int i = 0; i < kDim / 8; ++i) qf[n][i >> 1][i & 1] = w[i];
        mult[n][0] = mult[n][1] = a.scale_log2;
      }
    }
    int sum_unit = kE4M3 ? kUnitLeast : 0;
    float o[kNT][Ly::kMT][4], mx[kNT][2], l[kNT][2];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
#pragma unroll
      for (int m = 0; m < Ly::kMT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][m][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[n][e] = -INFINITY;
        l[n][e] = 0.0f;
      }
    }

    bool bad = false;
    for (int i = 0; i < steps; ++i, key0 += key_add) {
      copy_step(slot == 0 ? kStages - 1 : slot - 1);
      bool there = used++ < copied;  // not after a wait that gave up
      if (there && !__all_sync(0xffffffffu, mbar_wait(&s_full[warp][slot], phase))) {
        more = next.valid = then.valid = there = false;  // nothing more is copied; what is on its way is still waited for
        mv_set_error(a.err, kPagedAttnSite, MV_DEVERR_TIMEOUT);
      }
      bad |= !there || (bad_slots >> slot & 1u);
      const uint32_t at = queue + slot * Ly::kStage, ex_at = exps + slot * Ly::kExps;
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1;
      }
      if (key0 >= key_end) continue;

      // S^T: rows keys g, g + 8 of each tile, columns heads 2 t, 2 t + 1. Tiles behind the sequence's last hold what an
      // earlier step left: their scores are masked below, their products with V are left out. Two sums for one chain of
      // products where there is only one.
      constexpr int kSums = Ly::kSub * kNT == 1 ? 2 : 1;
      float x[kNT][Ly::kSub][4], x2[4] = {};
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int u = 0; u < Ly::kSub; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][u][e] = 0.0f;
#pragma unroll
      for (int i2 = 0; i2 < Ly::kRow / 64; ++i2) {
        uint4 kw[Ly::kSub][2];  // keys g, g + 8
#pragma unroll
        for (int u = 0; u < Ly::kSub; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            kw[u][r] = lds16(at + ((i2 >> 1) * Ly::kSub + u) * Ly::kRegion + (k_off ^ (i2 & 1) * 64) + r * 8 * Ly::kBox);
#pragma unroll
        for (int j = 0; j < (kE4M3 ? 4 : 2); ++j)
#pragma unroll
          for (int u = 0; u < Ly::kSub; ++u) {
            const uint32_t wl[4] = {kw[u][0].x, kw[u][0].y, kw[u][0].z, kw[u][0].w};
            const uint32_t wh[4] = {kw[u][1].x, kw[u][1].y, kw[u][1].z, kw[u][1].w};
            uint32_t f[4];
            if (kE4M3) {
              f[0] = e4m3x2_to_half2((uint16_t)wl[j]);
              f[1] = e4m3x2_to_half2((uint16_t)wh[j]);
              f[2] = e4m3x2_to_half2((uint16_t)(wl[j] >> 16));
              f[3] = e4m3x2_to_half2((uint16_t)(wh[j] >> 16));
            } else {
              f[0] = wl[(2 * j) & 3];
              f[1] = wh[(2 * j) & 3];
              f[2] = wl[(2 * j + 1) & 3];
              f[3] = wh[(2 * j + 1) & 3];
            }
            const int qi = (kE4M3 ? 4 : 2) * i2 + j;
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              mma<kE4M3>(kSums == 2 && (qi & 1) ? x2 : x[n][u], f[0], f[1], f[2], f[3], qf[n][qi][0], qf[n][qi][1]);
          }
      }
      if (kSums == 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[0][0][e] += x2[e];
      // scores into the exponent's base; the value rows' exponents
      int ev[Ly::kSub][2], top_ev = kUnitLeast;
#pragma unroll
      for (int u = 0; u < Ly::kSub; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int key = key0 + 16 * u + g + 8 * r;
          float ks = 1.0f;
          if (kE4M3) {
            const uint32_t ex = ex_at + 32 * u + g + 8 * r;
            ks = exp_byte_scale(lds_byte(ex));
            ev[u][r] = (int)lds_byte(ex + 16) - 127;
            top_ev = max(top_ev, key < len ? ev[u][r] : kUnitLeast);
          }
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& v = x[n][u][2 * r + e];
              v = key < len ? v * (kE4M3 ? ks * mult[n][e] : mult[n][e]) : -INFINITY;
            }
        }
      // the references: moved when a score outgrows them by 2^8, from nothing at the first key that is seen; the unit too
      bool grow = kE4M3 && top_ev > sum_unit + 7 && sum_unit < 0;
      float tx[kNT][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tx[n][e] = -INFINITY;
#pragma unroll
          for (int u = 0; u < Ly::kSub; ++u)
#pragma unroll
            for (int r = 0; r < 2; ++r) tx[n][e] = fmaxf(tx[n][e], x[n][u][2 * r + e]);
          grow |= tx[n][e] > mx[n][e] + 8.0f;
        }
      if (__any_sync(0xffffffffu, grow)) {
        float shift = 1.0f;
        if (kE4M3) {
          const int next = min(0, max(sum_unit, __reduce_max_sync(0xffffffffu, top_ev) - 7));
          shift = __uint_as_float((uint32_t)(127 + sum_unit - next) << 23);
          sum_unit = next;
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 4; w <= 16; w <<= 1) tx[n][e] = fmaxf(tx[n][e], __shfl_xor_sync(0xffffffffu, tx[n][e], w));
            const float nx = fmaxf(mx[n][e], tx[n][e]), f = weight(mx[n][e], nx), fo = f * shift;
            l[n][e] *= f;
#pragma unroll
            for (int m = 0; m < Ly::kMT; ++m) {
              o[n][m][e] *= fo;
              o[n][m][2 + e] *= fo;
            }
            mx[n][e] = nx;
          }
      }
      // weights, their sum, and P^T as the second operand
      uint32_t ph[kNT][Ly::kSub][2], pl[kNT][Ly::kSub][2];
      float least = 0.0f;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int u = 0; u < Ly::kSub; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& y = x[n][u][2 * r + e];
              y -= mx[n][e] == -INFINITY ? 0.0f : mx[n][e];
              p[e] = ex2(y);
              l[n][e] += p[e];
              if (kE4M3) {
                const float z = y + (float)(ev[u][r] - sum_unit);
                least = fminf(least, key0 + 16 * u + g + 8 * r < len ? z : 0.0f);
                p[e] = ex2(z);
              }
            }
            if (kE4M3) {
              ph[n][u][r] = transpose8x8(pack_f16x2(p[0], p[1]));
            } else {
              split_weights(p[0], p[1], ph[n][u][r], pl[n][u][r]);
            }
          }
      const bool low = kE4M3 && __any_sync(0xffffffffu, least < -14.0f || top_ev > 7);
      // O^T += V^T P^T; kWide: e4m3 rows times their scales in bf16, with ph and pl
      auto add_values = [&](auto wide) {
        constexpr bool kWide = decltype(wide)::value;
#pragma unroll
        for (int u = 0; u < Ly::kSub; ++u) {
          if (u > 0 && key0 + 16 * u >= len) break;
          const uint32_t vt = at + Ly::kV + u * Ly::kRegion;
          const int left = len - key0 - 16 * u;
          constexpr int kPieces = Ly::kBoxes, kWords = Ly::kVPiece / 4;
          uint32_t scales[2];  // of rows 2 t and 2 t + 1, 2 t + 8 and 2 t + 9
          if (kWide) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              uint32_t s[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int row = 2 * t + i + 8 * r, byte = (int)lds_byte(ex_at + 32 * u + 16 + row) - sum_unit;
                s[i] = row >= left ? 0u : byte > 0 ? (uint32_t)min(byte, 255) << 7 : 0x40u;
              }
              scales[r] = s[0] | s[1] << 16;
            }
          }
#pragma unroll
          for (int i2 = 0; i2 < kPieces; ++i2) {
            uint32_t w[4][4];  // rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t src = vt + i2 * Ly::kSub * Ly::kRegion + v_off[r & 1] + (r >> 1) * 8 * Ly::kBox;
              if (kWords == 4) {
                const uint4 v = lds16(src);
                w[r][0] = v.x;
                w[r][1] = v.y;
                w[r][2] = v.z;
                w[r][3] = v.w;
              } else {
                const uint2 v = lds8(src);
                w[r][0] = v.x;
                w[r][1] = v.y;
              }
            }
            if (left < 16) {  // rows behind the sequence hold anything: weight zero times a NaN would be one
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (2 * t + (r & 1) + 4 * (r & 2) >= left)
#pragma unroll
                  for (int j = 0; j < kWords; ++j) w[r][j] = 0u;
            }
            if (kE4M3) {
#pragma unroll
              for (int m = 0; m < 2 * kWords; ++m) {  // two of a word's four dims
                const uint32_t sel = m & 1 ? 0x7362u : 0x5140u;
                const uint32_t lo = __byte_perm(w[0][m >> 1], w[1][m >> 1], sel), hi = __byte_perm(w[2][m >> 1], w[3][m >> 1], sel);
                if (kWide) {
                  const uint32_t a0 = scaled_bf16x2((uint16_t)lo, scales[0]), a1 = scaled_bf16x2((uint16_t)(lo >> 16), scales[0]);
                  const uint32_t a2 = scaled_bf16x2((uint16_t)hi, scales[1]), a3 = scaled_bf16x2((uint16_t)(hi >> 16), scales[1]);
#pragma unroll
                  for (int n = 0; n < kNT; ++n) mma<false>(o[n][m], a0, a1, a2, a3, ph[n][u][0], ph[n][u][1]);
#pragma unroll
                  for (int n = 0; n < kNT; ++n) mma<false>(o[n][m], a0, a1, a2, a3, pl[n][u][0], pl[n][u][1]);
                } else {
                  const uint32_t a0 = e4m3x2_to_half2((uint16_t)lo), a1 = e4m3x2_to_half2((uint16_t)(lo >> 16));
                  const uint32_t a2 = e4m3x2_to_half2((uint16_t)hi), a3 = e4m3x2_to_half2((uint16_t)(hi >> 16));
#pragma unroll
                  for (int n = 0; n < kNT; ++n) mma<true>(o[n][m], a0, a1, a2, a3, ph[n][u][0], ph[n][u][1]);
                }
              }
            } else {
              uint32_t f[4][4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                f[j][0] = __byte_perm(w[0][j], w[1][j], 0x5410);
                f[j][1] = __byte_perm(w[0][j], w[1][j], 0x7632);
                f[j][2] = __byte_perm(w[2][j], w[3][j], 0x5410);
                f[j][3] = __byte_perm(w[2][j], w[3][j], 0x7632);
              }
#pragma unroll
              for (int n = 0; n < kNT; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  mma<false>(o[n][4 * i2 + j], f[j][0], f[j][1], f[j][2], f[j][3], ph[n][u][0], ph[n][u][1]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  mma<false>(o[n][4 * i2 + j], f[j][0], f[j][1], f[j][2], f[j][3], pl[n][u][0], pl[n][u][1]);
              }
            }
          }
        }
      };
      if (low) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int u = 0; u < Ly::kSub; ++u)
#pragma unroll
            for (int r = 0; r < 2; ++r) split_weights(ex2(x[n][u][2 * r]), ex2(x[n][u][2 * r + 1]), ph[n][u][r], pl[n][u][r]);
        add_values(std::integral_constant<bool, kE4M3>());
      } else {
        add_values(std::false_type());
      }
    }

    // ---- the entry's results: the warps' together, 8 heads at a time
    const bool whole = !kCluster && steps == nb;
    const int u0 = s - step0 - kUnitCost;                       // the unit's first place
    const int part = u0 <= s_first ? 0 : 1;                     // this CTA's partial result of it
    if (!kCluster && !whole && tid == 0) s_split[part] = {b, head0, n_heads, u0, nb};
    s += steps + kUnitCost;
    if (s < s_end) {  // the next entry's Q is on its way while this one's results are put together
      next_entry(here, s - kUnitCost);
      load_q(here);
    }
    const float unit_scale = __uint_as_float((uint32_t)(127 + sum_unit) << 23);
    if (one) {  // a unit of one warp: done here
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int w = 4; w <= 16; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
          const int h = 8 * n + 2 * t + e;
          const float f = len > 0 ? unit_scale / l[n][e] : 0.0f;
#pragma unroll
          for (int i2 = 0; i2 < kDim / 64; ++i2) {
            const int d = kE4M3 ? kDim / 8 * g + 8 * i2 : 8 * (g + 8 * i2);
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(o[n][4 * i2 + k][e] * f, o[n][4 * i2 + k][2 + e] * f);
            if (h < n_heads && d < a.c.dim && !bad)
              *reinterpret_cast<uint4*>(a.out.p + (int64_t)b * a.out.ts + (int64_t)(head0 + h) * a.out.hs + d) =
                  make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      continue;
    }
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w <= 16; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
        if (g == 0) {
          s_ml[warp][0][2 * t + e] = mx[n][e];
          s_ml[warp][1][2 * t + e] = l[n][e];
        }
      }
      if (lane == 0) {
        s_bad[warp] = bad;
        s_unit[warp] = unit_scale;
      }
      // warps 4-7 leave their output, 0-3 add it to theirs, then the four sums; warp 4 meanwhile what all have in common
      float* mine = s_merge + (warp & 3) * Ly::kSlot + lane;
      if (warp >= 4) {
#pragma unroll
        for (int m = 0; m < Ly::kMT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[(4 * m + e) * 32] = o[n][m][e];
      }
      __syncthreads();
      if (warp < 4) {
        float f[2], f4[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][0][2 * t + e]);
          f[e] = weight(mx[n][e], top) * unit_scale;
          f4[e] = weight(s_ml[warp + 4][0][2 * t + e], top) * s_unit[warp + 4];
        }
#pragma unroll
        for (int m = 0; m < Ly::kMT; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[(4 * m + e) * 32] = o[n][m][e] * f[e & 1] + mine[(4 * m + e) * 32] * f4[e & 1];
      } else if (warp == 4 && lane < 8) {
        float tx = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) tx = fmaxf(tx, s_ml[w][0][lane]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_ml[w][1][lane] * weight(s_ml[w][0][lane], tx);
        s_fin[0][lane] = len > 0 ? 1.0f / sum : 0.0f;
        s_fin[1][lane] = tx;
        s_fin[2][lane] = sum;
        bool any_bad = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) any_bad |= s_bad[w];
        s_fin[3][lane] = any_bad ? 1.0f : 0.0f;
      }
      __syncthreads();
      // thread: one head of the tile, 8 consecutive dims
      for (int e = tid; e < 8 * kDim / 8; e += kThreads) {
        const int ln = e & 31, odd = (e >> 5) & 1, i2 = e >> 6, hh = 2 * (ln & 3) + odd, h = 8 * n + hh;
        const int d = kE4M3 ? kDim / 8 * (ln >> 2) + 8 * i2 : 8 * ((ln >> 2) + 8 * i2);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float* src = s_merge + ((4 * (4 * i2 + (k >> 1))) + 2 * (k & 1) + odd) * 32 + ln;
          v[k] = (src[0] + src[Ly::kSlot]) + (src[2 * Ly::kSlot] + src[3 * Ly::kSlot]);
        }
        if (h >= n_heads) continue;
        if (whole) {
          const float f = s_fin[0][hh];
          if (d < a.c.dim && s_fin[3][hh] == 0.0f)
            *reinterpret_cast<uint4*>(a.out.p + (int64_t)b * a.out.ts + (int64_t)(head0 + h) * a.out.hs + d) =
                make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f),
                           pack_bf16x2(v[4] * f, v[5] * f), pack_bf16x2(v[6] * f, v[7] * f));
        } else {
          float* dst = kCluster ? reinterpret_cast<float*>(smem) : a.part + (int64_t)(2 * cta + part) * Ly::kPart;
          *reinterpret_cast<float4*>(dst + h * kDim + d) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(dst + h * kDim + d + 4) = make_float4(v[4], v[5], v[6], v[7]);
          if (d == 0) *reinterpret_cast<float4*>(dst + Ly::kHeads * kDim + 4 * h) =
                make_float4(s_fin[1][hh], s_fin[2][hh], s_fin[3][hh], 0.0f);
        }
      }
      __syncthreads();
    }
  }

  if (kCluster) {
    // ---- the cluster's partial results lie where the copies went; each CTA joins some heads' dims, in the order of ranks
    cluster_sync_all();
    const int kh = head_of(here.idx), head0 = kh * a.group + (here.idx - kh * a.parts) * Ly::kHeads;
    const int n_heads = min(Ly::kHeads, (kh + 1) * a.group - head0);
    const uint32_t base = smem_u32(smem);
    for (int e = c_rank + c_size * tid; e < Ly::kHeads * kDim / 8; e += c_size * kThreads) {
      const int h = e / (kDim / 8), d = e % (kDim / 8) * 8;
      if (h >= n_heads || d >= a.c.dim) continue;
      float4 ml[kClusterMost];
      float tx = -INFINITY, sum = 0.0f, bad = 0.0f, v[8] = {};
#pragma unroll
      for (int c = 0; c < kClusterMost; ++c) {
        if (c >= c_size) break;
        ml[c] = ld_cluster_f4(map_rank(base + (Ly::kHeads * kDim + 4 * h) * 4, c));
        tx = fmaxf(tx, ml[c].x);
        bad += ml[c].z;
      }
      if (bad != 0.0f) continue;
#pragma unroll
      for (int c = 0; c < kClusterMost; ++c) {
        if (c >= c_size) break;
        const uint32_t src = map_rank(base + (h * kDim + d) * 4, c);
        const float4 lo = ld_cluster_f4(src), hi = ld_cluster_f4(src + 16);
        const float f = weight(ml[c].x, tx), x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        sum += ml[c].y * f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += x[k] * f;
      }
      const float f = here.len > 0 ? 1.0f / sum : 0.0f;
      *reinterpret_cast<uint4*>(a.out.p + (int64_t)(head0 + h) * a.out.hs + d) =
          make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f), pack_bf16x2(v[4] * f, v[5] * f),
                     pack_bf16x2(v[6] * f, v[7] * f));
    }
    cluster_sync_all();  // nobody leaves while its results are read
    return;
  }

  // ---- units over several CTAs: the last one to come joins the partial results in the order of the line
  __syncthreads();
  auto cta_of = [&](int place) {  // the CTA whose piece holds a place: guessed, and put right
    int c = min(ctas - 1, (int)((unsigned)place / (unsigned)each));
    while (piece(c) > place) --c;
    return c;
  };
  if (tid < 2) {
    bool last = false;
    const Split& sp = s_split[tid];
    if (sp.n) {
      const int c0 = cta_of(sp.u0 + kUnitCost), c1 = cta_of(sp.u0 + kUnitCost + sp.n - 1);
      __threadfence();
      last = atomicAdd(a.count + c0, 1u) == (unsigned int)(c1 - c0);
      if (last) {
        atomicExch(a.count + c0, 0u);
        __threadfence();
      }
    }
    s_last[tid] = last;
  }
  __syncthreads();
  for (int which = 0; which < 2; ++which) {
    if (!s_last[which]) continue;
    const int b = s_split[which].b, head0 = s_split[which].head0, n_heads = s_split[which].n_heads;
    const int u0 = s_split[which].u0, c0 = cta_of(u0 + kUnitCost), c1 = cta_of(u0 + kUnitCost + s_split[which].n - 1);
    float *s_w = s_merge, *s_sum = s_merge + 8 * kMaxCtas;
    auto part_of = [&](int c) { return a.part + (int64_t)(2 * c + (c == c0 && u0 > piece(c0) ? 1 : 0)) * Ly::kPart; };
    for (int n = 0; n < kNT && 8 * n < n_heads; ++n) {
      // thread: one head, 8 dims, every kSets-th part (the first kAhead are asked for at once); then the sets
      constexpr int kSets = kThreads / kDim, kAhead = 4;
      const int e = tid % kDim, hh = e / (kDim / 8), d = e % (kDim / 8) * 8, first = c0 + tid / kDim;
      float4 lo[kAhead], hi[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int c = first + i * kSets;
        if (c <= c1 && 8 * n + hh < n_heads) {
          const float* src = part_of(c) + (8 * n + hh) * kDim + d;
          lo[i] = __ldcg(reinterpret_cast<const float4*>(src));
          hi[i] = __ldcg(reinterpret_cast<const float4*>(src + 4));
        }
      }
      // a warp for each head: the references' maximum, the parts' weights, the sum
      const int h = 8 * n + warp;
      const float4 none = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
      float4 ml[kMaxCtas / 32];
      float tx = -INFINITY, sum = 0.0f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < kMaxCtas / 32; ++i) {
        const int c = c0 + 32 * i + lane;
        ml[i] = c <= c1 && h < n_heads ? __ldcg(reinterpret_cast<const float4*>(part_of(c) + Ly::kHeads * kDim + 4 * h)) : none;
      }
#pragma unroll
      for (int i = 0; i < kMaxCtas / 32; ++i) {
        tx = fmaxf(tx, ml[i].x);
        bad |= ml[i].z != 0.0f;
      }
      bad = __any_sync(0xffffffffu, bad);
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) tx = fmaxf(tx, __shfl_xor_sync(0xffffffffu, tx, w));
#pragma unroll
      for (int i = 0; i < kMaxCtas / 32; ++i) {
        const float f = weight(ml[i].x, tx);
        s_w[warp * kMaxCtas + 32 * i + lane] = f;
        sum += ml[i].y * f;
      }
#pragma unroll
      for (int w = 16; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      if (lane == 0) {
        s_ml[0][0][warp] = 1.0f / sum;
        s_bad[warp] = bad;
      }
      __syncthreads();
      float v[8] = {};
      auto add = [&](const float4& lo, const float4& hi, float f) {
        v[0] += lo.x * f;
        v[1] += lo.y * f;
        v[2] += lo.z * f;
        v[3] += lo.w * f;
        v[4] += hi.x * f;
        v[5] += hi.y * f;
        v[6] += hi.z * f;
        v[7] += hi.w * f;
      };
      if (8 * n + hh < n_heads) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (first + i * kSets <= c1) add(lo[i], hi[i], s_w[hh * kMaxCtas + first + i * kSets - c0]);
#pragma unroll 4
        for (int c = first + kAhead * kSets; c <= c1; c += kSets) {
          const float* src = part_of(c) + (8 * n + hh) * kDim + d;
          add(__ldcg(reinterpret_cast<const float4*>(src)), __ldcg(reinterpret_cast<const float4*>(src + 4)),
              s_w[hh * kMaxCtas + c - c0]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s_sum[k * kThreads + tid] = v[k];
      __syncthreads();
      if (tid < kDim && 8 * n + hh < n_heads && d < a.c.dim && !s_bad[hh]) {
        const float f = s_ml[0][0][hh];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float x = s_sum[k * kThreads + tid];
#pragma unroll
          for (int i = 1; i < kSets; ++i) x += s_sum[k * kThreads + i * kDim + tid];
          v[k] = x * f;
        }
        *reinterpret_cast<uint4*>(a.out.p + (int64_t)b * a.out.ts + (int64_t)(head0 + 8 * n + hh) * a.out.hs + d) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
      }
      __syncthreads();
    }
  }
}

// Places on the line that a sequence of all that the table holds would take, steps of `keys` keys.
int64_t most_places(const AttnArgs& a, int keys) {
  return (int64_t)a.c.heads * a.parts *
         (((int64_t)a.c.max_pages * a.c.page_size + keys - 1) / keys + kUnitCost + kShortSteps);
}

// Clusters of `size` CTAs of the kernel that the device holds at once (found once for each device and size).
template <int kDim, bool kE4M3, int kNT>
int most_clusters(int size, int bytes) {
  static std::atomic<int> found[64][5];  // 0: not asked yet, else one more
  const int dev = mv_device(), log2 = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : size == 8 ? 3 : 4;
  if (dev < 0 || dev >= 64) return 0;
  int n = found[dev][log2].load();
  if (!n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim = {(unsigned)size, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, paged_attn_kernel<kDim, kE4M3, kNT, true>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    found[dev][log2].store(++n);
  }
  return n - 1;
}

template <int kDim, bool kE4M3, int kNT>
mv_status launch(const AttnArgs& args, cudaStream_t stream) {
  using Ly = Layout<kDim, kE4M3, kNT>;
  static int flags[64] = {}, c_flags[64] = {}, c_wide[64] = {};
  const int bytes = Ly::bytes(args.c.n_seq);
  if (!mv_set_smem_once((const void*)paged_attn_kernel<kDim, kE4M3, kNT, false>, Ly::bytes(kChunkSeq), flags))
    return MV_ERR_CUDA;
  const int units = args.c.heads * args.parts, sms = std::min(mv_sm_count(), kMaxCtas);
  const int grid = (int)std::min<int64_t>(args.c.n_seq * most_places(args, kWarps * Ly::kKeys), sms);
  AttnArgs a = args;
  // Sequences short enough for one warp to a unit: while there are units for every warp, up to kShortSteps of its steps (128
  // sequences of 160 keys, 8 kv heads: 15 us, cut across warps 28; of half as many steps at most, 128 of up to 300 keys take
  // 16 in place of 20, but those of 160 keys 28)
  a.short_keys = std::min(kShortSteps, 2 * (a.c.n_seq * units / grid)) * Ly::kKeys;
  const int page16 = a.c.page_size / 16;
  a.box_tiles = page16 % Ly::kSub == 0 ? Ly::kSub : Ly::kSub == 4 && page16 % 2 == 0 ? 2 : 1;
  a.groups_log2 = Ly::kSub / a.box_tiles == 4 ? 2 : Ly::kSub / a.box_tiles == 2 ? 1 : 0;
  a.page_inv = (uint64_t(1) << 36) / page16 + 1;  // exact for tile numbers below 2^27: 2^27 * 64 < 2^36
  a.page_add = kWarps * Ly::kSub / page16;
  a.tile_add = kWarps * Ly::kSub % page16;
  a.page_one = Ly::kSub / page16;
  a.tile_one = Ly::kSub % page16;
  // a pool as (dim, row of the page, page), boxes of box_tiles * 16 rows; dims behind the head's are filled with zeros
  CUtensorMap maps[2];
  const uint64_t row = (uint64_t)a.c.dim * (kE4M3 ? 1 : 2), rows = (uint64_t)a.c.heads * a.c.page_size;
  const uint64_t dims[3] = {(uint64_t)a.c.dim, rows, (uint64_t)a.c.n_pages}, strides[2] = {row, row * rows};
  const uint32_t box[3] = {(uint32_t)(kE4M3 ? Ly::kBox : Ly::kBox / 2), 16u * a.box_tiles, 1};
  for (int i = 0; i < 2; ++i)
    if (!mv_encode_tmap(&maps[i], kE4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        i ? a.c.v : a.c.k, dims, strides, box,
                        Ly::kBox == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return MV_ERR_CUDA;

  // One sequence: its units are alike, and a cluster for each, joined over distributed shared memory, is sooner done than
  // pieces of a line that are joined through the workspace (32 heads, 1027 keys: 7.9 and 10.2 us) as long as the clusters fill
  // most of the SMs.
  if (a.c.n_seq == 1) {
    int size = kClusterMost;
    while (size > 1 && units * size > sms) size /= 2;
    const void* fn = (const void*)paged_attn_kernel<kDim, kE4M3, kNT, true>;
    if (units * size <= sms && 4 * units * size >= 3 * sms && mv_set_smem_once(fn, Ly::bytes(1), c_flags)) {
      const int dev = mv_device();
      if (size > 8 && !c_wide[dev])
        c_wide[dev] = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess ? 1 : -1;
      if (size > 8 && c_wide[dev] < 0) cudaGetLastError();
      if ((size <= 8 || c_wide[dev] > 0) && most_clusters<kDim, kE4M3, kNT>(size, Ly::bytes(1)) >= units) {
        a.cluster = size;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(units * size);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Ly::bytes(1);
        cfg.stream = stream;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {(unsigned)size, 1, 1};
        at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = mv_pdl_enabled() ? 2 : 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<kDim, kE4M3, kNT, true>, maps[0], maps[1], a);
        return e == cudaSuccess ? mv_last_launch("paged_attention") : MV_ERR_CUDA;
      }
    }
  }
  const cudaError_t e =
      mv_launch(paged_attn_kernel<kDim, kE4M3, kNT, false>, dim3(grid), dim3(kThreads), bytes, stream, maps[0], maps[1], a);
  return e == cudaSuccess ? mv_last_launch("paged_attention") : MV_ERR_CUDA;
}

}  // namespace

extern "C" mv_status paged_attention_workspace(int32_t n_seq, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                               size_t* bytes) {
  if (!bytes || n_seq < 0) return MV_ERR_INVALID_ARG;
  if (n_seq > kPagedMaxSeq || n_kv_heads < 1 || n_heads < n_kv_heads || n_heads > kPagedMaxHeads ||
      n_heads % n_kv_heads || head_dim < 16 || head_dim > kPagedMaxDim || head_dim % 16)
    return MV_ERR_SHAPE;
  // counters, and two partial results of 16 heads for each CTA
  *bytes = kMaxCtas * sizeof(uint32_t) + (size_t)kMaxCtas * 2 * Layout<128, false, 2>::kPart * sizeof(float);
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
  const bool e4m3 = cache->dtype == MV_DTYPE_E4M3, big = a.c.dim > 64;
  // sequences of a launch: no more than have places in 31 bits, whatever their lengths
  const int chunk = (int)std::min<int64_t>(kChunkSeq, 0x7fffffff / most_places(a, e4m3 ? (big ? 256 : 512) : (big ? 128 : 256)));
  if (chunk < 1) return MV_ERR_SHAPE;
  for (int first = 0; first < n_seq; first += chunk) {
    a.c.n_seq = std::min(chunk, n_seq - first);
    a.c.table = block_table + (int64_t)first * ld_table;
    a.c.seq_lens = seq_lens + first;
    a.q = {static_cast<uint16_t*>(q.ptr) + first * q.token_stride, q.token_stride, q.head_stride};
    a.out = {static_cast<uint16_t*>(out.ptr) + first * out.token_stride, out.token_stride, out.head_stride};
    if (big)
      s = e4m3 ? (wide ? launch<128, true, 2>(a, st) : launch<128, true, 1>(a, st))
               : (wide ? launch<128, false, 2>(a, st) : launch<128, false, 1>(a, st));
    else
      s = e4m3 ? (wide ? launch<64, true, 2>(a, st) : launch<64, true, 1>(a, st))
               : (wide ? launch<64, false, 2>(a, st) : launch<64, false, 1>(a, st));
    if (s != MV_OK) return s;
  }
  return MV_OK;
}
