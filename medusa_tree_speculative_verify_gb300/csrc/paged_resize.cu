// Lengths, block table and free pages of a batch of sequences that grow and shrink; places of the rows that come.
//
// With exclusive sums over the sequences of rows that come, pages taken and pages given up, everything has a place of its
// own: page a of all that are given up (counted in the table's order) is pushed as number R - 1 - a of R, the j-th that is
// taken comes from the stack's place F + R - 1 - j of F + R, which is page j of those given up while j < R. So no page waits
// for another, and which page goes where does not depend on the order of threads.
//
// Bound by latency: lengths, sums, then one dependent load for each page or row. A cluster of CTAs, each of which does the
// sums for itself, moves the pages; all have read the lengths before the first of them writes (the cluster's barrier). One
// CTA took 41 us for 200 prompts of up to 8192 tokens let in and out where eight took 15.5; with four pages of a thread at once
// they take 12.5. More than kRowsHere rows go to a second kernel over the whole GPU, which looks them up in what the first one
// wrote (19200 rows: 10.8 us there and back, 13.0 without).
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace {

constexpr int kPlaceThreads = 512;
constexpr int kCluster = 8;
constexpr int kRowsHere = 8192;
constexpr uint32_t kMost = 0x7fffffffu;

struct ResizeArgs {
  const int32_t* by;
  int32_t *lens, *table, *free;  // free: how many, then the stack
  int n_seq, ld_table, page_size, n_pages;
  int64_t most;  // positions of a row of the table
  int32_t *cu, *positions;
  int64_t* slots;
  int n_rows;
  bool rows_here;
  unsigned int* err;
};

// the last b with sums[b] <= i, where sums[0] <= i < sums[n]
MV_DEV int find(const int* sums, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same for kAtOnce of them, whose steps do not wait for each other. top: the largest power of two below n, or 0.
template <int kAtOnce>
MV_DEV void find(const int* sums, int n, int top, const int (&i)[kAtOnce], int (&b)[kAtOnce]) {
#pragma unroll
  for (int k = 0; k < kAtOnce; ++k) b[k] = 0;
  for (int step = top; step; step >>= 1)
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int next = b[k] + step;
      if (next < n && sums[next] <= i[k]) b[k] = next;
    }
}

MV_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
MV_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int kThreads>
__global__ void __launch_bounds__(kThreads) paged_resize_kernel(const ResizeArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ int s_all[];
  const int n = a.n_seq;
  int *s_rows = s_all, *s_take = s_rows + n + 1, *s_give = s_take + n + 1, *s_len = s_give + n + 1, *s_by = s_len + n;
  __shared__ uint32_t s_scan[3][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)cluster_rank();
  pdl_trigger();
  pdl_wait();
  const int held = __ldcg(a.free);
  bool bad = false;
  // Sums stop at kMost, so that none is taken for a small one.
  auto add = [](uint32_t x, uint32_t y) { return min(x + y, kMost); };
  uint32_t carry[3] = {0, 0, 0};
  for (int base = 0; base < n; base += kThreads) {
    const int b = base + tid;
    uint32_t x[3] = {0, 0, 0};  // rows that come, pages taken, pages given up
    int len = 0, by = 0;
    if (b < n) {
      len = __ldcg(a.lens + b);
      by = __ldcg(a.by + b);
      const int64_t to = (int64_t)len + by;
      if (len < 0 || len > a.most || to < 0 || to > a.most) {
        bad = true;
        if (rank == 0) mv_set_error_detail(a.err, kPagedResizeSite, MV_DEVERR_INDEX, (uint32_t)b);
      } else {
        const int more = (int)((to + a.page_size - 1) / a.page_size) - (len + a.page_size - 1) / a.page_size;
        x[0] = (uint32_t)max(0, by);
        x[1] = (uint32_t)max(0, more);
        x[2] = (uint32_t)max(0, -more);
      }
    }
    uint32_t incl[3];
    const int used = min(kWarps, (n - base + 31) / 32);  // warps with a sequence
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      incl[k] = x[k];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, incl[k], o);
        if (lane >= o) incl[k] = add(incl[k], up);
      }
      if (lane == 31) s_scan[k][warp] = incl[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      uint32_t before = carry[k], all = carry[k];
      if (used <= 4) {  // one after the other, soonest for few
        for (int w = 0; w < used; ++w) {
          const uint32_t one = s_scan[k][w];
          if (w < warp) before = add(before, one);
          all = add(all, one);
        }
      } else {
        uint32_t to = lane < used ? s_scan[k][lane] : 0u;  // of the warps up to `lane`
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
          const uint32_t up = __shfl_up_sync(0xffffffffu, to, o);
          if (lane >= o) to = add(to, up);
        }
        const uint32_t one = __shfl_sync(0xffffffffu, to, max(warp - 1, 0));
        if (warp) before = add(before, one);
        all = add(all, __shfl_sync(0xffffffffu, to, kWarps - 1));
      }
      if (b < n) s_all[k * (n + 1) + b] = (int)(add(before, incl[k]) - x[k]);  // where nothing stopped at kMost
      carry[k] = all;
    }
    if (b < n) {
      s_len[b] = len;
      s_by[b] = by;
    }
    __syncthreads();
  }
  const bool over = held < 0 || carry[0] > (a.positions || a.slots ? (uint32_t)a.n_rows : kMost) ||
                    max(carry[0], max(carry[1], carry[2])) == kMost || (int64_t)held + carry[2] > a.n_pages ||
                    carry[1] > (int64_t)held + carry[2];
  if (over && rank == 0 && tid == 0) mv_set_error_detail(a.err, kPagedResizeSite, MV_DEVERR_INDEX, (uint32_t)n);
  bad = __syncthreads_or(bad || over);
  const int rows = bad ? 0 : (int)carry[0], take = bad ? 0 : (int)carry[1], give = bad ? 0 : (int)carry[2];
  if (tid == 0) {
    s_rows[n] = rows;
    s_take[n] = take;
    s_give[n] = give;
  }
  __syncthreads();

  auto pages_of = [&](int len) { return (int)((unsigned)(len + a.page_size - 1) / (unsigned)a.page_size); };
  auto given = [&](int i, int b) {  // page i of those given up, which is sequence b's
    const int left = pages_of(s_len[b]) - (s_give[b + 1] - s_give[b]);
    return __ldcg(a.table + (int64_t)b * a.ld_table + left + i - s_give[b]);
  };
  auto taken = [&](int j) { return j < give ? given(j, find(s_give, n, j)) : __ldcg(a.free + 1 + (held + give - 1 - j)); };
  cluster_arrive();  // this CTA has read what is overwritten at the end
  constexpr int kAtOnce = 4;
  const int step = kThreads * (int)gridDim.x, first = rank * kThreads + tid, top = n > 1 ? 1 << (31 - __clz(n - 1)) : 0;
  bool odd = false;  // a page outside the pool
  for (int64_t i0 = first; i0 < give; i0 += kAtOnce * step) {
    int i[kAtOnce], b[kAtOnce], page[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) i[k] = (int)min(i0 + k * step, (int64_t)give - 1);
    find(s_give, n, top, i, b);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) page[k] = given(i[k], b[k]);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (i0 + k * step >= give) break;
      odd |= page[k] < 0 || page[k] >= a.n_pages;
      a.free[1 + (held + give - 1 - i[k])] = page[k];  // at or over `held`: nothing here reads that
    }
  }
  for (int64_t j0 = first; j0 < take; j0 += kAtOnce * step) {
    int j[kAtOnce], b[kAtOnce], page[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      j[k] = (int)min(j0 + k * step, (int64_t)take - 1);
      page[k] = taken(j[k]);
    }
    find(s_take, n, top, j, b);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (j0 + k * step >= take) break;
      odd |= page[k] < 0 || page[k] >= a.n_pages;
      a.table[(int64_t)b[k] * a.ld_table + pages_of(s_len[b[k]]) + j[k] - s_take[b[k]]] = page[k];
    }
  }
  if (odd) mv_set_error_detail(a.err, kPagedResizeSite, MV_DEVERR_INDEX, (uint32_t)n + 1);
  if (a.rows_here)
    for (int64_t i = first; i < a.n_rows; i += step) {
      int pos = -1;
      int64_t slot = -1;
      if (i < rows) {
        const int b = find(s_rows, n, (int)i);
        pos = s_len[b] + (int)i - s_rows[b];
        if (a.slots) {
          const int nth = pos / a.page_size, had = pages_of(s_len[b]);
          const int page = nth < had ? __ldcg(a.table + (int64_t)b * a.ld_table + nth) : taken(s_take[b] + nth - had);
          slot = (int64_t)page * a.page_size + (pos - nth * a.page_size);
        }
      }
      if (a.positions) a.positions[i] = pos;
      if (a.slots) a.slots[i] = slot;
    }
  __syncwarp();
  cluster_wait();
  if (rank != 0) return;
  if (a.cu)
    for (int b = tid; b <= n; b += kThreads) a.cu[b] = bad ? 0 : s_rows[b];
  if (bad) return;
  for (int b = tid; b < n; b += kThreads) {
    if (s_by[b]) a.lens[b] = s_len[b] + s_by[b];
  }
  if (tid == 0) a.free[0] = held + give - take;
}

// positions and slots of all rows, from cu, the new lengths and the new table
__global__ void __launch_bounds__(kPlaceThreads) paged_places_kernel(const ResizeArgs a) {
  extern __shared__ int s_all[];
  const int n = a.n_seq;
  int *s_rows = s_all, *s_end = s_all + n + 1;  // s_end[b] + row = position
  pdl_trigger();
  pdl_wait();
  for (int b = threadIdx.x; b <= n; b += kPlaceThreads) {
    s_rows[b] = __ldcg(a.cu + b);
    if (b < n) s_end[b] = __ldcg(a.lens + b) - __ldcg(a.cu + b + 1);
  }
  __syncthreads();
  const int rows = s_rows[n];
  for (int64_t i = (int64_t)blockIdx.x * kPlaceThreads + threadIdx.x; i < a.n_rows; i += (int64_t)gridDim.x * kPlaceThreads) {
    int pos = -1;
    int64_t slot = -1;
    if (i < rows) {
      const int b = find(s_rows, n, (int)i);
      pos = s_end[b] + (int)i;
      if (a.slots) {
        const int nth = pos / a.page_size;
        slot = (int64_t)__ldcg(a.table + (int64_t)b * a.ld_table + nth) * a.page_size + (pos - nth * a.page_size);
      }
    }
    if (a.positions) a.positions[i] = pos;
    if (a.slots) a.slots[i] = slot;
  }
}

template <int kThreads>
mv_status launch_resize(const ResizeArgs& a, cudaStream_t st) {
  static int flags[64] = {};
  const auto fn = paged_resize_kernel<kThreads>;
  const auto bytes = [](int n_seq) { return (5 * n_seq + 3) * (int)sizeof(int); };
  if (!mv_set_smem_once((const void*)fn, bytes(kPagedMaxSeq), flags)) return MV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes(a.n_seq);
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {kCluster, 1, 1};
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = mv_pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, a) == cudaSuccess ? MV_OK : MV_ERR_CUDA;
}

}  // namespace

extern "C" mv_status paged_kv_resize(const int32_t* by, int32_t n_seq, int32_t page_size, int32_t n_pages,
                                     int32_t* block_table, int32_t ld_table, int32_t max_pages, int32_t* seq_lens,
                                     int32_t* free_pages, int32_t* cu_rows, int32_t* positions, int64_t* slots,
                                     int32_t n_rows, mv_stream stream) {
  if (n_seq < 0 || n_rows < 0) return MV_ERR_INVALID_ARG;
  if (n_seq > kPagedMaxSeq || n_pages < 1 || page_size < 16 || page_size > kPagedMaxPage || page_size % 16)
    return MV_ERR_SHAPE;
  if (max_pages < 1 || ld_table < max_pages || (int64_t)max_pages * page_size > 0x7fffffff - 1024) return MV_ERR_SHAPE;
  if (!free_pages || (n_seq && (!by || !block_table || !seq_lens))) return MV_ERR_INVALID_ARG;
  if (((positions || slots) && !cu_rows) || (reinterpret_cast<uintptr_t>(slots) & 7)) return MV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(by) | reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(free_pages) | reinterpret_cast<uintptr_t>(cu_rows) |
       reinterpret_cast<uintptr_t>(positions)) & 3)
    return MV_ERR_INVALID_ARG;
  ResizeArgs a;
  a.by = by;
  a.lens = seq_lens;
  a.table = block_table;
  a.free = free_pages;
  a.n_seq = n_seq;
  a.ld_table = ld_table;
  a.page_size = page_size;
  a.n_pages = n_pages;
  a.most = (int64_t)max_pages * page_size;
  a.cu = cu_rows;
  a.positions = positions;
  a.slots = slots;
  a.n_rows = positions || slots ? n_rows : 0;
  a.rows_here = a.n_rows <= kRowsHere;
  a.err = mv_error_word();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Few sequences have few pages, and fewer warps meet sooner: 48 growing by a token and back 5.5 us, with 512 threads 5.8; 200
  // prompts let in and out 13.7 and 12.5.
  const mv_status s = n_seq <= 64 ? launch_resize<256>(a, st) : launch_resize<512>(a, st);
  if (s != MV_OK) return s;
  if (!a.rows_here) {
    const int ctas = (int)std::min<int64_t>(2 * mv_sm_count(), ((int64_t)a.n_rows + kPlaceThreads - 1) / kPlaceThreads);
    if (mv_launch(paged_places_kernel, dim3(ctas), dim3(kPlaceThreads), (2 * n_seq + 1) * sizeof(int), st, a) != cudaSuccess)
      return MV_ERR_CUDA;
  }
  return mv_last_launch("paged_resize");
}
