// Causal attention over whole prompts packed in one call, and the plan that lays out its work.
//
// A warp computes one (token, query head) row: a lane holds four of the dim values, the warp goes over the row's keys
// with the running maximum and sum of the softmax.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "kernels.cuh"
#include "paged.cuh"

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
  int group, kv_heads, dim;
  float scale_log2;
  unsigned int* err;
};

MV_DEV float4 load4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

// One row by one warp: query token i of the prompt that starts at token t0, head h.
MV_DEV void row_by_warp(const PromptArgs& a, int t0, int i, int h) {
  const int lane = threadIdx.x & 31, d0 = lane * 4, kh = h / a.group;
  const bool on = d0 < a.dim;
  float4 q = make_float4(0.f, 0.f, 0.f, 0.f), o = q;
  if (on) q = load4(a.q.p + (int64_t)(t0 + i) * a.q.ts + (int64_t)h * a.q.hs + d0);
  float m = -INFINITY, l = 0.0f;
  for (int j = 0; j <= i; ++j) {
    float x = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      const float4 k = load4(a.k.p + (int64_t)(t0 + j) * a.k.ts + (int64_t)kh * a.k.hs + d0);
      v = load4(a.v.p + (int64_t)(t0 + j) * a.v.ts + (int64_t)kh * a.v.hs + d0);
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
  const float inv = 1.0f / l;
  if (on)
    *reinterpret_cast<uint2*>(a.out.p + (int64_t)(t0 + i) * a.out.ts + (int64_t)h * a.out.hs + d0) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

constexpr int kWarps = 16;

__global__ void __launch_bounds__(kWarps * 32) prompt_attn_kernel(const PromptArgs a) {
  pdl_trigger();
  pdl_wait();
  const int4 item = a.items[blockIdx.x / a.kv_heads];
  const int kh = blockIdx.x % a.kv_heads, warp = threadIdx.x >> 5;
  for (int s = 0; s < 2; ++s) {
    const int t = item.z + s, i0 = t / a.group * kRows, h = kh * a.group + t % a.group;
    for (int i = i0 + warp; i < min(i0 + kRows, item.y); i += kWarps) row_by_warp(a, item.x, i, h);
  }
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
  a.scale_log2 = scale * 1.4426950408889634f;
  a.err = mv_error_word();
  const int64_t grid = (int64_t)(plan->items.size() / 4) * n_kv_heads;  // at most 2^22 * 2^8
  const cudaError_t e = mv_launch(prompt_attn_kernel, dim3((unsigned)grid), dim3(kWarps * 32), 0,
                                  static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? mv_last_launch("prompt_attention") : MV_ERR_CUDA;
}
