// Norms of the heads of Q and K and their rotation by position, in one pass.
//
// A row x is one token's head of D elements: y = x / sqrt(mean x^2 + eps) * gain, then each pair of y's first R elements, (i,
// i + R/2) or (2 i, 2 i + 1), is turned by the angle position * f_i. In fp32, rounded once.
//
// Angles. f_i comes as a fraction of a turn in 64 bits, f_i / 2 pi = turns_i 2^-64, so position * turns_i modulo 2^64 is the
// angle without its whole turns, exact to position * 2^-64 turns: a position of 2^31 is as good as one of 1. (In fp32 an
// angle of a million radians is off by up to 0.03.)
//
// Bound by memory: 2 bytes read and 2 written for each element; about 110 instructions for 16 elements of a thread. A thread
// takes 16 elements of a row as two pieces of 16 bytes, chosen so that pairs meet in it; what is left to exchange is the sum
// of squares. A CTA takes the rows of a few tokens: their sines and cosines are computed once for all heads, while the first
// rows are on their way.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRopeDim = 256;
constexpr int kAhead = 2;        // rows of a thread on their way
constexpr int kResident = 3;     // CTAs of an SM
constexpr int kRows = 256;       // of a CTA, about
constexpr int kTokens = 16;      // of a CTA, at most

struct RopeArgs {
  RowsArgs q, k, q_out, k_out;
  const uint16_t *q_gain, *k_gain;  // [dim] or null
  const int32_t* positions;
  const uint64_t* turns;            // [rot / 2]
  float eps;
  int n_tokens, heads, kv_heads, dim, rot;
  int tokens, span;                 // tokens of a CTA, and heads (of Q and K together)
};

MV_DEV void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(x[i]);
    f[2 * i + 1] = bf16hi(x[i]);
  }
}
MV_DEV uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// kLanes threads a row, the power of two from dim / 16 up. kNeighbours: pairs (2 i, 2 i + 1).
template <int kLanes, bool kNeighbours>
__global__ void __launch_bounds__(kThreads, kResident) qk_norm_rope_kernel(const RopeArgs a) {
  __shared__ float s_cos[kTokens * kMaxRopeDim / 2], s_sin[kTokens * kMaxRopeDim / 2];
  __shared__ bool s_real[kTokens];
  constexpr int kGroups = kThreads / kLanes;  // rows at a time
  const int tid = threadIdx.x, j = tid % kLanes, group = tid / kLanes;
  const int half = a.rot / 2, turned = a.rot / 16;  // lanes whose elements are turned
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.n_tokens - t0);
  const int h0 = blockIdx.y * a.span, nh = min(a.span, a.heads + a.kv_heads - h0);
  const bool mine = j < a.dim / 16;
  // this thread's pieces of 8 elements: pairs of halves meet across R/2 elements, what is not turned lies side by side
  const bool rot = mine && j < turned;
  const int e0 = kNeighbours || !rot ? 16 * j : 8 * j, e1 = kNeighbours || !rot ? 16 * j + 8 : 8 * j + half;
  uint4 gain[2][2];
#pragma unroll
  for (int is_k = 0; is_k < 2; ++is_k) {
    const uint16_t* g = is_k ? a.k_gain : a.q_gain;
    const uint32_t one = 0x3f803f80u;
    gain[is_k][0] = gain[is_k][1] = make_uint4(one, one, one, one);
    if (g && mine) {
      gain[is_k][0] = *reinterpret_cast<const uint4*>(g + e0);
      gain[is_k][1] = *reinterpret_cast<const uint4*>(g + e1);
    }
  }
  pdl_trigger();
  pdl_wait();
  const int rows = nt * nh, add_t = kGroups / nh, add_h = kGroups - add_t * nh;
  int tok = group / nh, h = group - tok * nh;  // of the next row that is asked for
  uint4 x[kAhead][2];
  int at_t[kAhead], at_h[kAhead];
  auto ask = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      at_t[i] = tok;
      at_h[i] = h0 + h;
      x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (r0 + i * kGroups < rows && mine) {
        const bool is_k = at_h[i] >= a.heads;
        const RowsArgs& p = is_k ? a.k : a.q;
        const uint16_t* row = p.p + (int64_t)(t0 + tok) * p.ts + (int64_t)(is_k ? at_h[i] - a.heads : at_h[i]) * p.hs;
        x[i][0] = __ldcg(reinterpret_cast<const uint4*>(row + e0));
        x[i][1] = __ldcg(reinterpret_cast<const uint4*>(row + e1));
      }
      tok += add_t;
      h += add_h;
      if (h >= nh) {
        h -= nh;
        ++tok;
      }
    }
  };
  ask(group);
  for (int i = tid; i < nt * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const uint64_t angle = (uint64_t)(uint32_t)__ldcg(a.positions + t0 + t) * __ldg(a.turns + f);
    // in half turns, -1 .. 1
    sincospif((float)(int32_t)(angle >> 32) * 4.656612873077393e-10f, &s_sin[i], &s_cos[i]);
  }
  if (tid < nt) s_real[tid] = !a.positions || __ldcg(a.positions + t0 + tid) >= 0;
  __syncthreads();
  const float inv = 1.0f / (float)a.dim;
  for (int r0 = group; r0 < rows; r0 += kAhead * kGroups) {  // the lanes of a group stay together
    if (r0 != group) ask(r0);
    const unsigned int mask = kLanes == 32 ? 0xffffffffu : ((1u << kLanes) - 1u) << (tid & 31 & ~(kLanes - 1));
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const bool real = r0 + i * kGroups < rows && s_real[at_t[i]];
      float u[8], v[8], sum = 0.0f;
      unpack8(x[i][0], u);
      unpack8(x[i][1], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += u[e] * u[e] + v[e] * v[e];
#pragma unroll
      for (int o = kLanes >> 1; o >= 1; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
      if (!real || !mine) continue;
      const bool is_k = at_h[i] >= a.heads;
      const float f = rsqrtf(sum * inv + a.eps);
      float g[8];
      unpack8(is_k ? gain[1][0] : gain[0][0], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] *= f * g[e];
      unpack8(is_k ? gain[1][1] : gain[0][1], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= f * g[e];
      if (rot) {
        float c[8], s[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const int at = at_t[i] * half + 8 * j + e;
          const float4 c4 = *reinterpret_cast<const float4*>(s_cos + at), s4 = *reinterpret_cast<const float4*>(s_sin + at);
          c[e] = c4.x, c[e + 1] = c4.y, c[e + 2] = c4.z, c[e + 3] = c4.w;
          s[e] = s4.x, s[e + 1] = s4.y, s[e + 2] = s4.z, s[e + 3] = s4.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float& p = kNeighbours ? (e < 4 ? u[(2 * e) & 7] : v[(2 * e) & 7]) : u[e];
          float& q = kNeighbours ? (e < 4 ? u[(2 * e + 1) & 7] : v[(2 * e + 1) & 7]) : v[e];
          const float was = p;
          p = was * c[e] - q * s[e];
          q = q * c[e] + was * s[e];
        }
      }
      const RowsArgs& p = is_k ? a.k_out : a.q_out;
      uint16_t* row = p.p + (int64_t)(t0 + at_t[i]) * p.ts + (int64_t)(is_k ? at_h[i] - a.heads : at_h[i]) * p.hs;
      *reinterpret_cast<uint4*>(row + e0) = pack8(u);
      *reinterpret_cast<uint4*>(row + e1) = pack8(v);
    }
  }
}

template <int kLanes>
cudaError_t launch_rope(const RopeArgs& a, dim3 grid, bool neighbours, cudaStream_t st) {
  return neighbours ? mv_launch(qk_norm_rope_kernel<kLanes, true>, grid, dim3(kThreads), 0, st, a)
                    : mv_launch(qk_norm_rope_kernel<kLanes, false>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace

extern "C" mv_status qk_norm_rope(mv_rows q, mv_rows k, int32_t n_tokens, int32_t n_heads, int32_t n_kv_heads,
                                  int32_t head_dim, const mv_bf16* q_gain, const mv_bf16* k_gain, float eps,
                                  const int32_t* positions, const uint64_t* turns, int32_t rot_dim, int32_t neighbours,
                                  mv_rows q_out, mv_rows k_out, mv_stream stream) {
  if (n_tokens < 0) return MV_ERR_INVALID_ARG;
  if (n_heads < 0 || n_kv_heads < 0 || n_heads > kPagedMaxHeads || n_kv_heads > kPagedMaxHeads) return MV_ERR_SHAPE;
  if (head_dim < 16 || head_dim > kMaxRopeDim || head_dim % 16 || rot_dim < 0 || rot_dim > head_dim || rot_dim % 16)
    return MV_ERR_SHAPE;
  if (!(eps >= 0.0f && eps < INFINITY) || (neighbours != 0 && neighbours != 1)) return MV_ERR_INVALID_ARG;
  if (rot_dim && (!positions || !turns || (reinterpret_cast<uintptr_t>(turns) & 7))) return MV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(positions) & 3) ||
      ((reinterpret_cast<uintptr_t>(q_gain) | reinterpret_cast<uintptr_t>(k_gain)) & 15))
    return MV_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_heads + n_kv_heads == 0) return MV_OK;
  if (n_heads && (!mv_rows_ok(q, n_tokens, n_heads, head_dim) || !mv_out_rows_ok(q_out, n_tokens, n_heads, head_dim)))
    return MV_ERR_INVALID_ARG;
  if (n_kv_heads &&
      (!mv_rows_ok(k, n_tokens, n_kv_heads, head_dim) || !mv_out_rows_ok(k_out, n_tokens, n_kv_heads, head_dim)))
    return MV_ERR_INVALID_ARG;
  const auto rows = [](const mv_rows& r) { return RowsArgs{static_cast<uint16_t*>(r.ptr), r.token_stride, r.head_stride}; };
  RopeArgs a;
  a.q = rows(q);
  a.k = rows(k);
  a.q_out = rows(q_out);
  a.k_out = rows(k_out);
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.positions = positions;
  a.turns = turns;
  a.eps = eps;
  a.n_tokens = n_tokens;
  a.heads = n_heads;
  a.kv_heads = n_kv_heads;
  a.dim = head_dim;
  a.rot = rot_dim;
  int lanes = 1;
  while (16 * lanes < head_dim) lanes *= 2;
  // about kRows rows a CTA, of fewer tokens or heads where the GPU would not be full
  const int all = n_heads + n_kv_heads, groups = kThreads / lanes;
  const int64_t ctas = (int64_t)kResident * mv_sm_count();
  a.tokens = std::max(1, std::min(kTokens, kRows / all));
  a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>(a.tokens, n_tokens / ctas));
  a.span = a.tokens > 1 ? all : std::min(all, n_tokens >= ctas ? kRows : groups);
  const dim3 grid((n_tokens + a.tokens - 1) / a.tokens, (all + a.span - 1) / a.span);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = lanes == 16  ? launch_rope<16>(a, grid, neighbours, st)
                        : lanes == 8 ? launch_rope<8>(a, grid, neighbours, st)
                        : lanes == 4 ? launch_rope<4>(a, grid, neighbours, st)
                        : lanes == 2 ? launch_rope<2>(a, grid, neighbours, st)
                                     : launch_rope<1>(a, grid, neighbours, st);
  return e == cudaSuccess ? mv_last_launch("qk_norm_rope") : MV_ERR_CUDA;
}
