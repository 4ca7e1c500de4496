// Norms of the heads of Q and K and their rotation by position, in one pass.
//
// A row x is one token's head of D elements: y = x / sqrt(mean x^2 + eps) * gain, then each pair of y's first R elements, (i,
// i + R/2) or (2 i, 2 i + 1), is turned by the angle position * f_i. In fp32 (but see below), rounded once.
//
// Angles. f_i comes as a fraction of a turn in 64 bits, f_i / 2 pi = turns_i 2^-64, so position * turns_i modulo 2^64 is the
// angle without its whole turns, exact to position * 2^-64 turns: a position of 2^31 is as good as one of 1. (In fp32 an
// angle of a million radians is off by up to 0.03.)
//
// Bound by memory: 2 bytes read and 2 written for each element. A warp takes some heads of one token (few heads: of
// several), a group of lanes to a head: side by side in memory and then the next ones. A lane has 16 elements of a head as two
// pieces of 16 bytes, chosen so that pairs meet in it; what is left to exchange is the sum of squares. What a lane's elements
// are multiplied with but for the row's own factor, cosines and sines times gains, it computes once for all its heads.
//
// Sine and cosine are the special-function unit's, the angle being within half a turn of zero: off by 2^-21.1 at most, that is
// of the pair's length, where the result's rounding is 2^-9 of the element. (An element that nearly cancels, or is a sine
// of almost nothing, has the former.) The root's reciprocal is rsqrtf, 2 units of fp32.
#include <algorithm>

#include "kernels.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kMaxRopeDim = 256;
constexpr int kAhead = 4;         // rows of a group on their way
constexpr int kResident = 5;      // CTAs of an SM
constexpr int kWarpsWanted = 24;  // of an SM

struct RopeArgs {
  RowsArgs q, k, q_out, k_out;
  const uint16_t *q_gain, *k_gain;  // [dim] or null
  const int32_t* positions;
  const uint64_t* turns;            // [rot / 2]
  float eps;
  int n_tokens, heads, kv_heads, dim, rot;
  // For Q and for K: log2 of the tokens that a warp takes, the most of their heads that it does, and warps for all of these
  int tokens_log2[2], span[2];
  unsigned int spans[2], q_warps;   // q_warps: of Q
};

MV_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Eight bf16 as four pairs of fp32, and back
MV_DEV void unpack8(const uint4& w, uint64_t (&f)[4]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pack2(bf16lo(x[i]), bf16hi(x[i]));
}
MV_DEV uint4 pack8(const uint64_t (&f)[4]) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2(f[i]);
    x[i] = pack_bf16x2(v.x, v.y);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

MV_DEV void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MV_DEV uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// kLanes threads a row, the power of two from dim / 16 up. kNeighbours: pairs (2 i, 2 i + 1).
template <int kLanes, bool kNeighbours>
__global__ void __launch_bounds__(kThreads, kResident) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int kGroups = 32 / kLanes;
  __shared__ uint4 s_x[kAhead][2][kThreads];  // each thread's pieces on their way
  const int j = threadIdx.x % kLanes, group = threadIdx.x % 32 / kLanes;
  const unsigned int unit = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const bool mine = j < a.dim / 16;
  // this lane's pieces of 8 elements: pairs of halves meet across R/2 elements, what is not turned lies side by side
  const bool rot = mine && j < a.rot / 16;
  const int e0 = kNeighbours || !rot ? 16 * j : 8 * j, e1 = kNeighbours || !rot ? 16 * j + 8 : 8 * j + a.rot / 2;
  const int is_k = unit >= a.q_warps, log2 = a.tokens_log2[is_k], per_token = kGroups >> log2;  // groups of a token
  const unsigned int mine_of = is_k ? unit - a.q_warps : unit, block = mine_of / a.spans[is_k];
  const int h_from = (int)(mine_of - block * a.spans[is_k]) * a.span[is_k], heads = is_k ? a.kv_heads : a.heads;
  const int h_to = min(h_from + a.span[is_k], heads);
  const int64_t t_first = (int64_t)block << log2, t = t_first + group / per_token;
  const bool real = t < a.n_tokens;
  pdl_trigger();
  pdl_wait();
  if (t_first >= a.n_tokens) return;  // the whole warp
  const int pos = !real ? -1 : a.positions ? __ldcg(a.positions + t) : 0;
  const int h_first = h_from + group % per_token;
  const RowsArgs& from = is_k ? a.k : a.q;
  const uint16_t* src = from.p + t * from.ts + h_first * from.hs;
  const int64_t src_add = from.hs * per_token;
  const uint32_t mem = smem_u32(&s_x[0][0][threadIdx.x]);
  int asked = real ? h_first : h_to;
  auto ask = [&](int slot) {
    if (asked < h_to && mine) {
      cp_async16(mem + slot * (2 * kThreads * 16), src + e0);
      cp_async16(mem + slot * (2 * kThreads * 16) + kThreads * 16, src + e1);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asked += per_token;
    src += src_add;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) ask(i);
  uint4 g0 = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), g1 = g0;
  const uint16_t* gain = is_k ? a.k_gain : a.q_gain;
  if (gain && mine) {
    g0 = *reinterpret_cast<const uint4*>(gain + e0);  // from L1 but for the first: 27 us in place of 77 for 8192 tokens
    g1 = *reinterpret_cast<const uint4*>(gain + e1);
  }
  uint64_t turns[8];
  if (rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turns[i] = a.turns[8 * j + i];
  }
  // The first piece's elements times `a0`, plus the other element of their pairs times `b0`; the second piece's `a1`, `b1`.
  // Pairs of halves: the other piece's element of the same place. Neighbours: the one beside it.
  uint64_t a0[4], a1[4], b0[4] = {}, b1[4] = {};
  unpack8(g0, a0);
  unpack8(g1, a1);
  if (rot) {
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int32_t part_of = (int32_t)((uint64_t)(uint32_t)pos * turns[e] >> 32);  // of a turn, -2^31 .. 2^31 - 1
      const float angle = (float)part_of * 1.4629180792671596e-09f;                 // 2 pi / 2^32
      c[e] = __cosf(angle);
      s[e] = __sinf(angle);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 u = unpack2(a0[e]), v = unpack2(a1[e]);
      if (kNeighbours) {
        a0[e] = pack2(u.x * c[e], u.y * c[e]);
        b0[e] = pack2(-u.y * s[e], u.x * s[e]);
        a1[e] = pack2(v.x * c[4 + e], v.y * c[4 + e]);
        b1[e] = pack2(-v.y * s[4 + e], v.x * s[4 + e]);
      } else {
        a0[e] = pack2(u.x * c[2 * e], u.y * c[2 * e + 1]);
        b0[e] = pack2(-v.x * s[2 * e], -v.y * s[2 * e + 1]);
        a1[e] = pack2(v.x * c[2 * e], v.y * c[2 * e + 1]);
        b1[e] = pack2(u.x * s[2 * e], u.y * s[2 * e + 1]);
      }
    }
  }
  const float inv = 1.0f / (float)a.dim;
  const RowsArgs& to = is_k ? a.k_out : a.q_out;
  uint16_t* dst = to.p + t * to.ts + h_first * to.hs;
  const int64_t dst_add = to.hs * per_token;
  int slot = 0;
#pragma unroll 1
  for (int h0 = h_from; h0 < h_to; h0 += per_token) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    uint64_t u[4] = {}, v[4] = {}, sums = 0;
    if (mine) {
      unpack8(lds16(mem + slot * (2 * kThreads * 16)), u);
      unpack8(lds16(mem + slot * (2 * kThreads * 16) + kThreads * 16), v);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sums = fma2(u[e], u[e], fma2(v[e], v[e], sums));
    float sum = unpack2(sums).x + unpack2(sums).y;
#pragma unroll
    for (int o = kLanes >> 1; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    ask(slot);
    slot = slot + 1 == kAhead ? 0 : slot + 1;
    // first of all by the row's factor: |x| times it is sqrt(D) at most, while x times a gain may leave fp32's range
    const float by = rsqrtf(sum * inv + a.eps);
    uint64_t y0[4], y1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = mul2(u[e], pack2(by, by));
      v[e] = mul2(v[e], pack2(by, by));
      y0[e] = mul2(u[e], a0[e]);
      y1[e] = mul2(v[e], a1[e]);
    }
    if (rot)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = unpack2(u[e]), r = unpack2(v[e]);
        y0[e] = fma2(kNeighbours ? pack2(p.y, p.x) : v[e], b0[e], y0[e]);
        y1[e] = fma2(kNeighbours ? pack2(r.y, r.x) : u[e], b1[e], y1[e]);
      }
    if (mine && h0 + group % per_token < h_to && pos >= 0) {
      *reinterpret_cast<uint4*>(dst + e0) = pack8(y0);
      *reinterpret_cast<uint4*>(dst + e1) = pack8(y1);
    }
    dst += dst_add;
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
  if (rot_dim && ((!positions && n_tokens) || !turns || (reinterpret_cast<uintptr_t>(turns) & 7))) return MV_ERR_INVALID_ARG;
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
  // Fewer heads than a warp has groups: several tokens a warp. More: as many rounds of heads as leave kWarpsWanted warps to
  // every SM.
  const int groups = 32 / lanes;
  const int64_t warps = (int64_t)mv_sm_count() * kWarpsWanted;
  int64_t rounds = 0, all = 0;  // of a warp that does a token's heads, in all
  for (int i = 0; i < 2; ++i) {
    const int heads = i ? n_kv_heads : n_heads;
    a.tokens_log2[i] = 0;
    while (heads && groups >> (a.tokens_log2[i] + 1) >= heads) ++a.tokens_log2[i];
    const int per_token = groups >> a.tokens_log2[i];
    rounds = (heads + per_token - 1) / per_token;
    all += rounds * (((int64_t)n_tokens >> a.tokens_log2[i]) + 1);
  }
  const int64_t most = std::max<int64_t>(1, (all + warps - 1) / warps);
  int64_t total = 0;
  for (int i = 0; i < 2; ++i) {
    const int heads = i ? n_kv_heads : n_heads, per_token = groups >> a.tokens_log2[i];
    rounds = (heads + per_token - 1) / per_token;
    a.span[i] = per_token * (int)std::min(std::max<int64_t>(1, rounds), most);
    a.spans[i] = std::max(1, (heads + a.span[i] - 1) / a.span[i]);
    if (i == 1) a.q_warps = (unsigned int)total;
    if (heads) total += (((int64_t)n_tokens + (1 << a.tokens_log2[i]) - 1) >> a.tokens_log2[i]) * a.spans[i];
  }
  // (below 2^32: two warps a token where there are that many)
  const int64_t ctas = (total * 32 + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)ctas);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = lanes == 16  ? launch_rope<16>(a, grid, neighbours, st)
                        : lanes == 8 ? launch_rope<8>(a, grid, neighbours, st)
                        : lanes == 4 ? launch_rope<4>(a, grid, neighbours, st)
                        : lanes == 2 ? launch_rope<2>(a, grid, neighbours, st)
                                     : launch_rope<1>(a, grid, neighbours, st);
  return e == cudaSuccess ? mv_last_launch("qk_norm_rope") : MV_ERR_CUDA;
}
