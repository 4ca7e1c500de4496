// The paged cache as kernels see it, and the checks that its entry points share.
#pragma once

#include <math.h>

#include "common.cuh"

constexpr int kPagedMaxSeq = 4096, kPagedMaxHeads = 256, kPagedMaxDim = 128, kPagedMaxPage = 1024;

constexpr float kLog2E = 1.4426950408889634f;

// Sites of the device error word.
constexpr uint32_t kPagedRowsSite = 40, kPagedAttnSite = 41, kPagedResizeSite = 42;

// What a pool holds: bf16, or values of 8 bits with an exponent for each row, or of 4 bits with a scale for each group.
enum PagedFormat { kBf16 = 0, kE4M3 = 1, kE2M1 = 2 };
constexpr int kGroup = 16;          // elements of a 4-bit row that share a scale byte
constexpr uint32_t kTopScale = 0xE2u;  // 10240: 6 times as much is in fp16's range
constexpr uint32_t kNanScale = 0xFFu;

struct PagedArgs {
  uint8_t *k, *v;            // pages [n_pages][heads][page_size][dim] of 1 or 2 bytes, or 4 bits, an element
  uint8_t *k_exp, *v_exp;    // [n_pages][heads][page_size], e4m3; [n_pages][heads][page_size][dim / kGroup], e2m1
  const int32_t* table;      // [n_seq][ld_table]
  const int32_t* seq_lens;   // [n_seq]
  int n_pages, page_size, heads, dim;
  int ld_table, max_pages, n_seq;
};

struct RowsArgs {
  uint16_t* p;
  int64_t ts, hs;  // token and head stride, elements
};

inline bool mv_rows_ok(const mv_rows& r, int64_t tokens, int heads, int dim) {
  if (!r.ptr || (reinterpret_cast<uintptr_t>(r.ptr) & 15)) return false;
  if (r.token_stride < 0 || r.head_stride < 0 || (r.token_stride & 7) || (r.head_stride & 7)) return false;
  if (tokens > 1 && r.token_stride < dim) return false;
  if (heads > 1 && r.head_stride < dim) return false;
  // offsets stay inside 63 bits (at most 2^31 tokens and 2^8 heads), strides inside the 2^40 bytes of a tensor map
  return r.token_stride < (int64_t(1) << 30) && r.head_stride < (int64_t(1) << 39);
}

// Rows that a call writes: as above, and no two of them overlap.
inline bool mv_out_rows_ok(const mv_rows& r, int64_t tokens, int heads, int dim) {
  if (!mv_rows_ok(r, tokens, heads, dim)) return false;
  if (tokens == 1 || heads == 1) return true;
  return r.token_stride >= (heads - 1) * r.head_stride + dim || r.head_stride >= (tokens - 1) * r.token_stride + dim;
}

// The cache, the table and the lengths of a call; *a is filled in on MV_OK. n_seq > 0 here.
inline mv_status mv_paged_check(const mv_paged_kv* c, const int32_t* table, int32_t ld_table, int32_t max_pages,
                                const int32_t* seq_lens, int32_t n_seq, PagedArgs* a) {
  if (!c || !c->k || !c->v || !table || !seq_lens) return MV_ERR_INVALID_ARG;
  if (c->dtype != MV_DTYPE_BF16 && c->dtype != MV_DTYPE_E4M3 && c->dtype != MV_DTYPE_E2M1) return MV_ERR_INVALID_ARG;
  if (c->dtype != MV_DTYPE_BF16 && (!c->k_exp || !c->v_exp)) return MV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15) return MV_ERR_INVALID_ARG;
  if (c->dtype != MV_DTYPE_BF16 &&
      ((reinterpret_cast<uintptr_t>(c->k_exp) | reinterpret_cast<uintptr_t>(c->v_exp)) & 15))
    return MV_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_size < 16 || c->page_size > kPagedMaxPage || c->page_size % 16) return MV_ERR_SHAPE;
  if (c->n_kv_heads < 1 || c->n_kv_heads > kPagedMaxHeads) return MV_ERR_SHAPE;
  if (c->head_dim < 16 || c->head_dim > kPagedMaxDim || c->head_dim % (c->dtype == MV_DTYPE_E2M1 ? 32 : 16)) return MV_ERR_SHAPE;
  if (max_pages < 1 || ld_table < max_pages || n_seq > kPagedMaxSeq) return MV_ERR_SHAPE;
  if ((int64_t)max_pages * c->page_size > 0x7fffffff - 1024) return MV_ERR_SHAPE;
  a->k = static_cast<uint8_t*>(c->k);
  a->v = static_cast<uint8_t*>(c->v);
  a->k_exp = c->k_exp;
  a->v_exp = c->v_exp;
  a->table = table;
  a->seq_lens = seq_lens;
  a->n_pages = c->n_pages;
  a->page_size = c->page_size;
  a->heads = c->n_kv_heads;
  a->dim = c->head_dim;
  a->ld_table = ld_table;
  a->max_pages = max_pages;
  a->n_seq = n_seq;
  return MV_OK;
}

// Two e4m3 values (low byte first) as two halves, exactly.
MV_DEV uint32_t e4m3x2_to_half2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
// (lo, hi) rounded to e4m3, nearest even; what is over 448 becomes 448
MV_DEV uint16_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
MV_DEV float2 half2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// 2^(byte - 127). Bytes written by paged_kv_append lie in 27 .. 247; any byte gives its power (0: 2^-127).
MV_DEV float exp_byte_scale(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// A scale byte has the exponent and the first three fraction bits of an fp16 value: byte << 7 is that value.
// The byte of the scale nearest to x >= 0, finite: ties to even, at most kTopScale.
MV_DEV uint32_t scale_byte(float x) {
  const uint32_t b = __float_as_uint(x);
  if (x < 0x1p-14f) return (uint32_t)__float2int_rn(x * 0x1p17f);  // multiples of 2^-17; 8 of them are 0x08, 2^-14
  return min(kTopScale, ((b + 0x7ffffu + ((b >> 20) & 1u)) >> 20) - (112u << 3));
}
MV_DEV float scale_value(uint32_t byte) { return half2_to_float2(byte << 7).x; }
// Four elements as e2m1 (first one in the low 4 bits), nearest even; what is over 6 becomes 6
MV_DEV uint32_t float4_to_e2m1x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b8 x, y;\n\tcvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 y, %4, %3;\n\t"
      "mov.b32 %0, {x, y, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// The eight e2m1 values of a word as halves, exactly: h[i] has elements 2 i and 2 i + 1
MV_DEV void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
