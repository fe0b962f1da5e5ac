// 8-bit paged key/value cache: what its writer, reader and attention share
// (the format and the addressing are described in dflash.h).
//
// The scale of a vector is a power of two.  e4m3 is a floating format, so the
// scale only places its range and a power of two loses no precision against
// max|x| / 448; scaling, unscaling and widening to bf16 or f16 are then exact,
// and the one rounding of the whole path is the e4m3 rounding itself.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "dflash.h"
#include "internal.h"

namespace dfk {

// What every kernel of the cache knows about the call's rows and the cache.
struct Kv8Geom {
  uint8_t* codes;
  uint8_t* exps;
  const int* page_table;
  const int* row_start;
  const int* kv_len;
  int* err;
  int n_pages, page_tokens, heads, hd, pt_stride, nseq, rows;
  unsigned long long per_page;  // 2^32 / (groups of 16 tokens of a page), rounded up
};

constexpr int KV8_GROUP = 16;  // tokens whose values lie together, transposed
constexpr int KV8_NAN = 255;   // exponent byte of a vector that holds no numbers
constexpr int KV8_BIAS = 127;
constexpr int KV8_EMIN = -100, KV8_EMAX = 119;  // keeps c * 2^e finite and normal in bf16 and fp32

// The page-table entry of a sequence's 16-token group: exact for a group below
// 2^26 and at most 64 groups to a page.
inline unsigned long long kv8_per_page(int page_tokens) {
  return ((1ull << 32) + page_tokens / KV8_GROUP - 1) / (page_tokens / KV8_GROUP);
}
__device__ __forceinline__ int kv8_entry(const Kv8Geom& g, int group) {
  return (int)(((unsigned long long)(unsigned)group * g.per_page) >> 32);
}

// One sequence's rows: first row, number of rows, position of the first.
struct Kv8Seq {
  int row0, n, pos0;
};
// False (and the error bit) if the sequence's entries are out of range.
__device__ __forceinline__ bool kv8_seq(const Kv8Geom& g, int s, Kv8Seq& q) {
  const int a = g.row_start[s], b = g.row_start[s + 1], len = g.kv_len[s];
  q.row0 = a;
  q.n = b - a;
  q.pos0 = len - (b - a);
  return a >= 0 && b >= a && b <= g.rows && len >= 0 && len <= (long long)g.pt_stride * g.page_tokens;
}

// Sequence s owns the units from row_start[s] / 16 + 2 s on: its rows touch
// at most n / 16 + 2 aligned 16-token groups, so the units of two sequences
// never meet and no block has to add up the sequences before its own.
__host__ __device__ inline int kv8_units(int rows, int nseq) { return rows / KV8_GROUP + 2 * nseq; }
// The unit's sequence (or -1): the last one whose units do not start behind
// it, by a search over 32 sequences at a time.
__device__ __forceinline__ int kv8_unit_seq(const Kv8Geom& g, int unit) {
  const int lane = threadIdx.x & 31;
  int first = 0, n = g.nseq;  // it is among the n from `first` on, if any
  for (;;) {
    const int step = (n + 31) / 32, s = first + lane * step;
    const bool le = lane * step < n && (g.row_start[s] >> 4) + 2 * s <= unit;
    const int last = __popc(__ballot_sync(0xffffffffu, le)) - 1;
    if (last < 0 || step == 1) return first + last;
    first += last * step;
    n = min(step, n - last * step);
  }
}

__device__ __forceinline__ size_t kv8_code_at(const Kv8Geom& g, int page, int kv, int head) {
  return ((size_t)(page * 2 + kv) * g.heads + head) * g.page_tokens * g.hd;
}
__device__ __forceinline__ size_t kv8_exp_at(const Kv8Geom& g, int page, int head, int slot) {
  return (((size_t)page * g.heads + head) * g.page_tokens + slot) * 2;
}

// Exponent of a vector whose largest magnitude is `amax` (finite, >= 0): the
// smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int kv8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, KV8_EMIN), KV8_EMAX);
}
__device__ __forceinline__ float kv8_pow2(int e) { return __uint_as_float((uint32_t)(e + KV8_BIAS) << 23); }
// 2^(b - 127) of an exponent byte; NaN for a vector without numbers.
__device__ __forceinline__ float kv8_scale(int b) {
  return __uint_as_float(b == KV8_NAN ? 0x7FC00000u : (uint32_t)b << 23);
}

// Four e4m3 codes of four floats (to nearest even; magnitudes above 448 saturate).
__device__ __forceinline__ uint32_t kv8_pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Two codes (the low 16 bits) widened to f16, exactly.
__device__ __forceinline__ uint32_t kv8_widen2(uint32_t two) {
  uint32_t r;
  const uint16_t h = (uint16_t)two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
  return r;
}
__device__ __forceinline__ float2 kv8_value2(uint32_t two) {
  const uint32_t r = kv8_widen2(two);
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

inline bool kv8_aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The arguments all three calls share.
inline bool kv8_geom_ok(const Kv8Geom& g) {
  return g.codes && g.exps && g.page_table && g.row_start && g.kv_len && g.n_pages >= 1 && g.page_tokens >= 16 &&
         g.page_tokens <= 1024 && g.page_tokens % 16 == 0 && g.heads >= 1 && g.heads <= 65535 &&
         (g.hd == 64 || g.hd == 128) && g.pt_stride >= 1 && (long long)g.pt_stride * g.page_tokens <= (1 << 30) &&
         (long long)g.n_pages * 2 * g.heads <= 0x7fffffff && kv8_aligned(g.codes, 16) && kv8_aligned(g.exps, 16) &&
         kv8_aligned(g.page_table, 4) && kv8_aligned(g.row_start, 4) && kv8_aligned(g.kv_len, 4) &&
         kv8_aligned(g.err, 4);
}

}  // namespace dfk
