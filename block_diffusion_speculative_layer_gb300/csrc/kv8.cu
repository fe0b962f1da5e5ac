// 8-bit paged key/value cache: writing rows, reading rows back, and the
// attention of a chunk of new tokens over it (the format and the addressing
// are described in dflash.h).
//
// The scale of a vector is a power of two.  e4m3 is a floating format, so the
// scale only places its range and a power of two loses no precision against
// max|x| / 448; scaling, unscaling and widening to bf16 or f16 are then exact,
// and the one rounding of the whole path is the e4m3 rounding itself.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"
#include "dflash.h"
#include "internal.h"

namespace dfk {

// What every kernel of this file knows about the call's rows and the cache.
struct Kv8Geom {
  uint8_t* codes;
  uint8_t* exps;
  const int* page_table;
  const int* row_start;
  const int* kv_len;
  int* err;
  int n_pages, page_tokens, heads, hd, pt_stride, nseq, rows;
};

constexpr int KV8_GROUP = 16;  // tokens whose values lie together, transposed
constexpr int KV8_NAN = 255;   // exponent byte of a vector that holds no numbers
constexpr int KV8_BIAS = 127;
constexpr int KV8_EMIN = -100, KV8_EMAX = 119;  // keeps c * 2^e finite and normal in bf16 and fp32

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
__device__ __forceinline__ int kv8_unit_seq(const Kv8Geom& g, int unit) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int i = 0; i < g.nseq; i += 32) {
    const int s = i + lane;
    const bool le = s < g.nseq && (g.row_start[s] >> 4) + 2 * s <= unit;
    before += __popc(__ballot_sync(0xffffffffu, le));
  }
  return before - 1;
}

// The page of position `pos` of sequence s, or -1 (and the error bit).
__device__ __forceinline__ int kv8_page(const Kv8Geom& g, int s, int pos) {
  const int page = g.page_table[(size_t)s * g.pt_stride + pos / g.page_tokens];
  if (page >= 0 && page < g.n_pages) return page;
  flag_error(g.err, ERR_BOUNDS);
  return -1;
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

// Eight consecutive elements of a row.
__device__ __forceinline__ void kv8_load8(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void kv8_load8(const __nv_bfloat16* p, float* x) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void kv8_store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void kv8_store8(__nv_bfloat16* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Write: one block per (16-token group, head).  HD / 8 lanes hold a vector,
// eight elements each; the keys go straight to their rows, the values meet in
// shared memory so that a whole group leaves as 16-byte rows of the
// transposed plane (a partly written group byte by byte: its other tokens'
// bytes are not this call's).
constexpr int KV8_THREADS = 128;
template <typename T, int HD>
__global__ void __launch_bounds__(KV8_THREADS) kv8_write_kernel(Kv8Geom g, const T* __restrict__ k,
                                                                const T* __restrict__ v, long long ks, long long vs) {
  constexpr int LPV = HD / 8;                    // lanes per vector
  constexpr int VPP = KV8_THREADS / LPV;         // vectors per pass
  constexpr int PASSES = 2 * KV8_GROUP / VPP;
  __shared__ __align__(16) uint8_t sV[KV8_GROUP][HD];
  __shared__ uint8_t sE[KV8_GROUP][2];
  const int s = kv8_unit_seq(g, blockIdx.x), head = blockIdx.y;
  if (s < 0) return;
  Kv8Seq q;
  const bool ok = kv8_seq(g, s, q);
  const int group = (q.pos0 >> 4) + ((int)blockIdx.x - (q.row0 >> 4) - 2 * s);
  if (!ok) {
    if (threadIdx.x == 0) flag_error(g.err, ERR_BOUNDS);
    return;
  }
  const int t0 = max(max(group * KV8_GROUP, q.pos0), 0);
  const int t1 = min((group + 1) * KV8_GROUP, q.pos0 + q.n);
  if (t0 >= t1) return;
  const int page = kv8_page(g, s, t0);
  if (page < 0) return;
  const int slot0 = (group * KV8_GROUP) % g.page_tokens;
  const int sub = threadIdx.x % LPV;
  float x[PASSES][8];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {  // all loads first
    const int vec = threadIdx.x / LPV + i * VPP, pos = group * KV8_GROUP + (vec >> 1);
    const bool here = pos >= t0 && pos < t1;
    const size_t row = here ? (size_t)(q.row0 + pos - q.pos0) : 0;
    const T* src = ((vec & 1) ? v + row * vs : k + row * ks) + head * HD + sub * 8;
    if (here) {
      kv8_load8(src, x[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int vec = threadIdx.x / LPV + i * VPP, t = vec >> 1, kv = vec & 1;
    // largest magnitude as bits: infinities and NaNs are above every number
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool nan = top >= 0x7F800000u;
    const int e2 = kv8_exponent(__uint_as_float(top));
    const float inv = nan ? 0.f : kv8_pow2(-e2);
    uint32_t lo = 0, hi = 0;
    if (!nan) {
      lo = kv8_pack4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
      hi = kv8_pack4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
    }
    const int pos = group * KV8_GROUP + t;
    if (kv == 0) {
      if (pos >= t0 && pos < t1)
        *reinterpret_cast<uint2*>(g.codes + kv8_code_at(g, page, 0, head) + (size_t)(slot0 + t) * HD + sub * 8) =
            make_uint2(lo, hi);
    } else {
      *reinterpret_cast<uint2*>(&sV[t][sub * 8]) = make_uint2(lo, hi);
    }
    if (sub == 0) sE[t][kv] = (uint8_t)(nan ? KV8_NAN : e2 + KV8_BIAS);
  }
  __syncthreads();
  const int lo = t0 - group * KV8_GROUP, hi = t1 - group * KV8_GROUP;
  if ((int)threadIdx.x < HD) {
    const int d = threadIdx.x;
    uint8_t* dst = g.codes + kv8_code_at(g, page, 1, head) + ((size_t)(slot0 >> 4) * HD + d) * KV8_GROUP;
    if (hi - lo == KV8_GROUP) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)sV[4 * i][d] | ((uint32_t)sV[4 * i + 1][d] << 8) | ((uint32_t)sV[4 * i + 2][d] << 16) |
               ((uint32_t)sV[4 * i + 3][d] << 24);
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int t = lo; t < hi; ++t) dst[t] = sV[t][d];
    }
  }
  const int t = threadIdx.x;
  if (t >= lo && t < hi)
    *reinterpret_cast<uint16_t*>(g.exps + kv8_exp_at(g, page, head, slot0 + t)) =
        (uint16_t)(sE[t][0] | ((uint32_t)sE[t][1] << 8));
}

// Read: the same units, the other way.  The value plane is transposed through
// shared memory, so both outputs leave in rows.
template <typename T, int HD>
__global__ void __launch_bounds__(KV8_THREADS) kv8_read_kernel(Kv8Geom g, T* __restrict__ k, T* __restrict__ v) {
  constexpr int LPV = HD / 8;
  constexpr int VPP = KV8_THREADS / LPV;
  constexpr int PASSES = 2 * KV8_GROUP / VPP;
  __shared__ __align__(16) uint8_t sV[KV8_GROUP][HD];
  const int s = kv8_unit_seq(g, blockIdx.x), head = blockIdx.y;
  if (s < 0) return;
  Kv8Seq q;
  const bool ok = kv8_seq(g, s, q);
  const int group = (q.pos0 >> 4) + ((int)blockIdx.x - (q.row0 >> 4) - 2 * s);
  if (!ok) {
    if (threadIdx.x == 0) flag_error(g.err, ERR_BOUNDS);
    return;
  }
  const int t0 = max(group * KV8_GROUP, q.pos0), t1 = min((group + 1) * KV8_GROUP, q.pos0 + q.n);
  if (t0 >= t1) return;
  // a group before position 0 is padding: no page, zeros
  const int page = group >= 0 ? kv8_page(g, s, group * KV8_GROUP) : -1;
  const int slot0 = group >= 0 ? (group * KV8_GROUP) % g.page_tokens : 0;
  uint2 kc[PASSES];
  int ex[PASSES];
  const int sub = threadIdx.x % LPV;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int vec = threadIdx.x / LPV + i * VPP, t = vec >> 1;
    kc[i] = make_uint2(0, 0);
    ex[i] = 0;
    if (page >= 0) {
      if (!(vec & 1))
        kc[i] = *reinterpret_cast<const uint2*>(g.codes + kv8_code_at(g, page, 0, head) + (size_t)(slot0 + t) * HD +
                                                sub * 8);
      ex[i] = g.exps[kv8_exp_at(g, page, head, slot0 + t) + (vec & 1)];
    }
  }
  if (page >= 0 && (int)threadIdx.x < HD) {
    const int d = threadIdx.x;
    const uint4 w = *reinterpret_cast<const uint4*>(g.codes + kv8_code_at(g, page, 1, head) +
                                                    ((size_t)(slot0 >> 4) * HD + d) * KV8_GROUP);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int t = 0; t < KV8_GROUP; ++t) sV[t][d] = (uint8_t)(a[t >> 2] >> (8 * (t & 3)));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int vec = threadIdx.x / LPV + i * VPP, t = vec >> 1, kv = vec & 1, pos = group * KV8_GROUP + t;
    if (pos < t0 || pos >= t1) continue;
    float x[8];
    const uint2 c = kv ? *reinterpret_cast<const uint2*>(&sV[t][sub * 8]) : kc[i];
    const float sc = kv8_scale(ex[i]);
    const uint32_t two[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = kv8_value2(two[e]);
      x[2 * e] = page >= 0 ? f.x * sc : 0.f;
      x[2 * e + 1] = page >= 0 ? f.y * sc : 0.f;
    }
    T* dst = (kv ? v : k) + ((size_t)(q.row0 + pos - q.pos0) * g.heads + head) * HD + sub * 8;
    kv8_store8(dst, x);
  }
}

// Attention.
struct Kv8Attn {
  Kv8Geom g;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  long long qs, os;
  int q_heads, max_rows, causal, window;
  float scale;
};

// One warp per (row, query head), 32 positions at a time: a lane scores one
// position, then holds HD / 32 dims of the output.
template <int HD>
__global__ void __launch_bounds__(128) kv8_attention_kernel(Kv8Attn a) {
  const Kv8Geom& g = a.g;
  __shared__ float sq[4][HD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.z, hq = blockIdx.y, j = blockIdx.x * 4 + warp;
  Kv8Seq q;
  if (!kv8_seq(g, s, q) || q.n > a.max_rows) {
    if (threadIdx.x == 0) flag_error(g.err, ERR_BOUNDS);
    return;
  }
  if (j >= q.n) return;
  const int row = q.row0 + j, pos = q.pos0 + j, head = hq / (a.q_heads / g.heads);
  int lo = 0, hi = a.causal ? pos : q.pos0 + q.n - 1;
  if (a.window > 0) lo = max(0, pos - a.window + 1);
  if (pos < 0) hi = -1;
  for (int d = lane; d < HD; d += 32) sq[warp][d] = __bfloat162float(a.q[row * a.qs + hq * HD + d]);
  __syncwarp();
  constexpr int ND = HD / 32;
  float o[ND] = {}, m = -INFINITY, l = 0.f;
  const float sc2 = a.scale * 1.4426950408889634f;
  for (int t0 = lo & ~31; t0 <= hi; t0 += 32) {
    const int t = t0 + lane;
    float x = -INFINITY, vscale = 0.f;
    int page = -1;
    if (t >= lo && t <= hi) page = kv8_page(g, s, t);
    if (page >= 0) {
      const int slot = t % g.page_tokens;
      const uint4* kr = reinterpret_cast<const uint4*>(g.codes + kv8_code_at(g, page, 0, head) + (size_t)slot * HD);
      const uint8_t* ep = g.exps + kv8_exp_at(g, page, head, slot);
      float dot = 0.f;
      for (int i = 0; i < HD / 16; ++i) {
        const uint4 w = kr[i];
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f0 = kv8_value2(ws[e] & 0xFFFFu), f1 = kv8_value2(ws[e] >> 16);
          const float* qd = &sq[warp][i * 16 + e * 4];
          dot = fmaf(f0.x, qd[0], fmaf(f0.y, qd[1], fmaf(f1.x, qd[2], fmaf(f1.y, qd[3], dot))));
        }
      }
      x = dot * kv8_scale(ep[0]) * sc2;
      vscale = kv8_scale(ep[1]);
    }
    float mx = x;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    const float mn = fmaxf(m, mx);
    if (mn == -INFINITY && !__any_sync(0xffffffffu, x != x)) continue;
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float p = x == -INFINITY ? 0.f : exp2f(x - (mn == -INFINITY ? 0.f : mn));
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < ND; ++i) o[i] *= f;
    const float w = x == -INFINITY ? 0.f : p * vscale;
    for (int u = 0; u < 32; ++u) {
      const float wu = __shfl_sync(0xffffffffu, w, u);
      const int pu = __shfl_sync(0xffffffffu, page, u);
      if (pu < 0) continue;
      const int slot = (t0 + u) % g.page_tokens;
      const uint8_t* vr = g.codes + kv8_code_at(g, pu, 1, head) + (size_t)(slot >> 4) * HD * KV8_GROUP + (slot & 15);
#pragma unroll
      for (int i = 0; i < ND; ++i) o[i] = fmaf(wu, kv8_value2(vr[(lane + 32 * i) * KV8_GROUP]).x, o[i]);
    }
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
  const float inv = m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < ND; ++i) a.out[row * a.os + hq * HD + lane + 32 * i] = __float2bfloat16_rn(o[i] * inv);
  if (a.lse && lane == 0)
    a.lse[(size_t)row * a.q_heads + hq] = (m == -INFINITY ? (l == 0.f ? -INFINITY : l) : m * 0.6931471805599453f + logf(l));
}

// ------------------------------------------------------------- entry points
static bool kv8_aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The arguments all three calls share.
static bool kv8_geom_ok(const Kv8Geom& g) {
  return g.codes && g.exps && g.page_table && g.row_start && g.kv_len && g.n_pages >= 1 && g.page_tokens >= 16 &&
         g.page_tokens <= 1024 && g.page_tokens % 16 == 0 && g.heads >= 1 && g.heads <= 65535 &&
         (g.hd == 64 || g.hd == 128) && g.pt_stride >= 1 && (long long)g.pt_stride * g.page_tokens <= (1 << 30) &&
         (long long)g.n_pages * 2 * g.heads <= 0x7fffffff && kv8_aligned(g.codes, 16) && kv8_aligned(g.exps, 16) &&
         kv8_aligned(g.page_table, 4) && kv8_aligned(g.row_start, 4) && kv8_aligned(g.kv_len, 4) &&
         kv8_aligned(g.err, 4);
}

template <typename T>
static cudaError_t launch_kv8_write(const Kv8Geom& g, const void* k, const void* v, long long ks, long long vs,
                                    cudaStream_t st) {
  const dim3 grid(kv8_units(g.rows, g.nseq), g.heads);
  if (g.hd == 128)
    kv8_write_kernel<T, 128><<<grid, KV8_THREADS, 0, st>>>(g, (const T*)k, (const T*)v, ks, vs);
  else
    kv8_write_kernel<T, 64><<<grid, KV8_THREADS, 0, st>>>(g, (const T*)k, (const T*)v, ks, vs);
  return cudaGetLastError();
}
template <typename T>
static cudaError_t launch_kv8_read(const Kv8Geom& g, void* k, void* v, cudaStream_t st) {
  const dim3 grid(kv8_units(g.rows, g.nseq), g.heads);
  if (g.hd == 128)
    kv8_read_kernel<T, 128><<<grid, KV8_THREADS, 0, st>>>(g, (T*)k, (T*)v);
  else
    kv8_read_kernel<T, 64><<<grid, KV8_THREADS, 0, st>>>(g, (T*)k, (T*)v);
  return cudaGetLastError();
}

}  // namespace dfk

using namespace dfk;

extern "C" {

df_status df_op_kv8_write(const void* k_dev, const void* v_dev, int32_t dtype, int32_t rows, int64_t k_stride,
                          int64_t v_stride, void* codes_dev, void* exps_dev, int32_t n_pages, int32_t page_tokens,
                          int32_t n_kv_heads, int32_t head_dim, const int32_t* page_table_dev, int32_t pt_stride,
                          const int32_t* row_start_dev, const int32_t* kv_len_dev, int32_t nseq, int32_t* err_dev,
                          void* stream) {
  const Kv8Geom g{(uint8_t*)codes_dev, (uint8_t*)exps_dev, page_table_dev, row_start_dev, kv_len_dev, err_dev,
                  n_pages, page_tokens, n_kv_heads, head_dim, pt_stride, nseq, rows};
  if ((dtype != DF_FP32 && dtype != DF_BF16) || rows < 0 || nseq < 0 || nseq > (1 << 20)) return DF_EINVAL;
  if (rows == 0 || nseq == 0) return DF_OK;
  if (!k_dev || !v_dev || !kv8_geom_ok(g) || !kv8_aligned(k_dev, 16) || !kv8_aligned(v_dev, 16)) return DF_EINVAL;
  const int per16 = dtype == DF_FP32 ? 4 : 8;  // elements in 16 bytes
  const long long width = (long long)n_kv_heads * head_dim;
  if (k_stride < width || v_stride < width || k_stride % per16 || v_stride % per16) return DF_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DF_FP32 ? launch_kv8_write<float>(g, k_dev, v_dev, k_stride, v_stride, st)
                                         : launch_kv8_write<__nv_bfloat16>(g, k_dev, v_dev, k_stride, v_stride, st);
  return e == cudaSuccess ? DF_OK : DF_ECUDA;
}

df_status df_op_kv8_read(const void* codes_dev, const void* exps_dev, int32_t n_pages, int32_t page_tokens,
                         int32_t n_kv_heads, int32_t head_dim, const int32_t* page_table_dev, int32_t pt_stride,
                         const int32_t* row_start_dev, const int32_t* kv_len_dev, int32_t nseq, int32_t rows,
                         int32_t dtype, void* k_dev, void* v_dev, int32_t* err_dev, void* stream) {
  const Kv8Geom g{(uint8_t*)codes_dev, (uint8_t*)exps_dev, page_table_dev, row_start_dev, kv_len_dev, err_dev,
                  n_pages, page_tokens, n_kv_heads, head_dim, pt_stride, nseq, rows};
  if ((dtype != DF_FP32 && dtype != DF_BF16) || rows < 0 || nseq < 0 || nseq > (1 << 20)) return DF_EINVAL;
  if (rows == 0 || nseq == 0) return DF_OK;
  if (!k_dev || !v_dev || !kv8_geom_ok(g) || !kv8_aligned(k_dev, 16) || !kv8_aligned(v_dev, 16)) return DF_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DF_FP32 ? launch_kv8_read<float>(g, k_dev, v_dev, st)
                                         : launch_kv8_read<__nv_bfloat16>(g, k_dev, v_dev, st);
  return e == cudaSuccess ? DF_OK : DF_ECUDA;
}

df_status df_op_attention_kv8(const void* q_dev, int64_t q_stride, void* out_dev, int64_t out_stride, float* lse_dev,
                              int32_t rows, int32_t n_q_heads, const void* codes_dev, const void* exps_dev,
                              int32_t n_pages, int32_t page_tokens, int32_t n_kv_heads, int32_t head_dim,
                              const int32_t* page_table_dev, int32_t pt_stride, const int32_t* row_start_dev,
                              const int32_t* kv_len_dev, int32_t nseq, int32_t max_rows, int32_t max_len, float scale,
                              int32_t causal, int32_t window, int32_t cluster_ctas, int32_t* err_dev, void* stream) {
  Kv8Attn a{};
  a.g = Kv8Geom{(uint8_t*)codes_dev, (uint8_t*)exps_dev, page_table_dev, row_start_dev, kv_len_dev, err_dev,
                n_pages, page_tokens, n_kv_heads, head_dim, pt_stride, nseq, rows};
  if (rows < 0 || nseq < 0 || nseq > 65535 || max_rows < 0 || max_len < 0 || (causal != 0 && causal != 1) ||
      window < 0 || (window > 0 && !causal) || !isfinite(scale))
    return DF_EINVAL;
  if (cluster_ctas != 0 && cluster_ctas != 1 && cluster_ctas != 2 && cluster_ctas != 4 && cluster_ctas != 8 &&
      cluster_ctas != 16)
    return DF_EINVAL;
  if (rows == 0 || nseq == 0 || max_rows == 0) return DF_OK;
  if (!q_dev || !out_dev || !kv8_geom_ok(a.g) || !kv8_aligned(q_dev, 16) || !kv8_aligned(out_dev, 16) ||
      !kv8_aligned(lse_dev, 4))
    return DF_EINVAL;
  if (n_q_heads < n_kv_heads || n_q_heads % n_kv_heads || n_q_heads > 65535) return DF_EINVAL;
  const long long width = (long long)n_q_heads * head_dim;
  if (q_stride < width || out_stride < width || q_stride % 8 || out_stride % 8) return DF_EINVAL;
  a.q = reinterpret_cast<const __nv_bfloat16*>(q_dev);
  a.out = reinterpret_cast<__nv_bfloat16*>(out_dev);
  a.lse = lse_dev;
  a.qs = q_stride;
  a.os = out_stride;
  a.q_heads = n_q_heads;
  a.max_rows = max_rows < rows ? max_rows : rows;
  a.causal = causal;
  a.window = window;
  a.scale = scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((a.max_rows + 3) / 4, n_q_heads, nseq);
  if (head_dim == 128)
    kv8_attention_kernel<128><<<grid, 128, 0, st>>>(a);
  else
    kv8_attention_kernel<64><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ECUDA;
}

}  // extern "C"
