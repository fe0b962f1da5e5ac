// 8-bit paged key/value cache: writing rows and reading rows back.
#include "kv8.cuh"

namespace dfk {

// Eight consecutive elements of a row.  (Plain loads, here and below: the
// kernel may have started before the one that writes the rows had finished.)
__device__ __forceinline__ void kv8_load8(const float* p, float* x) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void kv8_load8(const __nv_bfloat16* p, float* x) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
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
__global__ void __launch_bounds__(KV8_THREADS) kv8_write_kernel(Kv8Geom g, const T* k,
                                                                const T* v, long long ks, long long vs) {
  constexpr int LPV = HD / 8;                    // lanes per vector
  constexpr int VPP = KV8_THREADS / LPV;         // vectors per pass
  constexpr int PASSES = 2 * KV8_GROUP / VPP;
  __shared__ __align__(16) uint8_t sV[KV8_GROUP][HD];
  __shared__ uint8_t sE[KV8_GROUP][2];
  pdl_trigger();
  pdl_wait();
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
__global__ void __launch_bounds__(KV8_THREADS) kv8_read_kernel(Kv8Geom g, T* k, T* v) {
  constexpr int LPV = HD / 8;
  constexpr int VPP = KV8_THREADS / LPV;
  constexpr int PASSES = 2 * KV8_GROUP / VPP;
  __shared__ __align__(16) uint8_t sV[KV8_GROUP][HD];
  pdl_trigger();
  pdl_wait();
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

// ------------------------------------------------------------- entry points
template <typename T>
static cudaError_t launch_kv8_write(const Kv8Geom& g, const void* k, const void* v, long long ks, long long vs,
                                    cudaStream_t st) {
  return launch_k(g.hd == 128 ? kv8_write_kernel<T, 128> : kv8_write_kernel<T, 64>,
                  dim3(kv8_units(g.rows, g.nseq), g.heads), dim3(KV8_THREADS), 0, st, g, (const T*)k, (const T*)v, ks, vs);
}
template <typename T>
static cudaError_t launch_kv8_read(const Kv8Geom& g, void* k, void* v, cudaStream_t st) {
  return launch_k(g.hd == 128 ? kv8_read_kernel<T, 128> : kv8_read_kernel<T, 64>,
                  dim3(kv8_units(g.rows, g.nseq), g.heads), dim3(KV8_THREADS), 0, st, g, (T*)k, (T*)v);
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

}  // extern "C"
