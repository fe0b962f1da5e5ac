// 8-bit paged key/value cache: writing rows and reading rows back.
#include "kv8.cuh"

namespace dfk {

// Eight consecutive elements of a row, as they lie and as floats.  (Plain
// loads, here and below: the kernel may have started before the one that
// writes the rows had finished.)
template <typename T>
struct Kv8Raw;
template <>
struct Kv8Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  // bits of the largest magnitude in the vector, which LPV lanes hold:
  // infinities and NaNs are above every number
  template <int LPV>
  __device__ __forceinline__ uint32_t largest() const {
    float x[8];
    floats(x);
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
  }
  __device__ __forceinline__ void floats(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <>
struct Kv8Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  template <int LPV>
  __device__ __forceinline__ uint32_t largest() const {  // two at a time
    uint32_t top = __vmaxu2(__vmaxu2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu), __vmaxu2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = LPV / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
    return max(top & 0xFFFF0000u, top << 16);
  }
  __device__ __forceinline__ void floats(float* x) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
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

// Both kernels move bytes and wait for a chain of look-ups (which sequence,
// where it lies, which page) before the first of them.  A block takes a
// 16-token group of one head (write) or two (read) and has all its loads in
// flight at once.  Measured with 1, 2 and 4 heads to a block of 128 threads:
// writing 8192 rows of 8 heads 11.0, 11.0 and 12.2 us and 32 rows 3.5, 4.1 and
// 5.1, reading 16500 rows back 21, 18 and 18 us (the bytes alone: 7.4 and 15
// us).  A writer that keeps its rows as they lie until it uses them needs 32
// registers (fp32 vectors of 128: 40), which allows 16 blocks to an SM; most
// of its time is instructions (issue slots 75% busy at 13.2 us, before maxima
// were taken two at a time and addresses once for all rows).  A reader held
// to 12 blocks spills, 22 us.
constexpr int KV8_THREADS = 128, KV8_WRITE_HEADS = 1, KV8_READ_HEADS = 2;

// What a block works on: positions [t0, t1) of group `group` of sequence s,
// rows from q.row0 + pos - q.pos0, page (or -1) and slot of the group.
struct Kv8Unit {
  Kv8Seq q;
  int s, group, t0, t1, page, slot0;
};
constexpr int KV8_PADDING = -2147483647;
// The page, or -1 (and the error bit if it should have been one).
__device__ __forceinline__ int kv8_checked(const Kv8Geom& g, int page) {
  if (page >= 0 && page < g.n_pages) return page;
  if (page != KV8_PADDING) flag_error(g.err, ERR_BOUNDS);
  return -1;
}
// False: nothing to do.
__device__ __forceinline__ bool kv8_unit(const Kv8Geom& g, Kv8Unit& u) {
  u.s = kv8_unit_seq(g, blockIdx.x);
  if (u.s < 0) return false;
  if (!kv8_seq(g, u.s, u.q)) {
    if (threadIdx.x == 0) flag_error(g.err, ERR_BOUNDS);
    return false;
  }
  u.group = (u.q.pos0 >> 4) + ((int)blockIdx.x - (u.q.row0 >> 4) - 2 * u.s);
  u.t0 = max(u.group * KV8_GROUP, u.q.pos0);
  u.t1 = min((u.group + 1) * KV8_GROUP, u.q.pos0 + u.q.n);
  if (u.t0 >= u.t1) return false;
  // a group before position 0 is padding: it has no page (KV8_PADDING); the
  // look-up is checked by kv8_checked, after the loads that do not need it
  const int entry = u.group >= 0 ? kv8_entry(g, u.group) : 0;
  u.page = u.group >= 0 ? g.page_table[(size_t)u.s * g.pt_stride + entry] : KV8_PADDING;
  u.slot0 = u.group >= 0 ? u.group * KV8_GROUP - entry * g.page_tokens : 0;
  return true;
}

// Write: HD / 8 lanes hold a vector, eight elements each; the keys go straight
// to their rows, the values meet in shared memory so that a whole group leaves
// as 16-byte rows of the transposed plane (a partly written group byte by
// byte: its other tokens' bytes are not this call's).
template <typename T, int HD>
__global__ void __launch_bounds__(KV8_THREADS, (HD * sizeof(T) > 256 ? 12 : 16))
    kv8_write_kernel(Kv8Geom g, const T* k, const T* v, long long ks, long long vs) {
  constexpr int HEADS = KV8_WRITE_HEADS;  // per block
  constexpr int LPV = HD / 8;             // lanes per vector
  constexpr int VPP = KV8_THREADS / LPV;  // vectors per pass
  constexpr int PASSES = 2 * KV8_GROUP * HEADS / VPP;
  __shared__ __align__(16) uint8_t sV[HEADS][KV8_GROUP][HD];
  __shared__ uint8_t sE[HEADS][KV8_GROUP][2];
  pdl_trigger();
  pdl_wait();
  Kv8Unit u;
  if (!kv8_unit(g, u)) return;
  const int head0 = blockIdx.y * HEADS, nh = min(HEADS, g.heads - head0);
  // this lane's vectors: keys or values of one head, tokens t, t + STEP, ...
  constexpr int STEP = VPP / (2 * HEADS);
  static_assert(VPP % (2 * HEADS) == 0, "a thread's vectors are of one head and kind");
  const int sub = threadIdx.x % LPV, vec = threadIdx.x / LPV;
  const int h = vec % HEADS, kv = vec / HEADS & 1, t = vec / (2 * HEADS), pos = u.group * KV8_GROUP + t;
  const long long stride = kv ? vs : ks;
  const T* src = (kv ? v : k) + (u.q.row0 + pos - u.q.pos0) * stride + (head0 + h) * HD + sub * 8;
  Kv8Raw<T> raw[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {  // all loads first
    if (pos + i * STEP >= u.t0 && pos + i * STEP < u.t1 && h < nh)
      raw[i].load(src + i * STEP * stride);
    else
      raw[i].zero();
  }
  u.page = kv8_checked(g, u.page);
  if (u.page < 0) return;
  uint8_t* keys = g.codes + kv8_code_at(g, u.page, 0, head0 + h) + (size_t)(u.slot0 + t) * HD + sub * 8;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const uint32_t top = raw[i].template largest<LPV>();
    const bool nan = top >= 0x7F800000u;
    const int e2 = kv8_exponent(__uint_as_float(top));
    const float inv = kv8_pow2(-e2);
    float x[8];
    raw[i].floats(x);
    uint2 c = make_uint2(kv8_pack4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                         kv8_pack4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
    if (nan) c = make_uint2(0, 0);
    if (kv)
      *reinterpret_cast<uint2*>(&sV[h][t + i * STEP][sub * 8]) = c;
    else if (pos + i * STEP >= u.t0 && pos + i * STEP < u.t1 && h < nh)
      *reinterpret_cast<uint2*>(keys + i * STEP * HD) = c;
    if (sub == 0) sE[h][t + i * STEP][kv] = (uint8_t)(nan ? KV8_NAN : e2 + KV8_BIAS);
  }
  __syncthreads();
  const int lo = max(u.t0, 0) - u.group * KV8_GROUP, hi = u.t1 - u.group * KV8_GROUP;
  for (int i = threadIdx.x; i < nh * HD; i += KV8_THREADS) {
    const int h = i / HD, d = i % HD;
    uint8_t* dst = g.codes + kv8_code_at(g, u.page, 1, head0 + h) + ((size_t)(u.slot0 >> 4) * HD + d) * KV8_GROUP;
    if (hi - lo == KV8_GROUP) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = (uint32_t)sV[h][4 * j][d] | ((uint32_t)sV[h][4 * j + 1][d] << 8) |
               ((uint32_t)sV[h][4 * j + 2][d] << 16) | ((uint32_t)sV[h][4 * j + 3][d] << 24);
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int t = lo; t < hi; ++t) dst[t] = sV[h][t][d];
    }
  }
  const int eh = threadIdx.x / KV8_GROUP, et = threadIdx.x % KV8_GROUP;
  if (eh < nh && et >= lo && et < hi)
    *reinterpret_cast<uint16_t*>(g.exps + kv8_exp_at(g, u.page, head0 + eh, u.slot0 + et)) =
        (uint16_t)(sE[eh][et][0] | ((uint32_t)sE[eh][et][1] << 8));
}

// Read: the same, the other way.  The value plane is transposed through
// shared memory, so both outputs leave in rows.
template <typename T, int HD>
__global__ void __launch_bounds__(KV8_THREADS) kv8_read_kernel(Kv8Geom g, T* k, T* v) {
  constexpr int HEADS = KV8_READ_HEADS;
  constexpr int LPV = HD / 8;
  constexpr int VPP = KV8_THREADS / LPV;
  constexpr int PASSES = 2 * KV8_GROUP * HEADS / VPP;
  constexpr int VROWS = (HEADS * HD + KV8_THREADS - 1) / KV8_THREADS;  // rows of the value plane a thread brings
  __shared__ __align__(16) uint8_t sV[HEADS][KV8_GROUP][HD];
  pdl_trigger();
  pdl_wait();
  Kv8Unit u;
  if (!kv8_unit(g, u)) return;
  u.page = kv8_checked(g, u.page);
  const int head0 = blockIdx.y * HEADS, nh = min(HEADS, g.heads - head0);
  const int sub = threadIdx.x % LPV;
  uint2 kc[PASSES];
  uint4 vc[VROWS];
  int ex[PASSES];
#pragma unroll
  for (int i = 0; i < VROWS; ++i) {
    const int h = (threadIdx.x + i * KV8_THREADS) / HD, d = threadIdx.x % HD;
    vc[i] = make_uint4(0, 0, 0, 0);
    if (u.page >= 0 && h < nh)
      vc[i] = *reinterpret_cast<const uint4*>(g.codes + kv8_code_at(g, u.page, 1, head0 + h) +
                                              ((size_t)(u.slot0 >> 4) * HD + d) * KV8_GROUP);
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int vec = threadIdx.x / LPV + i * VPP, h = vec % HEADS, kv = (vec / HEADS) & 1,
              t = vec / (2 * HEADS);
    kc[i] = make_uint2(0, 0);
    ex[i] = 0;
    if (u.page >= 0 && h < nh) {
      if (!kv)
        kc[i] = *reinterpret_cast<const uint2*>(g.codes + kv8_code_at(g, u.page, 0, head0 + h) +
                                                (size_t)(u.slot0 + t) * HD + sub * 8);
      ex[i] = g.exps[kv8_exp_at(g, u.page, head0 + h, u.slot0 + t) + kv];
    }
  }
#pragma unroll
  for (int i = 0; i < VROWS; ++i) {
    const int h = (threadIdx.x + i * KV8_THREADS) / HD, d = threadIdx.x % HD;
    if (h >= HEADS) break;
    const uint32_t a[4] = {vc[i].x, vc[i].y, vc[i].z, vc[i].w};
#pragma unroll
    for (int t = 0; t < KV8_GROUP; ++t) sV[h][t][d] = (uint8_t)(a[t >> 2] >> (8 * (t & 3)));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int vec = threadIdx.x / LPV + i * VPP, h = vec % HEADS, kv = (vec / HEADS) & 1,
              t = vec / (2 * HEADS), pos = u.group * KV8_GROUP + t;
    if (pos < u.t0 || pos >= u.t1 || h >= nh) continue;
    float x[8];
    const uint2 c = kv ? *reinterpret_cast<const uint2*>(&sV[h][t][sub * 8]) : kc[i];
    const float sc = kv8_scale(ex[i]);
    const uint32_t two[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = kv8_value2(two[e]);
      x[2 * e] = u.page >= 0 ? f.x * sc : 0.f;
      x[2 * e + 1] = u.page >= 0 ? f.y * sc : 0.f;
    }
    kv8_store8((kv ? v : k) + ((size_t)(u.q.row0 + pos - u.q.pos0) * g.heads + head0 + h) * HD + sub * 8, x);
  }
}

template <typename T>
static cudaError_t launch_kv8_write(const Kv8Geom& g, const void* k, const void* v, long long ks, long long vs,
                                    cudaStream_t st) {
  return launch_k(g.hd == 128 ? kv8_write_kernel<T, 128> : kv8_write_kernel<T, 64>,
                  dim3(kv8_units(g.rows, g.nseq), (g.heads + KV8_WRITE_HEADS - 1) / KV8_WRITE_HEADS), dim3(KV8_THREADS), 0, st, g,
                  (const T*)k, (const T*)v, ks, vs);
}
template <typename T>
static cudaError_t launch_kv8_read(const Kv8Geom& g, void* k, void* v, cudaStream_t st) {
  return launch_k(g.hd == 128 ? kv8_read_kernel<T, 128> : kv8_read_kernel<T, 64>,
                  dim3(kv8_units(g.rows, g.nseq), (g.heads + KV8_READ_HEADS - 1) / KV8_READ_HEADS), dim3(KV8_THREADS), 0, st, g,
                  (T*)k, (T*)v);
}

}  // namespace dfk

using namespace dfk;

extern "C" {

df_status df_op_kv8_write(const void* k_dev, const void* v_dev, int32_t dtype, int32_t rows, int64_t k_stride,
                          int64_t v_stride, void* codes_dev, void* exps_dev, int32_t n_pages, int32_t page_tokens,
                          int32_t n_kv_heads, int32_t head_dim, const int32_t* page_table_dev, int32_t pt_stride,
                          const int32_t* row_start_dev, const int32_t* kv_len_dev, int32_t nseq, int32_t* err_dev,
                          void* stream) {
  Kv8Geom g{(uint8_t*)codes_dev, (uint8_t*)exps_dev, page_table_dev, row_start_dev, kv_len_dev, err_dev,
                  n_pages, page_tokens, n_kv_heads, head_dim, pt_stride, nseq, rows, 0};
  if ((dtype != DF_FP32 && dtype != DF_BF16) || rows < 0 || nseq < 0 || nseq > (1 << 20)) return DF_EINVAL;
  if (rows == 0 || nseq == 0) return DF_OK;
  if (!k_dev || !v_dev || !kv8_geom_ok(g) || !kv8_aligned(k_dev, 16) || !kv8_aligned(v_dev, 16)) return DF_EINVAL;
  const int per16 = dtype == DF_FP32 ? 4 : 8;  // elements in 16 bytes
  const long long width = (long long)n_kv_heads * head_dim;
  if (k_stride < width || v_stride < width || k_stride % per16 || v_stride % per16) return DF_EINVAL;
  g.per_page = kv8_per_page(page_tokens);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DF_FP32 ? launch_kv8_write<float>(g, k_dev, v_dev, k_stride, v_stride, st)
                                         : launch_kv8_write<__nv_bfloat16>(g, k_dev, v_dev, k_stride, v_stride, st);
  return e == cudaSuccess ? DF_OK : DF_ECUDA;
}

df_status df_op_kv8_read(const void* codes_dev, const void* exps_dev, int32_t n_pages, int32_t page_tokens,
                         int32_t n_kv_heads, int32_t head_dim, const int32_t* page_table_dev, int32_t pt_stride,
                         const int32_t* row_start_dev, const int32_t* kv_len_dev, int32_t nseq, int32_t rows,
                         int32_t dtype, void* k_dev, void* v_dev, int32_t* err_dev, void* stream) {
  Kv8Geom g{(uint8_t*)codes_dev, (uint8_t*)exps_dev, page_table_dev, row_start_dev, kv_len_dev, err_dev,
                  n_pages, page_tokens, n_kv_heads, head_dim, pt_stride, nseq, rows, 0};
  if ((dtype != DF_FP32 && dtype != DF_BF16) || rows < 0 || nseq < 0 || nseq > (1 << 20)) return DF_EINVAL;
  if (rows == 0 || nseq == 0) return DF_OK;
  if (!k_dev || !v_dev || !kv8_geom_ok(g) || !kv8_aligned(k_dev, 16) || !kv8_aligned(v_dev, 16)) return DF_EINVAL;
  g.per_page = kv8_per_page(page_tokens);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DF_FP32 ? launch_kv8_read<float>(g, k_dev, v_dev, st)
                                         : launch_kv8_read<__nv_bfloat16>(g, k_dev, v_dev, st);
  return e == cudaSuccess ? DF_OK : DF_ECUDA;
}

}  // extern "C"
