// Attention of a chunk of new tokens over the 8-bit paged cache, on the
// tensor cores (tcgen05 + TMEM + TMA), sm_103a.
//
// A tile is up to N (16, 32 or 64) query rows of one sequence and KV head:
// row r of the tile is query token r / G, head r % G of the group.  The keys
// come in chunks of 128 positions.  Per chunk
//   S^T [128 keys][N]   = K [128][hd] . Q^T            A = K,   B = Q
//   P^T                 = 2^(s c_t + e_t - M_r)
//   O^T [hd][N]        += V^T [hd][128] . P^T          A = V^T, B = P^T
// with keys (and head dims) on the tensor core's 128 lanes and query rows on
// its columns.  That way round a thread holds one key of S, so the key's and
// the value's power-of-two scale is one number per thread (c_t = 2^(b_k - 127)
// scale log2 e, and e_t = b_v - 127 added to the exponent), and both codes
// reach the tensor core as A operands through tensor memory: each thread
// widens its key's codes (its head dim's codes of 128 values: the cache keeps
// values transposed) to f16, exactly, and stores them to its own lane.  No
// widened tile passes through shared memory, and the cache's 8-bit bytes are
// all that is staged there.
//
// Softmax: M_r bounds (up to 2^8) the size s c_t + e_t of the terms that
// enter the product, so P fits f16 whatever the values' scales.  It moves
// only when a term passes it by more than 2^8 (then O is rescaled in tensor
// memory); a chunk in which no term does, which one vote over the 128 threads
// tells, needs no maximum over the keys.  P holds 2^6 for a term at M_r, so
// terms down to 2^-20 M_r keep f16's 11 bits.  The sum l_r adds the terms in
// fp32 with the values' scales taken out (2^-e_t).  A row's decisions depend
// on its own scores alone, and a chunk that it does not see adds exact zeros,
// so its bits do not depend on the other rows of its tile.
//
// The CTAs of a cluster take every C-th chunk of a tile and add their parts
// through distributed shared memory in rank order.
//
// Roles (160 threads): warps 0-3 widen, run the softmax and (thread 0) issue
// the tensor-core instructions; warp 4 stages keys, values and exponents by
// TMA in two stages each, and owns the tensor memory.  Two CTAs fit on an SM
// (256 columns and less than 113 KB each) and fill each other's waits.
//
// Every wait is bounded (about two seconds).  A thread whose wait ran out
// flags it and goes on without waiting, so all threads reach every barrier.
#include <cuda.h>
#include <math.h>

#include <atomic>

#include "kv8.cuh"

namespace dfk {

struct Kv8Attn {
  Kv8Geom g;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  long long qs, os;  // row strides (elements)
  int q_heads, group, max_rows, causal, window, tiles;
  float scale_log2;
};

constexpr int K8_CHUNK = 128;     // keys per chunk: one per tensor-memory lane
constexpr int K8_STAGES = 2;
constexpr int K8_THREADS = 160;
constexpr int K8_SMS = 152;
constexpr int K8_COLS = 256;      // tensor-memory columns of a CTA
constexpr float K8_SLACK = 8.f;   // how far (log2) a term may pass M before M moves
constexpr float K8_BIAS = 6.f;    // P = 2^K8_BIAS for a term at M
constexpr unsigned long long K8_WAIT_NS = 2000000000ull;

// Shared memory of a CTA (offsets from a 1024-byte boundary).
template <int HD, int N>
struct K8Smem {
  static constexpr int TILE = K8_CHUNK * HD;            // one stage of key (or value) codes
  static constexpr int K = 0;
  static constexpr int V = K + K8_STAGES * TILE;
  static constexpr int Q = V + K8_STAGES * TILE;        // [hd / 64][N rows][128 B] f16, 128-byte swizzle
  static constexpr int P = Q + (HD / 64) * N * 128;     // [128 keys][128 B], row r at f16 column r, 128-byte swizzle
  static constexpr int E = P + K8_CHUNK * 128;          // exponent bytes: [stage][128 keys][k|v]
  static constexpr int END = E + K8_STAGES * K8_CHUNK * 2;
  static constexpr int BYTES = END + 1024;
  // partial results for the merge, over the code stages: [N][HD] floats
  static constexpr int OLD = HD + 4;
  static_assert(N * OLD * 4 <= Q, "a tile's partial output fits over the stages");
  static_assert(2 * (BYTES + 4096) <= 227 * 1024, "two CTAs on an SM");
};

__device__ __forceinline__ uint32_t k8_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void k8_bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void k8_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void k8_arrive_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool k8_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool k8_wait_slow(uint32_t bar, uint32_t parity, int* err) {
  const unsigned long long t0 = device_ns();
  for (uint32_t it = 1; it < (1u << 30); ++it) {
    if (k8_test(bar, parity)) return true;
    if ((it & 1023u) == 0 && device_ns() - t0 > K8_WAIT_NS) break;
  }
  flag_error(err, ERR_TIMEOUT);
  return false;
}
// Bounded wait; once one has run out (`ok` false) the thread waits no more.
__device__ __forceinline__ void k8_wait(uint32_t bar, uint32_t parity, bool& ok, int* err) {
  if (ok && !k8_test(bar, parity)) ok = k8_wait_slow(bar, parity, err);
}
__device__ __forceinline__ void k8_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool k8_vote(bool any) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(any ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void k8_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void k8_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void k8_fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 key rows (16 x HD bytes) of slab (page, k, head) into swizzled rows.
__device__ __forceinline__ void k8_load_keys(uint32_t dst, const CUtensorMap* map, uint32_t bar, int slot, int slab) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(slot), "r"(slab)
      : "memory");
}
__device__ __forceinline__ void k8_load_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Shared-memory descriptor of a B operand in the 128-byte swizzle, 8-row
// groups 1024 bytes apart.  Q: K-major (rows = query rows).  P: MN-major
// (rows = keys, query rows along a 128-byte row).
__device__ __forceinline__ uint64_t k8_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor of kind::f16: f16 A and B, fp32 accumulator, 128 x N.
__host__ __device__ constexpr uint32_t k8_idesc(int n, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// D += A . B with A in tensor memory.
__device__ __forceinline__ void k8_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void k8_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 16 columns of the thread's tensor-memory lane.  The load's registers are
// valid once k8_ld_wait has passed them through.
__device__ __forceinline__ void k8_ld16(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void k8_ld_wait16(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
template <int N>
__device__ __forceinline__ void k8_ld(uint32_t addr, float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 16) k8_ld16(addr + i, v + i);
#pragma unroll
  for (int i = 0; i < N; i += 16) k8_ld_wait16(v + i);
}
__device__ __forceinline__ void k8_st16(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void k8_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t k8_pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void k8_unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t k8_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t k8_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t k8_mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float k8_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Largest value over the warp (numbers win over NaN).
__device__ __forceinline__ float k8_warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t k8_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t k8_cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t k8_remote(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float k8_remote_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 k8_remote_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void k8_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Widen 16 codes (one 16-byte piece) to 8 f16 pairs.
__device__ __forceinline__ void k8_widen16(uint4 w, uint32_t* r) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = kv8_widen2(a[i] & 0xFFFFu);
    r[2 * i + 1] = kv8_widen2(a[i] >> 16);
  }
}

template <int HD, int N>
__global__ void __launch_bounds__(K8_THREADS, 2)
    kv8_attention_kernel(const __grid_constant__ Kv8Attn a, const __grid_constant__ CUtensorMap kmap) {
  using L = K8Smem<HD, N>;
  constexpr int KCOLS = HD / 2;              // tensor-memory columns: widened keys,
  constexpr int VCOL = KCOLS;                // widened values (128 keys, two to a column),
  constexpr int SCOL = KCOLS + 64;           // S,
  constexpr int OCOL = SCOL + N;             // O
  static_assert(OCOL + N <= K8_COLS, "tensor-memory columns");
  extern __shared__ __align__(128) uint8_t k8_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(k8_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t s_fk[K8_STAGES], s_fv[K8_STAGES], s_ek[K8_STAGES], s_ev[K8_STAGES], s_s, s_o;
  __shared__ uint32_t s_tmem;
  __shared__ int s_live[K8_STAGES];                        // groups of the chunk that hold positions
  __shared__ __align__(16) float s_m[N], s_neg[N], s_fac[N], s_qf[N], s_l[N];
  __shared__ __align__(16) int s_lo[N], s_hi[N];
  __shared__ float s_red[4][N];

  const Kv8Geom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = (int)k8_cluster_size(), rank = (int)k8_rank();
  const int head = blockIdx.y, s = (int)(blockIdx.x / C) / a.tiles, tile = (int)(blockIdx.x / C) % a.tiles;
  const int G = a.group;

  // The tile's rows; every CTA of a cluster takes the same way out.
  Kv8Seq sq;
  const bool fine = kv8_seq(g, s, sq) && sq.n <= a.max_rows;
  if (!fine) {
    if (threadIdx.x == 0) flag_error(g.err, ERR_BOUNDS);
    return;
  }
  const int r0 = tile * N, nr = min(N, sq.n * G - r0);
  if (nr <= 0) return;
  const int len = sq.pos0 + sq.n;

  // ---- what each row sees, its query as f16, and the barriers
  for (int r = threadIdx.x; r < N; r += K8_THREADS) {
    int lo = 0x7fffffff, hi = -1;
    if (r < nr) {
      const int pos = sq.pos0 + (r0 + r) / G;
      lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      hi = pos < 0 ? -1 : a.causal ? pos : len - 1;
    }
    s_lo[r] = lo;
    s_hi[r] = hi;
    s_m[r] = -INFINITY;   // no term yet
    s_neg[r] = K8_BIAS;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < K8_STAGES; ++i) {
      k8_bar_init(k8_addr(&s_fk[i]), 1);
      k8_bar_init(k8_addr(&s_fv[i]), 1);
      k8_bar_init(k8_addr(&s_ek[i]), 4);
      k8_bar_init(k8_addr(&s_ev[i]), 4);
    }
    k8_bar_init(k8_addr(&s_s), 1);
    k8_bar_init(k8_addr(&s_o), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
  }
  if (warp == 4) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(k8_addr(&s_tmem)),
                 "n"(K8_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  k8_fence_before();
  __syncthreads();
  k8_fence_after();
  const uint32_t tmem = s_tmem;

  // Chunks of this CTA: chunk c of the sequence belongs to rank c % C.  The
  // rows are in position order, so the first and the last bound the tile.
  const int hi_last = s_hi[nr - 1], lo_first = s_lo[0];
  const int c_end = hi_last < 0 ? 0 : hi_last / K8_CHUNK + 1;
  int c_first = min(lo_first, len) / K8_CHUNK;
  c_first += (rank - c_first % C + C) % C;
  const int n_mine = c_end > c_first ? (c_end - c_first + C - 1) / C : 0;

  bool ok = true;
  if (warp == 4) {
    // ============================================================== producer
    // lanes 0-7 bring a chunk's groups of 16 keys with their exponents, lanes 8-15 its groups of values
    const int gr = lane & 7;
    for (int i = 0; i < n_mine; ++i) {
      const int st = i % K8_STAGES, c = c_first + i * C;
      const int pos = c * K8_CHUNK + gr * 16;
      int page = -1;
      if (lane < 16 && pos < len) {
        page = g.page_table[(size_t)s * g.pt_stride + pos / g.page_tokens];
        if (page < 0 || page >= g.n_pages) {
          page = -1;
          flag_error(g.err, ERR_BOUNDS);
        }
      }
      const uint32_t live = __ballot_sync(0xffffffffu, page >= 0) & 0xffu;
      if (i >= K8_STAGES) {
        k8_wait(k8_addr(&s_ek[st]), (uint32_t)(i / K8_STAGES - 1) & 1u, ok, g.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      const int slot = pos % g.page_tokens;
      if (lane == 0) {
        s_live[st] = (int)live;
        k8_arrive_tx(k8_addr(&s_fk[st]), __popc(live) * (16 * HD + 32));
      }
      __syncwarp();
      if (lane < 8 && page >= 0) {
        k8_load_keys(k8_addr(sm + L::K + st * L::TILE + gr * 16 * HD), &kmap, k8_addr(&s_fk[st]), slot,
                     (page * 2) * g.heads + head);
        k8_load_bytes(k8_addr(sm + L::E + st * K8_CHUNK * 2 + gr * 32), g.exps + kv8_exp_at(g, page, head, slot), 32,
                      k8_addr(&s_fk[st]));
      }
      if (i >= K8_STAGES) {
        k8_wait(k8_addr(&s_ev[st]), (uint32_t)(i / K8_STAGES - 1) & 1u, ok, g.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      if (lane == 0) k8_arrive_tx(k8_addr(&s_fv[st]), __popc(live) * 16 * HD);
      __syncwarp();
      if (lane >= 8 && page >= 0)
        k8_load_bytes(k8_addr(sm + L::V + st * L::TILE + gr * 16 * HD),
                      g.codes + kv8_code_at(g, page, 1, head) + (size_t)slot * HD, 16 * HD, k8_addr(&s_fv[st]));
    }
    // The consumers wait for every tile, so no copy is in flight when they are
    // done; if a wait ran out, give the copies issued the same time to land.
    if (!ok)
      for (int b = 0; b < K8_STAGES; ++b)
        for (uint32_t p = 0; p < 2; ++p) {
          (void)(k8_test(k8_addr(&s_fk[b]), p) || k8_wait_slow(k8_addr(&s_fk[b]), p, g.err));
          (void)(k8_test(k8_addr(&s_fv[b]), p) || k8_wait_slow(k8_addr(&s_fv[b]), p, g.err));
        }
    __syncwarp();
  } else {
    // ==================================== widening, softmax, tensor-core issue
    const int t = threadIdx.x;  // tensor-memory lane: the chunk's key t, and head dim t
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);

    // Q as f16: exact unless a row holds a magnitude of 2^15 or more, which
    // brings that row a power of two of its own (magnitudes below 2^-14 round
    // to multiples of 2^-24).
    constexpr int LPR = HD / 8;  // lanes per row, 8 elements each
    bool scaled = false;
    for (int r = t / LPR; r < N; r += 128 / LPR) {
      const int sub = t % LPR;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r < nr && s_hi[r] >= 0)
        w = *reinterpret_cast<const uint4*>(a.q + (long long)(sq.row0 + (r0 + r) / G) * a.qs +
                                            (size_t)(head * G + (r0 + r) % G) * HD + sub * 8);
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(ws[i] & 0x7FFFu, (ws[i] >> 16) & 0x7FFFu));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int over = min(max((int)(top >> 7) - 127 - 14, 0), 113);  // exponent above 2^14
      const float down = kv8_pow2(-over);
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 v = __floats2half2_rn(__uint_as_float(ws[i] << 16) * down,
                                            __uint_as_float(ws[i] & 0xFFFF0000u) * down);
        h[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(sm + L::Q + (sub >> 3) * N * 128 + r * 128 + (((sub & 7) ^ (r & 7)) << 4)) =
          make_uint4(h[0], h[1], h[2], h[3]);
      if (sub == 0) s_qf[r] = kv8_pow2(over);
      scaled = scaled || over > 0;
    }
    k8_fence_smem();
    const bool any_scaled = k8_vote(scaled);

    // rows that exist: positions every one of them sees
    const int full_lo = s_lo[nr - 1], full_hi = s_hi[0];
    float l[N];
#pragma unroll
    for (int r = 0; r < N; ++r) l[r] = 0.f;
    if (HD < 128 && t >= HD) {  // lanes past the head dims add zeros to rows of O nobody reads
      const uint32_t z[16] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) k8_st16(lane_base + VCOL + 16 * i, z);
    }

    const uint64_t qd = k8_desc(k8_addr(sm + L::Q)), pd = k8_desc(k8_addr(sm + L::P));
    float ct = 0.f, et = 0.f, ie = 1.f;
    int live = 0;
    bool pending = true;  // some row has no term yet

    // Chunk i's keys: exponents to registers, codes widened into this lane; then S^T = K Q^T.
    auto keys = [&](int i) {
      const int st = i % K8_STAGES;
      k8_wait(k8_addr(&s_fk[st]), (uint32_t)(i / K8_STAGES) & 1u, ok, g.err);
      live = s_live[st];
      const uint32_t ee = *reinterpret_cast<const uint16_t*>(sm + L::E + st * K8_CHUNK * 2 + t * 2);
      const uint8_t* row = sm + L::K + st * L::TILE + t * HD;
      uint32_t w[KCOLS];
#pragma unroll
      for (int p = 0; p < HD / 16; ++p) {
        const int at = HD == 128 ? (p ^ (t & 7)) : (p ^ ((t >> 1) & 3));
        k8_widen16(*reinterpret_cast<const uint4*>(row + at * 16), w + 8 * p);
      }
      __syncwarp();
      if (lane == 0) k8_arrive(k8_addr(&s_ek[st]));
#pragma unroll
      for (int p = 0; p < KCOLS / 16; ++p) k8_st16(lane_base + 16 * p, w + 16 * p);
      const bool here = (live >> (t >> 4)) & 1;
      const int bk = ee & 255, bv = ee >> 8;
      ct = here ? kv8_scale(bk) * a.scale_log2 : 0.f;
      et = !here ? 0.f : bv == KV8_NAN ? __uint_as_float(0x7FC00000u) : (float)(bv - KV8_BIAS);
      ie = !here || bv == KV8_NAN ? 1.f : __uint_as_float((uint32_t)(254 - bv) << 23);
      k8_st_wait();
      k8_fence_before();
      k8_sync();
      if (t == 0) {
        k8_fence_after();
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          k8_mma(tmem + SCOL, tmem + 8 * kk, qd + (uint64_t)(((kk >> 2) * N * 128 + (kk & 3) * 32) >> 4),
                 k8_idesc(N, false), kk > 0);
        k8_commit(k8_addr(&s_s));
      }
    };

    if (n_mine > 0) keys(0);
    for (int i = 0; i < n_mine; ++i) {
      const int st = i % K8_STAGES, key0 = (c_first + i * C) * K8_CHUNK;
      // ---- values (V^T and P are read by the last chunk's product until it is done)
      if (i > 0) k8_wait(k8_addr(&s_o), (uint32_t)(i - 1) & 1u, ok, g.err);
      k8_fence_after();
      k8_wait(k8_addr(&s_fv[st]), (uint32_t)(i / K8_STAGES) & 1u, ok, g.err);
      if (HD == 128 || t < HD) {
        const uint8_t* row = sm + L::V + st * L::TILE + t * 16;
        const bool tail = live != 0xff || key0 + K8_CHUNK > len;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t w[16];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int gr = 2 * h + u;
            uint4 v = *reinterpret_cast<const uint4*>(row + gr * 16 * HD);
            if (tail) {  // bytes behind the last position may be anything: zeros
              const int n = (live >> gr) & 1 ? len - key0 - gr * 16 : 0;
              v.x = n >= 4 ? v.x : n <= 0 ? 0u : v.x & ((1u << (8 * n)) - 1);
              v.y = n >= 8 ? v.y : n <= 4 ? 0u : v.y & ((1u << (8 * (n - 4))) - 1);
              v.z = n >= 12 ? v.z : n <= 8 ? 0u : v.z & ((1u << (8 * (n - 8))) - 1);
              v.w = n >= 16 ? v.w : n <= 12 ? 0u : v.w & ((1u << (8 * (n - 12))) - 1);
            }
            k8_widen16(v, w + 8 * u);
          }
          k8_st16(lane_base + VCOL + 16 * h, w);
        }
      }
      __syncwarp();
      if (lane == 0) k8_arrive(k8_addr(&s_ev[st]));

      // ---- softmax of key t's column of scores
      k8_wait(k8_addr(&s_s), (uint32_t)i & 1u, ok, g.err);
      k8_fence_after();
      const bool masked = live != 0xff || key0 < full_lo || key0 + K8_CHUNK - 1 > full_hi;
      const int pos = ((live >> (t >> 4)) & 1) && key0 + t < len ? key0 + t : -1;
      const uint64_t ct2 = k8_pair(ct, ct), et2 = k8_pair(et, et), ie2 = k8_pair(ie, ie);
      float y[N];
      auto scores = [&] {
        k8_ld<N>(lane_base + SCOL, y);
        if (any_scaled)
#pragma unroll
          for (int r = 0; r < N; ++r) y[r] *= s_qf[r];
#pragma unroll
        for (int r = 0; r < N; r += 4) {
          const float4 m = *reinterpret_cast<const float4*>(s_neg + r);
          k8_unpair(k8_fma2(k8_pair(y[r], y[r + 1]), ct2, k8_add2(et2, k8_pair(m.x, m.y))), y[r], y[r + 1]);
          k8_unpair(k8_fma2(k8_pair(y[r + 2], y[r + 3]), ct2, k8_add2(et2, k8_pair(m.z, m.w))), y[r + 2], y[r + 3]);
        }
        if (masked)
#pragma unroll
          for (int r = 0; r < N; r += 4) {
            const int4 lo = *reinterpret_cast<const int4*>(s_lo + r), hi = *reinterpret_cast<const int4*>(s_hi + r);
            y[r] = pos >= lo.x && pos <= hi.x ? y[r] : -INFINITY;
            y[r + 1] = pos >= lo.y && pos <= hi.y ? y[r + 1] : -INFINITY;
            y[r + 2] = pos >= lo.z && pos <= hi.z ? y[r + 2] : -INFINITY;
            y[r + 3] = pos >= lo.w && pos <= hi.w ? y[r + 3] : -INFINITY;
          }
      };
      scores();
      float top = y[0];
#pragma unroll
      for (int r = 1; r < N; ++r) top = fmaxf(top, y[r]);
      if (k8_vote(pending || top > K8_SLACK + K8_BIAS)) {
        // M of some row moves: the chunk's largest term of every row.  A row
        // without a term so far takes it as M, another only if it is past the slack.
#pragma unroll
        for (int r = 0; r < N; ++r) {
          const float w = k8_warp_max(y[r]);
          if (lane == (r & 31)) s_red[warp][r] = w;
        }
        k8_sync();
        bool wait = false;
        if (t < N) {
          const float ym = fmaxf(fmaxf(s_red[0][t], s_red[1][t]), fmaxf(s_red[2][t], s_red[3][t]));
          float fac = 1.f, m = s_m[t];
          if (m == -INFINITY) {
            if (ym > -INFINITY) m = ym - K8_BIAS;
          } else if (ym > K8_SLACK + K8_BIAS) {
            m += ym - K8_BIAS;
            fac = k8_ex2(s_m[t] - m);
          }
          if (m > -INFINITY) s_neg[t] = K8_BIAS - m;
          s_m[t] = m;
          s_fac[t] = fac;
          wait = t < nr && s_hi[t] >= 0 && m == -INFINITY;
        }
        pending = k8_vote(wait);
#pragma unroll
        for (int r = 0; r < N; ++r) l[r] *= s_fac[r];
        if (i > 0) {
#pragma unroll
          for (int cc = 0; cc < N; cc += 16) {
            float o[16];
            k8_ld<16>(lane_base + OCOL + cc, o);
            uint32_t w[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) w[r] = __float_as_uint(o[r] * s_fac[cc + r]);
            k8_st16(lane_base + OCOL + cc, w);
          }
        }
        scores();
      }
      uint8_t* prow = sm + L::P + t * 128;
#pragma unroll
      for (int r = 0; r < N; r += 8) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
          const float p0 = k8_ex2(y[r + u]), p1 = k8_ex2(y[r + u + 1]);
          k8_unpair(k8_fma2(k8_pair(p0, p1), ie2, k8_pair(l[r + u], l[r + u + 1])), l[r + u], l[r + u + 1]);
          const __half2 h = __floats2half2_rn(p0, p1);
          w[u / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(prow + (((r >> 3) ^ (t & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      k8_st_wait();
      k8_fence_smem();
      k8_fence_before();
      k8_sync();
      if (t == 0) {
        k8_fence_after();
#pragma unroll
        for (int kk = 0; kk < K8_CHUNK / 16; ++kk)
          k8_mma(tmem + OCOL, tmem + VCOL + 8 * kk, pd + (uint64_t)((kk * 2048) >> 4), k8_idesc(N, true),
                 i > 0 || kk > 0);
        k8_commit(k8_addr(&s_o));
      }
      if (i + 1 < n_mine) keys(i + 1);
    }
    if (n_mine > 0) k8_wait(k8_addr(&s_o), (uint32_t)(n_mine - 1) & 1u, ok, g.err);
    k8_fence_after();

    // ---- sums over the keys: halve the rows a lane carries, the same tree for every row
    {
      float v[N];
#pragma unroll
      for (int r = 0; r < N; ++r) v[r] = l[r];
      int base = 0;
#pragma unroll
      for (int o = 16, n = N; o > 0; o >>= 1) {
        if (n > 1) {
          n >>= 1;
          const bool up = (lane & o) != 0;
#pragma unroll
          for (int r = 0; r < N / 2; ++r)
            if (r < n) {
              const float send = up ? v[r] : v[r + n], keep = up ? v[r + n] : v[r];
              v[r] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
          base += up ? n : 0;
        } else {
          v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
      }
      constexpr int LEFT = N > 32 ? N / 32 : 1;
#pragma unroll
      for (int r = 0; r < LEFT; ++r) s_red[warp][base + r] = v[r];
    }
    k8_sync();
    if (t < N) s_l[t] = ((s_red[0][t] + s_red[1][t]) + s_red[2][t]) + s_red[3][t];
    k8_sync();

    if (C == 1) {
      // the whole of every row is here
      if (t < nr) s_fac[t] = s_l[t] == 0.f ? 0.f : 1.f / s_l[t];
      if (t < nr && a.lse)
        a.lse[(size_t)(sq.row0 + (r0 + t) / G) * a.q_heads + head * G + (r0 + t) % G] =
            s_l[t] == 0.f ? -INFINITY : (s_m[t] == -INFINITY ? s_l[t] : 0.6931471805599453f * (s_m[t] - K8_BIAS) + logf(s_l[t]));
      k8_sync();
#pragma unroll 1
      for (int cc = 0; cc < N && cc < nr; cc += 16) {
        float o[16];
        if (n_mine > 0) k8_ld<16>(lane_base + OCOL + cc, o);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int rr = cc + r;
          if (rr >= nr || t >= HD) continue;
          const float v = n_mine > 0 && s_l[rr] != 0.f ? o[r] * s_fac[rr] : 0.f;
          a.out[(long long)(sq.row0 + (r0 + rr) / G) * a.os + (size_t)(head * G + (r0 + rr) % G) * HD + t] =
              __float2bfloat16_rn(v);
        }
      }
    } else if (n_mine > 0) {
      float* part = reinterpret_cast<float*>(sm);
#pragma unroll 1
      for (int cc = 0; cc < N && cc < nr; cc += 16) {
        float o[16];
        k8_ld<16>(lane_base + OCOL + cc, o);
        if (t < HD)
#pragma unroll
          for (int r = 0; r < 16; ++r) part[(cc + r) * L::OLD + t] = o[r];
      }
    } else {
      if (t < N) s_l[t] = 0.f;
    }
  }
  k8_fence_before();
  __syncthreads();
  if (warp == 4) {
    k8_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(K8_COLS) : "memory");
  }
  if (C == 1) return;

  // ---- merge: rank q finishes rows q, q + C, ..., HD / 4 threads to a row
  k8_cluster_sync();
  constexpr int TPR = HD / 4, RPP = 128 / TPR;
  if (warp < 4) {
    const uint32_t part = k8_addr(sm), sl = k8_addr(s_l), smx = k8_addr(s_m);
    const int d = (threadIdx.x % TPR) * 4;
    for (int r = rank + C * (threadIdx.x / TPR); r < nr; r += C * RPP) {
      float M = -INFINITY;
      for (int q = 0; q < C; ++q) M = fmaxf(M, k8_remote_f(k8_remote(smx + r * 4, q)));
      float sum = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < C; ++q) {
        const float lq = k8_remote_f(k8_remote(sl + r * 4, q));
        if (lq == 0.f) continue;  // no key of this row there
        const float w = k8_ex2(k8_remote_f(k8_remote(smx + r * 4, q)) - M);
        const float4 x = k8_remote_f4(k8_remote(part + (r * L::OLD + d) * 4, q));
        sum = fmaf(lq, w, sum);
        o.x = fmaf(x.x, w, o.x);
        o.y = fmaf(x.y, w, o.y);
        o.z = fmaf(x.z, w, o.z);
        o.w = fmaf(x.w, w, o.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const long long row = sq.row0 + (r0 + r) / G;
      const int hq = head * G + (r0 + r) % G;
      const __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x * inv, o.y * inv),
                           b1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(a.out + row * a.os + (size_t)hq * HD + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
      if (d == 0 && a.lse)
        a.lse[(size_t)row * a.q_heads + hq] =
            sum == 0.f ? -INFINITY : (M == -INFINITY ? sum : 0.6931471805599453f * (M - K8_BIAS) + logf(sum));
    }
  }
  k8_cluster_sync();  // nobody leaves while another CTA may still read its part
}

// ------------------------------------------------------------------ launching
// TMA map of the cache's rows: HD bytes x page_tokens x (page, k|v, head),
// boxes of 16 rows, swizzled so that 32 threads reading the same 16-byte piece
// of 32 rows meet no bank conflict.
typedef CUresult (*PFN_k8Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static bool k8_tmap(CUtensorMap* map, const Kv8Geom& g) {
  static const PFN_k8Encode enc = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_k8Encode>(fn);
  }();
  if (!enc) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)g.hd, (cuuint64_t)g.page_tokens, (cuuint64_t)g.n_pages * 2 * g.heads};
  const cuuint64_t stride[2] = {(cuuint64_t)g.hd, (cuuint64_t)g.hd * g.page_tokens};
  const cuuint32_t box[3] = {(cuuint32_t)g.hd, 16, 1}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, g.codes, dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             g.hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, int N>
static cudaError_t k8_attrs() {
  cudaError_t e = cudaFuncSetAttribute(kv8_attention_kernel<HD, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       K8Smem<HD, N>::BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv8_attention_kernel<HD, N>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

template <int HD, int N>
static cudaError_t k8_launch(const Kv8Attn& a, const CUtensorMap& map, int cluster, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0};  // devices whose attributes are set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    if ((e = k8_attrs<HD, N>()) != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((long long)cluster * a.g.nseq * a.tiles), a.g.heads, 1);
  c.blockDim = dim3(K8_THREADS);
  c.dynamicSmemBytes = K8Smem<HD, N>::BYTES;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&c, kv8_attention_kernel<HD, N>, a, map);
}

}  // namespace dfk

using namespace dfk;

extern "C" {

df_status df_op_attention_kv8(const void* q_dev, int64_t q_stride, void* out_dev, int64_t out_stride, float* lse_dev,
                              int32_t rows, int32_t n_q_heads, const void* codes_dev, const void* exps_dev,
                              int32_t n_pages, int32_t page_tokens, int32_t n_kv_heads, int32_t head_dim,
                              const int32_t* page_table_dev, int32_t pt_stride, const int32_t* row_start_dev,
                              const int32_t* kv_len_dev, int32_t nseq, int32_t max_rows, int32_t max_len, float scale,
                              int32_t causal, int32_t window, int32_t cluster_ctas, int32_t* err_dev, void* stream) {
  Kv8Attn a{};
  a.g = Kv8Geom{(uint8_t*)codes_dev, (uint8_t*)exps_dev, page_table_dev, row_start_dev, kv_len_dev, err_dev,
                n_pages, page_tokens, n_kv_heads, head_dim, pt_stride, nseq, rows};
  if (rows < 0 || nseq < 0 || nseq > (1 << 20) || max_rows < 0 || max_len < 0 || (causal != 0 && causal != 1) ||
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
  a.group = n_q_heads / n_kv_heads;
  a.max_rows = max_rows < rows ? max_rows : rows;
  a.causal = causal;
  a.window = window;
  a.scale_log2 = (float)(scale * 1.4426950408889634);
  // the narrowest tile that holds a sequence's rows, or the widest
  const long long wanted = (long long)a.max_rows * a.group;
  const int n = wanted <= 16 ? 16 : wanted <= 32 ? 32 : 64;
  const long long tiles = (wanted + n - 1) / n;
  if (tiles * nseq > 0x7fffffff / 16) return DF_EINVAL;
  a.tiles = (int)tiles;
  // enough CTAs for two on every SM, but two chunks at least for each
  int cluster = cluster_ctas;
  if (!cluster) {
    const long long chunks = ((long long)max_len + K8_CHUNK - 1) / K8_CHUNK, work = tiles * nseq * n_kv_heads;
    cluster = 1;
    while (cluster < 16 && work * cluster < 2 * K8_SMS && chunks >= 4 * cluster) cluster *= 2;
  }
  CUtensorMap map;
  if (!k8_tmap(&map, a.g)) return DF_ECUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (head_dim == 128)
    e = n == 16 ? k8_launch<128, 16>(a, map, cluster, st)
                : n == 32 ? k8_launch<128, 32>(a, map, cluster, st) : k8_launch<128, 64>(a, map, cluster, st);
  else
    e = n == 16 ? k8_launch<64, 16>(a, map, cluster, st)
                : n == 32 ? k8_launch<64, 32>(a, map, cluster, st) : k8_launch<64, 64>(a, map, cluster, st);
  return e == cudaSuccess ? DF_OK : DF_ECUDA;
}

}  // extern "C"
