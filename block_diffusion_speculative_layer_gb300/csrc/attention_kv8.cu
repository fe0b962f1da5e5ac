// Attention of a chunk of new tokens over the 8-bit paged cache, on the
// tensor cores (tcgen05 + TMEM + TMA), sm_103a.
//
// A tile is up to N (16, 32, 64 or 128) query rows of one sequence and KV
// head: row r of the tile is query token r / G, head r % G of the group.  The keys
// come in chunks of 128 positions.  Per chunk
//   S^T [128 keys][N]  = K [128][hd] . (Qhi + Qlo)^T   A = K (e4m3, as cached)
//   P^T                = 2^(s c_t + e_t - M_r)
//   O^T [hd][N]       += V^T [hd][128] . P^T           A = V^T (f16), B = P^T (f16)
// with keys (and head dims) on the tensor core's 128 lanes and query rows on
// its columns.  That way round a thread holds one key of S, so the key's and
// the value's power-of-two scale is one number per thread (c_t = 2^(b_k - 127)
// scale log2 e, and e_t = b_v - 127 added to the exponent).
//
// Keys go from the cache's bytes to the tensor core without a conversion: a
// bf16 query has 8 bits, so 64 q is the sum of two e4m3 numbers of 4 bits each,
// exactly down to |q| = 2^-8 and to within 2^-16 below.  A row whose largest
// magnitude is outside [1/4, 7] is first brought to (3.5, 7] by a power of two
// f_r, and the scores of its tile are multiplied by f_r (5% of a long chunk's
// time, so not for every tile).  Both products go to one accumulator.
// Values need P at more than 8 bits and a wide range, so their product is f16:
// a thread widens its head dim's codes of 128 values (the cache keeps values
// transposed), exactly, and stores them to its own lane of tensor memory, the
// A operand.  No widened tile passes through shared memory.
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
// Roles: GROUPS groups of four warps widen values and run the softmax, each
// group on its N / GROUPS query rows (a thread's columns of S) and its share
// of the chunk's values; three warps stage keys, values and exponents by TMA;
// one issues the tensor-core instructions and owns the tensor memory.  S
// leaves tensor memory for registers at once, so the next chunk's S is
// computed while the softmax of this one runs.  Tiles of up to 64 rows run two
// CTAs to an SM (256 columns, less than 113 KB and 2 groups each), which fill
// each other's waits; tiles of 128 rows run one (512 columns, 4 groups) and
// widen a value and read an A operand for twice the rows.
//
// Every wait is bounded (about two seconds).  A thread whose wait ran out
// flags it and goes on without waiting, so all threads reach every barrier.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <iterator>

#include "kv8.cuh"

namespace dfk {

struct Kv8Attn {
  Kv8Geom g;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  long long qs, os;  // row strides (elements)
  int q_heads, group, max_rows, causal, window, tiles;
  unsigned solo;                // tiles that one CTA takes alone
  unsigned long long per_cluster;  // 2^32 / (CTAs of a cluster), rounded up
  float scale_log2;
};

constexpr int K8_CHUNK = 128;     // keys per chunk: one per tensor-memory lane
constexpr int K8_SMS = 152;
constexpr float K8_SLACK = 8.f;   // how far (log2) a term may pass M before M moves
constexpr float K8_BIAS = 6.f;    // P = 2^K8_BIAS for a term at M
constexpr float K8_QSCALE = 64.f; // queries are staged times this (7 * 64 = 448, the largest e4m3 number)
constexpr unsigned long long K8_WAIT_NS = 2000000000ull;

// Shapes and shared memory of a CTA (offsets from a 1024-byte boundary).
template <int HD, int N>
struct K8 {
  static constexpr int GROUPS = N == 128 ? 4 : 2;
  static constexpr int W = N / GROUPS;                  // query rows (columns of S) of a thread
  static constexpr int CTHREADS = 128 * GROUPS;         // threads that widen and run the softmax
  static constexpr int THREADS = CTHREADS + 128;        // and four warps that stage and issue
  static constexpr int PER_SM = N == 128 ? 1 : 2;       // CTAs on an SM
  // Registers of a thread: the kernel's at launch, then those of the softmax
  // and of the staging warps (their sum stays within the launch's)
  static constexpr int REGS = 65536 / PER_SM / THREADS / 16 * 16, CREGS = N == 128 ? 104 : 96, AREGS = N == 128 ? 64 : 48;
  static_assert(CTHREADS * CREGS + 128 * AREGS <= THREADS * REGS, "registers of the launch");
  static constexpr int COLS = 512 / PER_SM;             // tensor-memory columns of a CTA:
  static constexpr int VCOL = 0;                        // widened values of an even and an odd chunk (two to a column),
  static constexpr int SCOL = 128;                      // S,
  static constexpr int OCOL = SCOL + N;                 // O
  static_assert(OCOL + N <= COLS, "tensor-memory columns");
  static constexpr int STAGES = 2 * (3 - PER_SM);
  static constexpr int TILE = K8_CHUNK * HD;            // one stage of key (or value) codes
  static constexpr int KOFF = 0;
  static constexpr int VOFF = KOFF + STAGES * TILE;
  static constexpr int QOFF = VOFF + STAGES * TILE;     // [hi, lo][N rows][HD] e4m3, swizzled as the keys
  static constexpr int POFF = QOFF + 2 * N * HD;        // [N / 64][128 keys][128 B] f16, row r at column r, 128-byte swizzle
  static constexpr int EOFF = POFF + (N + 63) / 64 * K8_CHUNK * 128;  // exponent bytes: [stage][128 keys][k|v]
  static constexpr int BOFF = EOFF + STAGES * K8_CHUNK * 2;             // barriers (offsets from BOFF):
  static constexpr int FK = 0, FV = FK + 8 * STAGES;    // a stage's keys, values and exponents have landed,
  static constexpr int EK = FV + 8 * STAGES, EV = EK + 8 * STAGES;      // are read,
  static constexpr int SS = EV + 8 * STAGES;            // S computed,
  static constexpr int SR = SS + 8;                     // S read, one arrival per softmax warp,
  static constexpr int PW = SR + 8;                     // V^T and P written,
  static constexpr int OU = PW + 8;                     // O updated
  static constexpr int BYTES = BOFF + 256 + 1024;
  static constexpr int OLD = HD + 4;                    // the merge's partial output, over the code stages: [N][OLD] floats
  static_assert(N * OLD * 4 <= QOFF, "a tile's partial output fits over the stages");
  static_assert(PER_SM * (BYTES + 1024 + 128 * N + 1024) <= 228 * 1024, "CTAs on an SM");
};

__device__ __forceinline__ uint32_t k8_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void k8_bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// One arrival for the warp, after what its lanes did before.
__device__ __forceinline__ void k8_arrive_warp(uint32_t bar) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void k8_arrive_tx(uint32_t one, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar),
      "r"(bytes), "r"(one)
      : "memory");
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
// (Inline: the register split does not allow calls.)
__device__ __forceinline__ bool k8_wait_slow(uint32_t bar, uint32_t parity, bool ok, int* err) {
  if (!ok) return false;
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
  if (!k8_test(bar, parity)) ok = k8_wait_slow(bar, parity, ok, err);
}
// Barriers of a group of four warps (ids 1..8), and of all that widen (9).
__device__ __forceinline__ void k8_group_sync(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}
template <int THREADS>
__device__ __forceinline__ void k8_all_sync() {
  asm volatile("bar.sync 9, %0;" ::"n"(THREADS) : "memory");
}
__device__ __forceinline__ bool k8_vote(int group, bool any) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(any ? 1u : 0u), "r"(5 + group)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void k8_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void k8_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void k8_fence_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint4 k8_lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t k8_lds2(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void k8_sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void k8_sts8(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// One lane of the converged warp.  The instructions below that one thread
// issues are executed by the whole warp and predicated on it, so that their
// operands stay in uniform registers (under a divergent branch each of them
// costs its issuing thread about 80 cycles of register moves).
__device__ __forceinline__ uint32_t k8_elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r));
  return r;
}

// 16 key rows (16 x HD bytes) of slab (page, k, head) into swizzled rows.
__device__ __forceinline__ void k8_load_keys(uint32_t dst, const CUtensorMap* map, uint32_t bar, int slot, int slab) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "@p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(slot), "r"(slab)
      : "memory");
}
__device__ __forceinline__ void k8_load_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n}\n" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Shared-memory descriptors.  Rows of 128 bytes in the 128-byte swizzle (8-row
// groups 1024 bytes apart) or of 64 bytes in the 64-byte swizzle (512 bytes
// apart).  K and Q: K-major.  P: MN-major (rows = keys, 64 query rows along a row;
// `block` bytes between such column blocks).
template <int ROW>
__device__ __forceinline__ uint64_t k8_desc(uint32_t addr, uint32_t block = 16) {
  static_assert(ROW == 128 || ROW == 64, "row bytes");
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)((8 * ROW) >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)(ROW == 128 ? 2 : 4) << 61);
}
// Instruction descriptor: A and B f16 (kind::f16) or e4m3 (kind::f8f6f4), fp32 accumulator, 128 x N.
__host__ __device__ constexpr uint32_t k8_idesc(int n, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// D = (acc) D + A . B, e4m3, both in shared memory.
__device__ __forceinline__ void k8_mma_codes(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one)
      : "memory");
}
// D = (acc) D + A . B, f16, A in tensor memory.
__device__ __forceinline__ void k8_mma(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one)
      : "memory");
}
__device__ __forceinline__ void k8_commit(uint32_t one, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(one)
      : "memory");
}

// W columns (8, 16 or 32) of the thread's tensor-memory lane.
template <int W>
__device__ __forceinline__ void k8_ld(uint32_t addr, float* v) {
  if constexpr (W == 8)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
        : "r"(addr)
        : "memory");
  else if constexpr (W == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void k8_st8(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
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
__device__ __forceinline__ float k8_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// W values per lane, each reduced over the warp in the tree xor 16, 8, 4, 2,
// 1: as long as a lane holds several, it keeps half of them at each step.  The
// lane's result is v[0], of value number `base`.
template <int W, typename Op>
__device__ __forceinline__ int k8_reduce(float* v, Op op) {
  const int lane = threadIdx.x & 31;
  int base = 0;
#pragma unroll
  for (int o = 16, n = W; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int r = 0; r < W / 2; ++r)
        if (r < n) {
          const float send = up ? v[r] : v[r + n], keep = up ? v[r + n] : v[r];
          v[r] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
      base += up ? n : 0;
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return base;
}

template <int HD, int N>
__global__ void __launch_bounds__(K8<HD, N>::THREADS, K8<HD, N>::PER_SM)
    kv8_attention_kernel(const __grid_constant__ Kv8Attn a, const __grid_constant__ CUtensorMap kmap) {
  using L = K8<HD, N>;
  constexpr int W = L::W, STAGES = L::STAGES, CT = L::CTHREADS;
  extern __shared__ __align__(128) uint8_t k8_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(k8_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smb = k8_addr(sm), bars = smb + L::BOFF;
  __shared__ uint32_t s_tmem;
  __shared__ int s_scaled;                                 // some row was brought into range
  __shared__ int s_live[STAGES];                           // groups of the chunk that hold positions
  __shared__ __align__(16) float s_m[N], s_neg[N], s_del[N], s_fac[N], s_qf[N], s_l[N];
  __shared__ __align__(16) int s_lo[N], s_hi[N];           // positions a row sees
  __shared__ int s_tok[N], s_hd[N];                        // a row's token and query head
  __shared__ float s_red[4][N];

  const Kv8Geom& g = a.g;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int ISSUER = CT / 32, KEYS = ISSUER + 1, VALUES = ISSUER + 2;  // and the exponents' warp

  // The first `solo` CTAs take a tile each, the clusters behind them share one.
  // Of a causal sequence's tiles the last, which sees the most, starts first.
  const bool alone = blockIdx.x < a.solo;
  const int C = alone ? 1 : (int)k8_cluster_size(), rank = alone ? 0 : (int)k8_rank();
  auto over_c = [&](unsigned x) { return alone ? x : (unsigned)(((unsigned long long)x * a.per_cluster) >> 32); };
  const unsigned unit = alone ? blockIdx.x : a.solo + over_c(blockIdx.x - a.solo);
  const int head = (int)(unit / (unsigned)(a.tiles * g.nseq)), in_head = (int)unit - head * a.tiles * g.nseq;
  const int s = in_head / a.tiles, nth = in_head - s * a.tiles;
  const int tile = a.causal && a.window == 0 ? a.tiles - 1 - nth : nth;
  const int G = a.group;

  // Barriers and tensor memory first: an earlier kernel may still run, and
  // nothing that it writes is read before the wait.
  pdl_trigger();
  if (warp == ISSUER) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(k8_addr(&s_tmem)),
                 "n"(L::COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    k8_fence_before();
  }
  if (warp == KEYS && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    s_scaled = 0;
    for (int i = 0; i < STAGES; ++i) {
      k8_bar_init(bars + L::FK + i * 8, 1);
      k8_bar_init(bars + L::FV + i * 8, 2);
      k8_bar_init(bars + L::EK + i * 8, 1);
      k8_bar_init(bars + L::EV + i * 8, CT / 32);
    }
    k8_bar_init(bars + L::SS, 1);        // S computed
    k8_bar_init(bars + L::SR, CT / 32);  // S read, one arrival per softmax warp
    k8_bar_init(bars + L::PW, CT / 32);  // V^T and P written
    k8_bar_init(bars + L::OU, 1);        // O updated
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();

  // Pages of the first stages, looked up while the sequence's entries are on
  // their way: without a window chunk c of rank r starts at r + c C whatever
  // the lengths are.
  int early[STAGES];
#pragma unroll
  for (int i = 0; i < STAGES; ++i) {
    early[i] = -1;
    if (warp > ISSUER && lane < 8 && a.window == 0) {
      const int entry = kv8_entry(g, (rank + i * C) * (K8_CHUNK / 16) + lane);
      if (entry < g.pt_stride) early[i] = g.page_table[(size_t)s * g.pt_stride + entry];
    }
  }


  // The tile's rows; every CTA of a cluster takes the same way out.
  Kv8Seq sq;
  const bool fine = kv8_seq(g, s, sq) && sq.n <= a.max_rows;
  const int r0 = tile * N, nr = fine ? min(N, sq.n * G - r0) : 0;
  if (nr <= 0) {
    if (!fine && threadIdx.x == 0) flag_error(g.err, ERR_BOUNDS);
    __syncthreads();
    k8_fence_after();
    if (warp == ISSUER)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "n"(L::COLS) : "memory");
    return;
  }
  const int len = sq.pos0 + sq.n;

  // Positions the rows see: they are in position order, so the first and the
  // last row bound the tile, and what both see all see.  Chunk c of the
  // sequence belongs to rank c % C.
  auto lowest = [&](int pos) { return a.window > 0 ? max(0, pos - a.window + 1) : 0; };
  auto highest = [&](int pos) { return pos < 0 ? -1 : a.causal ? pos : len - 1; };
  // row r of the tile: head (g0 + r) % G of the group, of token j0 + (g0 + r) / G
  // (the quotient of small numbers by a reciprocal: off by less than half a step)
  const int j0 = r0 / G, g0 = r0 - j0 * G;
  const float inv_g = 1.f / (float)G;
  auto token = [&](int r) { return j0 + (int)(((float)(g0 + r) + 0.5f) * inv_g); };
  const int pos_first = sq.pos0 + j0, pos_last = sq.pos0 + token(nr - 1);
  const int full_lo = lowest(pos_last), full_hi = highest(pos_first), end = highest(pos_last) + 1;
  const int c_end = (end + K8_CHUNK - 1) / K8_CHUNK;
  // positions [begin, end) are what the tile sees: pages of others are not
  // looked at (a window may have left them), bytes of others count as zeros
  const int begin = min(lowest(pos_first), len);
  int c_first = begin / K8_CHUNK;
  const int from = c_first - (int)over_c(c_first) * C;  // the first chunk's rank
  c_first += rank - from + (rank < from ? C : 0);
  const unsigned n_mine = c_end > c_first ? over_c(c_end - c_first + C - 1) : 0;

  bool ok = true;
  // Staging: a chunk's 8 groups of 16 keys, of values and of exponents are 24
  // copies, each of which costs the warp that issues it about 100 cycles, so
  // three warps share them.  Pages are looked up a chunk ahead, in lanes 0-7.
  struct Place {
    int page, slot;  // page -2: no such group
  };
  auto place = [&](unsigned i, int known = 0x7fffffff) {
    Place p{-2, 0};
    if (i < n_mine && lane < 8) {
      const unsigned group = (unsigned)(c_first + (int)i * C) * (K8_CHUNK / 16) + lane;
      const int entry = kv8_entry(g, (int)group);
      p.slot = (int)(group * 16 - entry * g.page_tokens);
      if ((int)group * 16 < end && (int)group * 16 + 16 > begin)
        p.page = known != 0x7fffffff ? known : g.page_table[(size_t)s * g.pt_stride + entry];
    }
    return p;
  };
  // (apart from the look-up, which would otherwise be waited for at once)
  auto checked = [&](Place p) {
    if (p.page != -2 && (p.page < 0 || p.page >= g.n_pages)) {
      p.page = -2;
      flag_error(g.err, ERR_BOUNDS);
    }
    return p;
  };
  // Everything a copy needs is in registers before the wait for its stage: the
  // copies then follow one another without waiting for a shuffle or a product.
  auto produce = [&](unsigned i, Place p, uint32_t one) {
    const int st = i % STAGES;
    const uint32_t live = __ballot_sync(0xffffffffu, p.page >= 0);
    if (warp == KEYS) {
      int slab[8], slot[8];
#pragma unroll
      for (int gr = 0; gr < 8; ++gr) {
        slab[gr] = __shfl_sync(0xffffffffu, p.page * 2 * g.heads + head, gr);
        slot[gr] = __shfl_sync(0xffffffffu, p.slot, gr);
      }
      if (i >= STAGES) k8_wait(bars + L::EK + st * 8, (i / STAGES - 1) & 1u, ok, g.err);
      if (!__all_sync(0xffffffffu, ok)) return;
      k8_arrive_tx(one, bars + L::FK + st * 8, __popc(live) * 16 * HD);
#pragma unroll
      for (int gr = 0; gr < 8; ++gr)
        if (live >> gr & 1)
          k8_load_keys(smb + (L::KOFF + st * L::TILE + gr * 16 * HD), &kmap, bars + L::FK + st * 8, slot[gr], slab[gr]);
    } else {
      // values are the second plane of a page; exponents of both kinds lie together
      const bool values = warp == VALUES;
      const unsigned long long at =
          ((unsigned long long)(values ? p.page * 2 + 1 : p.page) * g.heads + head) * g.page_tokens + p.slot;
      const unsigned long long lane_src =
          values ? (unsigned long long)g.codes + at * HD : (unsigned long long)g.exps + at * 2;
      const uint32_t bytes = values ? 16 * HD : 32;
      const uint32_t dst = smb + (values ? L::VOFF + st * L::TILE : L::EOFF + st * K8_CHUNK * 2);
      unsigned long long src[8];
#pragma unroll
      for (int gr = 0; gr < 8; ++gr) src[gr] = __shfl_sync(0xffffffffu, lane_src, gr);
      if (i >= STAGES) k8_wait(bars + L::EV + st * 8, (i / STAGES - 1) & 1u, ok, g.err);
      if (!__all_sync(0xffffffffu, ok)) return;
      if (values && lane == 0) s_live[st] = (int)live;
      __syncwarp();
      k8_arrive_tx(one, bars + L::FV + st * 8, __popc(live) * bytes);
#pragma unroll
      for (int gr = 0; gr < 8; ++gr)
        if (live >> gr & 1) k8_load_bytes(dst + gr * bytes, (const void*)src[gr], bytes, bars + L::FV + st * 8);
    }
  };

  // Q: LPR lanes to a row, 8 elements each; the loads start here.
  constexpr int LPR = HD / 8, RPP = CT / LPR, QPASS = (N + RPP - 1) / RPP;
  const int sub = threadIdx.x % LPR;
  uint4 qw[QPASS];

  if (warp > ISSUER) {
    // (nothing that the others wait for, but that they are here)
    asm volatile("bar.arrive 12, %0;" ::"n"(L::THREADS) : "memory");
  } else if (warp < ISSUER) {
#pragma unroll
    for (int i = 0; i < QPASS; ++i) {
      const int r = threadIdx.x / LPR + i * RPP;
      qw[i] = make_uint4(0, 0, 0, 0);
      if (r < nr) {
        const int j = token(r), h = head * G + (r0 + r) - j * G;
        if (sq.pos0 + j >= 0)
          qw[i] = *reinterpret_cast<const uint4*>(a.q + (sq.row0 + j) * a.qs + (size_t)h * HD + sub * 8);
        if (sub == 0) {
          s_tok[r] = sq.row0 + j;
          s_hd[r] = h;
          s_lo[r] = lowest(sq.pos0 + j);
          s_hi[r] = highest(sq.pos0 + j);
        }
      } else if (r < N && sub == 0) {
        s_lo[r] = 0x7fffffff;
        s_hi[r] = -1;
      }
      if (r < N && sub == 0) {
        s_m[r] = -INFINITY;  // no term yet
        s_neg[r] = K8_BIAS;
      }
    }
  }
  if (warp <= ISSUER) asm volatile("bar.sync 12, %0;" ::"n"(L::THREADS) : "memory");
  k8_fence_after();
  const uint32_t tmem = warp <= ISSUER ? __shfl_sync(0xffffffffu, s_tmem, 0) : 0;
  if (warp >= ISSUER)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::AREGS));
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::CREGS));

  if (warp > ISSUER) {
    const uint32_t one = k8_elect();
    asm volatile("bar.sync 11, 96;" ::: "memory");  // the barriers are initialised
#pragma unroll
    for (unsigned i = 0; i < STAGES; ++i)
      if (i < n_mine) produce(i, checked(a.window == 0 ? place(i, early[i]) : place(i)), one);
    Place next = place(STAGES);
    for (unsigned i = STAGES; i < n_mine; ++i) {
      const Place p = checked(next);
      next = place(i + 1);
      produce(i, p, one);
    }
    // The other warps wait for every tile, so no copy is in flight when they
    // are done; if a wait ran out, give the copies issued the same time to land.
    if (!__all_sync(0xffffffffu, ok))
      for (int b = 0; b < STAGES; ++b)
        for (uint32_t q = 0; q < 2; ++q) {
          (void)(k8_test(bars + L::FK + b * 8, q) || k8_wait_slow(bars + L::FK + b * 8, q, true, g.err));
          (void)(k8_test(bars + L::FV + b * 8, q) || k8_wait_slow(bars + L::FV + b * 8, q, true, g.err));
        }
    __syncwarp();
  } else if (warp == ISSUER) {
    const uint32_t one = k8_elect();
    asm volatile("bar.sync 10, %0;" ::"n"(CT + 32) : "memory");  // Q is in shared memory
    if (n_mine > 0) {
      const uint64_t kd = k8_desc<HD>(smb + (L::KOFF)), qd = k8_desc<HD>(smb + (L::QOFF)),
                     pd = k8_desc<128>(smb + (L::POFF), K8_CHUNK * 128);
      // S^T of chunk i; its key tile is free when that is done
      auto scores = [&](unsigned i) {
        const int st = i % STAGES;
        k8_wait(bars + L::FK + st * 8, (i / STAGES) & 1u, ok, g.err);
        k8_fence_after();
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)  // the queries' high halves, then the low ones
          k8_mma_codes(one, tmem + L::SCOL, kd + (uint64_t)((st * L::TILE + kk % (HD / 32) * 32) >> 4),
                       qd + (uint64_t)((kk / (HD / 32) * N * HD + kk % (HD / 32) * 32) >> 4), k8_idesc(N, false),
                       kk > 0);
        k8_commit(one, bars + L::SS);
        k8_commit(one, bars + L::EK + st * 8);
      };
      scores(0);
      for (unsigned i = 0; i < n_mine; ++i) {
        if (i + 1 < n_mine) {
          k8_wait(bars + L::SR, i & 1u, ok, g.err);
          scores(i + 1);
        }
        k8_wait(bars + L::PW, i & 1u, ok, g.err);
        k8_fence_after();
#pragma unroll
        for (int kk = 0; kk < K8_CHUNK / 16; ++kk)
          k8_mma(one, tmem + L::OCOL, tmem + L::VCOL + (i & 1) * 64 + 8 * kk, pd + (uint64_t)((kk * 2048) >> 4),
                 k8_idesc(N, true), i > 0 || kk > 0);
        k8_commit(one, bars + L::OU);
      }
      // every product has finished before tensor memory is freed
      bool done = true;
      k8_wait(bars + L::OU, (n_mine - 1) & 1u, done, g.err);
    }
    __syncwarp();
  } else {
    const int t = threadIdx.x & 127, group = threadIdx.x >> 7;  // t: tensor-memory lane = the chunk's key, and head dim
    const int w0 = group * W;                                   // the thread's first column
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);

    // Q as two e4m3 numbers
#pragma unroll
    for (int i = 0; i < QPASS; ++i) {
      const int r = threadIdx.x / LPR + i * RPP;
      const uint32_t ws[4] = {qw[i].x, qw[i].y, qw[i].z, qw[i].w};
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) top = max(top, max(ws[u] & 0x7FFFu, (ws[u] >> 16) & 0x7FFFu));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      // the power of two taken out of the row (a row that holds no numbers becomes NaN)
      const int e = (int)(top >> 7) - 127;
      const bool fits = top == 0 || (top >= 0x3E80u && top <= 0x40E0u);  // bf16 bits of 1/4 and 7
      const int out = fits ? 0 : min(max(e - 2 + ((top & 0x7Fu) > 0x60u ? 1 : 0), -113), 120);
      const float by = top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : K8_QSCALE * kv8_pow2(-out);
      float x[8], hi[8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[2 * u] = __uint_as_float(ws[u] << 16) * by;
        x[2 * u + 1] = __uint_as_float(ws[u] & 0xFFFF0000u) * by;
      }
      const uint2 ch = make_uint2(kv8_pack4(x[0], x[1], x[2], x[3]), kv8_pack4(x[4], x[5], x[6], x[7]));
      const uint32_t two[4] = {ch.x & 0xFFFFu, ch.x >> 16, ch.y & 0xFFFFu, ch.y >> 16};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f = kv8_value2(two[u]);
        hi[2 * u] = f.x;
        hi[2 * u + 1] = f.y;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] -= hi[u];
      const uint2 cl = make_uint2(kv8_pack4(x[0], x[1], x[2], x[3]), kv8_pack4(x[4], x[5], x[6], x[7]));
      if (r < N) {
        const int piece = sub >> 1, at = HD == 128 ? (piece ^ (r & 7)) : (piece ^ ((r >> 1) & 3));
        const uint32_t dst = smb + L::QOFF + r * HD + at * 16 + (sub & 1) * 8;
        k8_sts8(dst, ch);
        k8_sts8(dst + N * HD, cl);
        if (sub == 0) s_qf[r] = kv8_pow2(out);
        if (out != 0) s_scaled = 1;
      }
    }
    k8_fence_smem();
    asm volatile("bar.arrive 10, %0;" ::"n"(CT + 32) : "memory");
    k8_all_sync<CT>();  // s_qf, s_scaled
    const bool any_scaled = s_scaled != 0;

    float l[W];
#pragma unroll
    for (int r = 0; r < W; ++r) l[r] = 0.f;
    constexpr int VSHARE = 8 / L::GROUPS;  // groups of 16 values this thread widens
    const int v0 = group * VSHARE;
    if (HD < 128 && t >= HD) {  // lanes past the head dims add zeros to rows of O nobody reads
      const uint32_t z[8] = {};
#pragma unroll
      for (int i = 0; i < 2 * VSHARE; ++i)
        k8_st8(lane_base + L::VCOL + (i / VSHARE) * 64 + (v0 + i % VSHARE) * 8, z);
    }
    bool pending = true;  // some row has no term yet
    // this key's 16-byte piece of P for column w0 (w0 is a multiple of W, so piece p of the thread is at prow ^ 16 p)
    const uint32_t prow = smb + L::POFF + (w0 >> 6) * K8_CHUNK * 128 + t * 128 + ((((w0 & 63) >> 3) ^ (t & 7)) << 4);

    for (unsigned i = 0; i < n_mine; ++i) {
      const int st = i % STAGES, key0 = (c_first + (int)i * C) * K8_CHUNK;
      // ---- this key's scales
      k8_wait(bars + L::FV + st * 8, (i / STAGES) & 1u, ok, g.err);
      const int live = s_live[st];
      const uint32_t ee = k8_lds2(smb + L::EOFF + st * K8_CHUNK * 2 + t * 2);
      const bool here = (live >> (t >> 4)) & 1;
      const int bk = ee & 255, bv = ee >> 8;
      const float ct = here ? kv8_scale(bk) * a.scale_log2 : 0.f;
      const float et = !here ? 0.f : bv == KV8_NAN ? __uint_as_float(0x7FC00000u) : (float)(bv - KV8_BIAS);
      const float ie = !here || bv == KV8_NAN ? 1.f : __uint_as_float((uint32_t)(254 - bv) << 23);
      const uint64_t ct2 = k8_pair(ct, ct), et2 = k8_pair(et, et), ie2 = k8_pair(ie, ie);
      const bool masked = live != 0xff || key0 < full_lo || key0 + K8_CHUNK - 1 > full_hi;
      const int pos = here && key0 + t < len ? key0 + t : -1;

      // ---- values (the product of two chunks ago has read this buffer: O's wait below)
      if (HD == 128 || t < HD) {
        const uint32_t row = smb + L::VOFF + st * L::TILE + v0 * 16 * HD + t * 16;
        uint4 v[VSHARE];
#pragma unroll
        for (int q = 0; q < VSHARE; ++q) v[q] = k8_lds16(row + q * 16 * HD);
        if (live != 0xff || key0 < begin || key0 + K8_CHUNK > end) {  // bytes outside may be anything: zeros
#pragma unroll
          for (int q = 0; q < VSHARE; ++q) {
            const int gr = v0 + q, n = (live >> gr) & 1 ? end - key0 - gr * 16 : 0, m = begin - key0 - gr * 16;
            auto first = [](int k) { return k >= 4 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << (8 * k)) - 1; };  // k bytes
            v[q].x &= first(n) & ~first(m);
            v[q].y &= first(n - 4) & ~first(m - 4);
            v[q].z &= first(n - 8) & ~first(m - 8);
            v[q].w &= first(n - 12) & ~first(m - 12);
          }
        }
#pragma unroll
        for (int q = 0; q < VSHARE; q += 2) {
          uint32_t w[16];
          k8_widen16(v[q], w);
          k8_widen16(v[q + 1], w + 8);
          k8_st16(lane_base + L::VCOL + (i & 1) * 64 + (v0 + q) * 8, w);
        }
      }
      k8_arrive_warp(bars + L::EV + st * 8);

      // ---- its terms' exponents, straight from tensor memory
      k8_wait(bars + L::SS, i & 1u, ok, g.err);
      k8_fence_after();
      float y[W];
      k8_ld<W>(lane_base + L::SCOL + w0, y);
      k8_fence_before();
      k8_arrive_warp(bars + L::SR);  // the next chunk's scores may overwrite these
      if (any_scaled)
#pragma unroll
        for (int r = 0; r < W; r += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s_qf + w0 + r);
          y[r] *= f.x, y[r + 1] *= f.y, y[r + 2] *= f.z, y[r + 3] *= f.w;
        }
#pragma unroll
      for (int r = 0; r < W; r += 4) {
        const float4 m = *reinterpret_cast<const float4*>(s_neg + w0 + r);
        k8_unpair(k8_fma2(k8_pair(y[r], y[r + 1]), ct2, k8_add2(et2, k8_pair(m.x, m.y))), y[r], y[r + 1]);
        k8_unpair(k8_fma2(k8_pair(y[r + 2], y[r + 3]), ct2, k8_add2(et2, k8_pair(m.z, m.w))), y[r + 2], y[r + 3]);
      }
      if (masked)
#pragma unroll
        for (int r = 0; r < W; r += 4) {
          const int4 lo = *reinterpret_cast<const int4*>(s_lo + w0 + r);
          const int4 hi = *reinterpret_cast<const int4*>(s_hi + w0 + r);
          y[r] = pos >= lo.x && pos <= hi.x ? y[r] : -INFINITY;
          y[r + 1] = pos >= lo.y && pos <= hi.y ? y[r + 1] : -INFINITY;
          y[r + 2] = pos >= lo.z && pos <= hi.z ? y[r + 2] : -INFINITY;
          y[r + 3] = pos >= lo.w && pos <= hi.w ? y[r + 3] : -INFINITY;
        }
      float t4[4] = {y[0], y[1], y[2], y[3]};
#pragma unroll
      for (int r = 4; r + 8 <= W; r += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) t4[e] = k8_max3(t4[e], y[r + 2 * e], y[r + 2 * e + 1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) t4[e] = fmaxf(t4[e], y[W - 4 + e]);
      const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
      if (k8_vote(group, pending || top > K8_SLACK + K8_BIAS)) {
        // M of some row moves: the chunk's largest term of every row.  A row
        // without a term so far takes it as M, another only if it is past the slack.
#pragma unroll
        for (int c = 0; c < W; c += 8) {
          float v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) v[r] = y[c + r];
          const int base = k8_reduce<8>(v, [](float p, float q) { return fmaxf(p, q); });
          s_red[warp & 3][w0 + c + base] = v[0];
        }
        k8_group_sync(group);
        bool wait = false;
        if (t < W) {
          const int r = w0 + t;
          const float ym = fmaxf(fmaxf(s_red[0][r], s_red[1][r]), fmaxf(s_red[2][r], s_red[3][r]));
          float fac = 1.f, m = s_m[r];
          if (m == -INFINITY) {
            if (ym > -INFINITY) m = ym - K8_BIAS;
          } else if (ym > K8_SLACK + K8_BIAS) {
            m += ym - K8_BIAS;
            fac = k8_ex2(s_m[r] - m);
          }
          const float neg = m > -INFINITY ? K8_BIAS - m : K8_BIAS;
          s_del[r] = neg - s_neg[r];
          s_neg[r] = neg;
          s_m[r] = m;
          s_fac[r] = fac;
          wait = r < nr && s_hi[r] >= 0 && m == -INFINITY;
        }
        pending = k8_vote(group, wait);
#pragma unroll
        for (int r = 0; r < W; r += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s_fac + w0 + r);
          const float4 d = *reinterpret_cast<const float4*>(s_del + w0 + r);
          l[r] *= f.x, l[r + 1] *= f.y, l[r + 2] *= f.z, l[r + 3] *= f.w;
          y[r] += d.x, y[r + 1] += d.y, y[r + 2] += d.z, y[r + 3] += d.w;
        }
        if (i > 0) {
          k8_wait(bars + L::OU, (i - 1) & 1u, ok, g.err);
          k8_fence_after();
#pragma unroll
          for (int cc = 0; cc < W; cc += 8) {
            float o[8];
            k8_ld<8>(lane_base + L::OCOL + w0 + cc, o);
            uint32_t w[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) w[r] = __float_as_uint(o[r] * s_fac[w0 + cc + r]);
            k8_st8(lane_base + L::OCOL + w0 + cc, w);
          }
        }
      }

      // ---- terms and their sums
      uint32_t pk[W / 2];
#pragma unroll
      for (int r = 0; r < W; r += 2) {
        const float p0 = k8_ex2(y[r]), p1 = k8_ex2(y[r + 1]);
        k8_unpair(k8_fma2(k8_pair(p0, p1), ie2, k8_pair(l[r], l[r + 1])), l[r], l[r + 1]);
        const __half2 h = __floats2half2_rn(p0, p1);
        pk[r / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }

      // ---- P, once the last chunk's product has read its own
      if (i > 0) k8_wait(bars + L::OU, (i - 1) & 1u, ok, g.err);
      k8_fence_after();
#pragma unroll
      for (int r = 0; r < W; r += 8)
        k8_sts16(prow ^ (r * 2), pk[r / 2], pk[r / 2 + 1], pk[r / 2 + 2], pk[r / 2 + 3]);
      k8_st_wait();
      k8_fence_smem();
      k8_fence_before();
      k8_arrive_warp(bars + L::PW);
    }
    if (n_mine > 0) k8_wait(bars + L::OU, (n_mine - 1) & 1u, ok, g.err);
    k8_fence_after();

    // ---- sums over the keys
    const int base = k8_reduce<W>(l, [](float p, float q) { return p + q; });
    s_red[warp & 3][w0 + base] = l[0];
    k8_group_sync(group);
    if (t < W) s_l[w0 + t] = ((s_red[0][w0 + t] + s_red[1][w0 + t]) + s_red[2][w0 + t]) + s_red[3][w0 + t];
    k8_group_sync(group);

    if (C == 1) {
      // the whole of every row is here
      if (t < W && w0 + t < nr) {
        const int r = w0 + t;
        const float sum = s_l[r];
        s_fac[r] = sum == 0.f ? 0.f : 1.f / sum;
        if (a.lse)
          a.lse[(size_t)s_tok[r] * a.q_heads + s_hd[r]] =
              sum == 0.f ? -INFINITY : (s_m[r] == -INFINITY ? sum : 0.6931471805599453f * (s_m[r] - K8_BIAS) + logf(sum));
      }
      k8_group_sync(group);
      // through shared memory (the tiles have been read): stores of 16 bytes
      // instead of 2, 1118 rows of 19 sequences 153 us, 161 with the latter
      float o[W];
      k8_ld<W>(lane_base + L::OCOL + w0, o);  // anything if no product was made: not used then
      __nv_bfloat16* rows = reinterpret_cast<__nv_bfloat16*>(sm) + w0 * HD;
      if (t < HD)
#pragma unroll
        for (int r = 0; r < W; r += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s_fac + w0 + r);
          rows[r * HD + t] = __float2bfloat16_rn(f.x == 0.f ? 0.f : o[r] * f.x);
          rows[(r + 1) * HD + t] = __float2bfloat16_rn(f.y == 0.f ? 0.f : o[r + 1] * f.y);
          rows[(r + 2) * HD + t] = __float2bfloat16_rn(f.z == 0.f ? 0.f : o[r + 2] * f.z);
          rows[(r + 3) * HD + t] = __float2bfloat16_rn(f.w == 0.f ? 0.f : o[r + 3] * f.w);
        }
      k8_group_sync(group);
      for (int r = t / LPR; r < W && w0 + r < nr; r += 128 / LPR)
        *reinterpret_cast<uint4*>(a.out + s_tok[w0 + r] * a.os + s_hd[w0 + r] * HD + t % LPR * 8) =
            *reinterpret_cast<const uint4*>(rows + r * HD + t % LPR * 8);
    } else if (n_mine > 0) {
      float* part = reinterpret_cast<float*>(sm);
      float o[W];
      k8_ld<W>(lane_base + L::OCOL + w0, o);
      if (t < HD)
#pragma unroll
        for (int r = 0; r < W; ++r) part[(w0 + r) * L::OLD + t] = o[r];
    }
  }
  k8_fence_before();
  __syncthreads();
  if (warp == ISSUER) {
    k8_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(L::COLS) : "memory");
  }
  if (C == 1) return;

  // ---- merge: rank q finishes rows q, q + C, ..., HD / 4 lanes to a row, lane
  // i of them reading rank i's maximum and sum beside everyone's part
  k8_cluster_sync();
  if (warp < ISSUER) {
    constexpr int TPR = HD / 4;
    const uint32_t lanes = TPR == 32 ? 0xffffffffu : 0xffffu << (lane & 16);
    const int sub4 = lane % TPR, d = sub4 * 4;
    for (int row = rank + C * (threadIdx.x / TPR); row < nr; row += C * (CT / TPR)) {
      const uint32_t part = smb + (row * L::OLD + d) * 4;
      float m = -INFINITY, lq = 0.f;
      if (sub4 < C) {
        m = k8_remote_f(k8_remote(k8_addr(s_m) + row * 4, sub4));
        lq = k8_remote_f(k8_remote(k8_addr(s_l) + row * 4, sub4));
      }
      float4 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)  // (a rank without a chunk left no part: its weight is 0, its bytes are not used)
        if (q < C) x[q] = k8_remote_f4(k8_remote(part, q));
      float M = m;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(lanes, M, o));
      const float w = lq == 0.f ? 0.f : k8_ex2(m - M);  // 0: no key of this row there
      float sum = lq * w;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
      M = __shfl_sync(lanes, M, 0, TPR);
      sum = __shfl_sync(lanes, sum, 0, TPR);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](const float4& p, int q) {
        const float wq = __shfl_sync(lanes, w, q, TPR);
        if (wq != 0.f) {
          o.x = fmaf(p.x, wq, o.x);
          o.y = fmaf(p.y, wq, o.y);
          o.z = fmaf(p.z, wq, o.z);
          o.w = fmaf(p.w, wq, o.w);
        }
      };
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < C) add(x[q], q);
      if (C > 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (8 + q < C) x[q] = k8_remote_f4(k8_remote(part, 8 + q));
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (8 + q < C) add(x[q], 8 + q);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const long long at = s_tok[row];
      const int hq = s_hd[row];
      const __nv_bfloat162 b0 = __floats2bfloat162_rn(o.x * inv, o.y * inv),
                           b1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(a.out + at * a.os + (size_t)hq * HD + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
      if (d == 0 && a.lse)
        a.lse[(size_t)at * a.q_heads + hq] =
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
                                       K8<HD, N>::BYTES);
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
  return launch_kcl(kv8_attention_kernel<HD, N>, dim3(a.solo + ((unsigned)a.tiles * a.g.nseq * a.g.heads - a.solo) * cluster, 1, 1),
                    dim3(K8<HD, N>::THREADS), (size_t)K8<HD, N>::BYTES, st, dim3(cluster, 1, 1), a, map);
}

// Estimate (us) of a call in tiles of n rows, c CTAs to a tile, from times
// measured with 8 to 256 tiles of 3 to 257 chunks: what a CTA takes for a chunk
// and for the rest, what joining the parts adds, and what CTAs cost one another
// (a second on an SM; with c = 1 from fewer).  More clusters than run at once
// cost a second round (that depends on how the SMs are grouped: 16 tiles of 64
// rows, 2048 positions: 15 us with 4 or 8 CTAs to a tile, 25 with 16), and sizes
// between the powers of two fill more SMs (23 tiles of 128 rows, 6000
// positions: 24 us with 6, 29 with 4, 41 with 8).  Estimate and time of 16 rows
// of 4 heads, c = 1, 4, 8: one sequence at 512, 8 tiles, 12.1 11.1 10.1 and
// 12.1 10.9 10.0; two at 1024, 16.3 12.2 13.3 and 16.5 12.2 14.1; four at
// 8192, 75 35 26 and 77 35 27.  Tiles of 64 and 128, c = 1: 32 rows of one
// sequence at 1024, 16.3 20.7 and 16.8 20.8; 64 rows of eight at 8192, 111 94
// and 108 98.
static float k8_time(int n, int c, long long work, long long chunks) {
  constexpr int fit[2][8] = {{304, 152, 96, 74, 46, 35, 22, 14}, {152, 76, 46, 36, 23, 15, 8, 7}};  // clusters at once
  constexpr float chunk[4] = {0.66f, 0.8f, 1.05f, 1.3f}, rest[4] = {4.7f, 5.4f, 6.8f, 9.f},
                  join[4] = {1.3f, 1.6f, 2.2f, 3.2f};
  const int i = n == 16 ? 0 : n == 32 ? 1 : n == 64 ? 2 : 3;
  const int j = c <= 4 ? c - 1 : c == 6 ? 4 : c == 8 ? 5 : c == 12 ? 6 : 7;
  const long long ctas = work * c, rounds = (work + fit[i == 3][j] - 1) / fit[i == 3][j];
  const bool shared = i < 3 && ctas > K8_SMS, busy = i < 3 && ctas > K8_SMS / 2;
  const float slower = shared ? (c == 1 ? 1.5f : 1.6f) : busy ? 1.4f : i < 3 && c == 1 && ctas > K8_SMS / 4 ? 1.2f : 1.f;
  const float fixed = rest[i] + (c == 1 ? 0.f : c == 2 || c == 16 ? 1.4f * join[i] : join[i]);
  return (float)rounds *
         (fixed * (shared ? 1.25f : busy ? 1.15f : 1.f) + (float)((chunks + c - 1) / c) * chunk[i] * slower);
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
                n_pages, page_tokens, n_kv_heads, head_dim, pt_stride, nseq, rows, 0};
  if (rows < 0 || nseq < 0 || nseq > (1 << 20) || max_rows < 0 || max_len < 0 || (causal != 0 && causal != 1) ||
      window < 0 || (window > 0 && !causal) || !isfinite(scale))
    return DF_EINVAL;
  constexpr int sizes[] = {1, 2, 3, 4, 6, 8, 12, 16};
  if (cluster_ctas && std::find(std::begin(sizes), std::end(sizes), cluster_ctas) == std::end(sizes)) return DF_EINVAL;
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
  a.g.per_page = kv8_per_page(page_tokens);
  a.scale_log2 = (float)(scale * (1.4426950408889634 / K8_QSCALE));
  // The narrowest tile that holds a sequence's rows; more than 64 rows are cut
  // into tiles of 64 or 128.  A sequence's tiles are at most so many, and of
  // all that many hold rows at most:
  const long long wanted = (long long)a.max_rows * a.group;
  auto all_of = [&](int n) { return (wanted + n - 1) / n * nseq * n_kv_heads; };
  auto work_of = [&](int n) { return std::min(all_of(n), ((long long)rows * a.group / n + nseq) * n_kv_heads); };
  auto chunks_of = [&](int n) {  // of the longest sequence, or of a tile's window
    const long long span = window ? (long long)window + (n - 1) / a.group + 1 : max_len;
    return (std::min<long long>(span, max_len) + K8_CHUNK - 1) / K8_CHUNK;
  };
  int n = wanted <= 16 ? 16 : wanted <= 32 ? 32 : 64, cluster = 1;
  float best = INFINITY;
  for (int m = n; m <= (wanted > 64 ? 128 : n); m *= 2)
    for (const int c : sizes) {
      if (cluster_ctas ? c != cluster_ctas : c > 1 && c / 2 >= chunks_of(m)) continue;
      const float t = k8_time(m, c, work_of(m), chunks_of(m));
      if (t < best) best = t, n = m, cluster = c;
    }
  const long long tiles = (wanted + n - 1) / n;
  if (all_of(n) > (1 << 29) / 16) return DF_EINVAL;
  a.tiles = (int)tiles;
  // Tiles that fill the GPU several times, and half of it or less at the end:
  // those last ones are shared by two CTAs each (2048 rows at 6144, 512 tiles:
  // 294 us, 315 without; 40 single rows at 8192, 320 tiles: 120 and 139; below
  // 32 chunks there is nothing to gain: 48 blocks at 1024 43 and 39 us).
  const long long room = (long long)K8_SMS * (n == 128 ? K8<128, 128>::PER_SM : K8<128, 64>::PER_SM);
  if (!cluster_ctas && cluster == 1 && all_of(n) > room && all_of(n) == work_of(n) && chunks_of(n) >= 32 &&
      all_of(n) % room && all_of(n) % room * 2 <= room) {
    cluster = 2;
    a.solo = (unsigned)(all_of(n) / room * room);
  }
  a.per_cluster = ((1ull << 32) + cluster - 1) / cluster;  // exact for CTAs below 2^29
  CUtensorMap map;
  if (!k8_tmap(&map, a.g)) return DF_ECUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (head_dim == 128)
    e = n == 16   ? k8_launch<128, 16>(a, map, cluster, st)
        : n == 32 ? k8_launch<128, 32>(a, map, cluster, st)
        : n == 64 ? k8_launch<128, 64>(a, map, cluster, st)
                  : k8_launch<128, 128>(a, map, cluster, st);
  else
    e = n == 16   ? k8_launch<64, 16>(a, map, cluster, st)
        : n == 32 ? k8_launch<64, 32>(a, map, cluster, st)
        : n == 64 ? k8_launch<64, 64>(a, map, cluster, st)
                  : k8_launch<64, 128>(a, map, cluster, st);
  return e == cudaSuccess ? DF_OK : DF_ECUDA;
}

}  // extern "C"
