// pa_device.cuh -- device-side building blocks shared by libpa's sm_100a kernels:
// mbarriers with bounded waits, TMA tensor loads, tcgen05 (TMEM allocation, MMA issue,
// commit, TMEM loads/stores) and the parameter blocks of every kernel.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pa.h"

namespace pa {

// ------------------------------------------------------------------ kernel parameters
struct AttnTables {
  int P, G, QG;
  int part_off[PA_MAX_P + 1];     // token bounds of the partitions
  int qg_row0[PA_MAX_P + 1];      // token bounds of the query groups
  int tile_start[PA_MAX_P + 1];   // prefix over query groups of 128-row query tiles (0 for idle groups)
  uint32_t fresh_bits[PA_MAX_P][PA_MAX_P / 32];  // per query group: partitions to compute
};

struct TcParams {
  CUtensorMap tm_q, tm_k, tm_v;   // 3-D maps {D, N, B*H}, box {64, 128, 1}, 128-byte swizzle
  void* o_part;
  float* lse_part;
  int* status;                    // context status word (PA_ETIMEOUT on a bounded-wait give-up)
  int BH, N, D;
  int tiles_total;                // query tiles per (b, h)
  float scale_log2;               // scale * log2(e)
  AttnTables t;
};

// Launch order of the work units of a bf16 attention grid of a few waves: CTA i processes
// unit unit[i] (a permutation of 0 .. units - 1, longest units first).
constexpr int kMaxOrderedUnits = 2048;
struct TcUnitOrder {
  uint16_t unit[kMaxOrderedUnits];
};

struct F32AttnParams {
  const float* q;
  const float* k;
  const float* v;
  float* o_part;
  float* lse_part;
  int BH, N, D;
  int tiles_total;                // 64-row query tiles per (b, h) over active query groups
  float scale;
  AttnTables t;
};

struct MergeParams {
  const void* o_fresh;
  const float* lse_fresh;
  const void* o_cached;
  const float* lse_cached;
  void* o;
  float* lse;
  float* w_partial;               // [blocks][P] per-block importance sums, or null
  int BH, N, D, P, G, QG;
  int cached_per_group;           // cached arrays hold one composed state per KV group
  int blocks_per_bh;              // row blocks per (b, h)
  int part_off[PA_MAX_P + 1];
  int qg_row0[PA_MAX_P + 1];
  int blk_start[PA_MAX_P + 1];    // prefix over query groups of row blocks
  uint32_t fresh_bits[PA_MAX_P][PA_MAX_P / 32];
};

struct ImportanceParams {
  const float* lse_part;
  const float* lse;
  float* w_partial;
  int BH, N, P, QG;
  int blocks_per_bh;
  int qg_row0[PA_MAX_P + 1];
  int blk_start[PA_MAX_P + 1];
};

struct ReduceWParams {
  const float* w_partial;         // [BH * blocks_per_bh][P]
  float* w;                       // [QG][P]
  int BH, P, QG, blocks_per_bh;
  int blk_start[PA_MAX_P + 1];
  double inv_count[PA_MAX_P];     // 1 / (BH * rows of the query group), 0 for empty groups
};


// ------------------------------------------------------------------ small helpers
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__host__ __device__ __forceinline__ bool fresh_bit(const uint32_t (*bits)[PA_MAX_P / 32], int qg, int p) {
  return (bits[qg][p >> 5] >> (p & 31)) & 1u;
}

// ------------------------------------------------------------------ mbarrier
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Record `code` in the context status word unless a graver one is there: the codes are negative, a
// wait that gave up (results are missing) is the lowest and a bad length or offset the highest.
__device__ __forceinline__ void record_status(int* status, int code) { atomicMin(status, code); }

// A device-side wait never spins for ever: after kWaitLimitNs it records PA_ETIMEOUT in
// the context status word, raises the block's abort flag (so every other role stops at
// its next wait) and returns false.
constexpr uint64_t kWaitLimitNs = 4000000000ull;   // 4 s; a whole launch takes milliseconds

__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int* status, uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      record_status(status, PA_ETIMEOUT);
      return false;
    }
  }
}

// Whole-warp form of mbar_wait: lane 0 waits (bounded) and broadcasts the outcome, so
// every lane takes the same branch afterwards (warp-uniform control flow).
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               int* status, uint64_t limit_ns = kWaitLimitNs) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  bool ok = false;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_flag, status, limit_ns);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// True on one lane of the (fully active) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// Short bounded wait used only while draining after an abort.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > 100000000ull) return;   // 0.1 s
  }
}

// ------------------------------------------------------------------ TMA
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// Box of shared memory to a tensor (rows outside it are not written), and the wait until all of the
// thread's stores are done.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(m), "r"(src), "r"(x),
               "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_store_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

// 3-D tiled load into this CTA's own shared memory, completing `bar`'s transaction count.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ void tmem_alloc(uint32_t slot_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot_smem),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// D[tmem] (+)= A[smem desc] * B[smem desc], kind::f16 (bf16 operands, fp32 accumulate).
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive once on `bar` when every tcgen05 operation this thread issued so far completes.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle, sm_100 version field.
//   K-major operand:  lbo unused (16), sbo = 1024 (stride of 8-row groups)
//   MN-major operand: lbo = stride between 64-element MN atoms, sbo = stride of 8-row K groups
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor for kind::f16: bf16 A and B, fp32 accumulator, dense.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn_major ? 1u : 0u) << 15) |
         ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 lanes x 32 columns of 32-bit TMEM words -> 32 registers per thread (row = lane).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// 32 lanes x 16 columns of 32-bit TMEM words <-> 16 registers per thread (row = lane).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}

// 32 lanes x 64 columns in one instruction -> 64 registers per thread (row = lane).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

}  // namespace pa

namespace pa {
// Hardware base-2 exponential / logarithm (MUFU ex2 / lg2, flush-to-zero).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
}  // namespace pa

namespace pa {
struct ComposeParams {
  const void* o_part;             // [P][B][H][N][D]
  const float* lse_part;          // [P][B][H][N]
  void* o_group;                  // [C][B][H][N][D], C = ceil(P / factor)
  float* lse_group;               // [C][B][H][N]
  int BH, N, P, factor;
  int nblk;                       // 128-row blocks per (b, h)
};

struct DriftParams {
  const void* o_new;              // [P][B][H][N][D]
  const void* o_ref;              // [P][B][H][N][D]
  float* partial;                 // [blocks][2][P]: sums of (new - ref)^2, ref^2
  int BH, N, P, G, QG;
  int blocks_per_bh;
  int qg_row0[PA_MAX_P + 1];
  int blk_start[PA_MAX_P + 1];
  uint32_t sel_bits[PA_MAX_P][PA_MAX_P / 32];
};

struct ReducePairParams {
  const float* partial;           // [BH * blocks_per_bh][2][P]
  float* d2;                      // [QG][P]
  float* r2;                      // [QG][P]
  int BH, P, QG, blocks_per_bh;
  int blk_start[PA_MAX_P + 1];
};
}  // namespace pa

namespace pa {
// ------------------------------------------------------------------ backward, 8-bit cache
// Attention's backward pass.  tq: query groups as owners of row tiles, fresh_bits[g] the KV
// partitions of their fresh pairs; tk: KV groups as owners, fresh_bits[g] the query partitions.
struct BwdParams {
  const void* q;
  const void* k;
  const void* v;
  const void* dout;
  const float* lse;               // [B][H][N] merged
  const float* delta;             // [B][H][N] dO.O - dLSE
  void* dq;
  void* dk;
  void* dv;
  int BH, N, D;
  int tiles_q, tiles_k;           // owner tiles per (b, h)
  float scale;
  AttnTables tq, tk;
};

// Owners of row tiles in the bf16 backward pass: their groups with the partitions they stream, and
// the launch order of the units (group, head, tile): groups with the most to stream first.  Sized
// by the number of partitions, up to 32 or up to PA_MAX_P: the parameters of a launch are then 2
// or 9 KB, and the smaller launch is microseconds sooner on its way.
template <int MP>
struct BwdSide {
  static constexpr int kWords = MP / 32;
  int P, QG, units;
  int part_off[MP + 1];
  int qg_row0[MP + 1];
  int unit_start[MP + 1];         // by place in the order
  uint32_t fresh_bits[MP][kWords];  // of empty partitions: as the one before (0 for the first)
  int tiles[MP];                  // that a group streams
  uint8_t shorts[MP];             // some of its ranges are shorter than a tile
  uint8_t order[MP];
};

template <int MP>
struct BwdTcParams {
  CUtensorMap tm_q, tm_k, tm_v, tm_do;
  const float* lse;
  const float* delta;
  void* dq;
  void* dk;
  void* dv;
  int* status;
  int N;
  float scale, scale_log2;
  BwdSide<MP> kv, q;
};
static_assert(sizeof(BwdTcParams<32>) <= 2048 && sizeof(BwdTcParams<PA_MAX_P>) <= 9 * 1024 + 128, "the sizes named above");

struct CacheStoreParams {
  const void* k;                  // [B][Hk][T][D]
  const void* v;
  const int32_t* start;           // [B] or null (0)
  void* k_codes;                  // [B][Hk][M][D]
  void* v_codes;
  float* k_scale;                 // [B][Hk][blocks]
  float* v_scale;
  int* status;
  int Hk, T, M, blocks;
  int touched;                    // cache blocks that T rows can touch
};

struct CacheAttnParams {
  const void* q;                  // [B][Hk][R][D]
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  const int32_t* lens;            // [B] or null (M)
  void* o;
  float* lse;
  float* ws_o;                    // [splits][B * Hk * R][D] when splits > 1 | [slots][slot_rows][D]
  float* ws_lse;                  // [splits][B * Hk * R]                    | [slots][slot_rows]
  int* status;
  long long rows;                 // B * Hk * R
  int B, Hk, R, M, D, blocks;
  int splits;                     // of the token axis
  int row_tiles, shares;          // few rows: 16-row tiles per KV head, equal shares of the work,
  int slot_rows;                  // rows of a scratch slot (two slots per share); 0: blocks take whole units
  float scale;
};

struct CacheAttnRowsParams {
  CUtensorMap tm_k, tm_v;         // {D, M, B * Hk} codes, boxes of 16 tokens, swizzled over a row
  CacheAttnParams c;
};

struct CacheAttnTcParams {
  CUtensorMap tm_q, tm_o;         // {D, R, B * Hk}
  CacheAttnParams c;
  int row_blocks;                 // 256-row blocks per KV head
  float scale_log2;
};

// Four e4m3 codes as two f16 pairs, lowest byte first.  Exact: f16 holds every e4m3 value.
__device__ __forceinline__ void e4m3_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// The maximal run of selected partitions at or after `from` that holds tokens, as the token
// range [s0, s1) (neighbouring partitions join); returns where to go on.  s0 == s1 at the end.
// Empty partitions carry the bit of the one before them (0 for the first), so a run of selected
// partitions is a run of set bits.  (A walk over single partitions took the producer of the bf16
// backward pass 1500 cycles for 8 of them, 2900 for 27, before its first load.)
__host__ __device__ __forceinline__ int first_bit(uint32_t x) {      // of x != 0
#ifdef __CUDA_ARCH__
  return __ffs(x) - 1;
#else
  return __builtin_ctz(x);
#endif
}
template <typename Tables>
__host__ __device__ __forceinline__ int next_range(const Tables& t, int g, int from, int& s0, int& s1) {
  constexpr int kWords = sizeof(t.fresh_bits[0]) / sizeof(uint32_t);
  s0 = s1 = 0;
  if (from >= t.P) return t.P;
  int w = from >> 5;
  uint32_t set = t.fresh_bits[g][w] & (~0u << (from & 31));
  while (set == 0) {
    if (++w == kWords) return t.P;
    set = t.fresh_bits[g][w];
  }
  const int a = w * 32 + first_bit(set);
  uint32_t clear = ~t.fresh_bits[g][w] & (~0u << (a & 31));
  while (clear == 0 && ++w < kWords) clear = ~t.fresh_bits[g][w];
  int b = t.P;
  if (clear != 0 && w * 32 + first_bit(clear) < b) b = w * 32 + first_bit(clear);
  s0 = t.part_off[a];
  s1 = t.part_off[b];
  return b;
}

// Tokens per split of a request of `len` tokens: whole cache blocks.
__device__ __forceinline__ int split_chunk(int len, int splits) {
  const int blocks = (len + PA_CACHE_BLOCK - 1) / PA_CACHE_BLOCK;
  return (blocks + splits - 1) / splits * PA_CACHE_BLOCK;
}

// Tokens held by request b's cache; a length outside [0, M] is recorded and clamped.
__device__ __forceinline__ int cache_len(const CacheAttnParams& prm, int b) {
  if (!prm.lens) return prm.M;
  const int n = prm.lens[b];
  if (n >= 0 && n <= prm.M) return n;
  record_status(prm.status, PA_EINVAL);
  return n < 0 ? 0 : prm.M;
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

}  // namespace pa
