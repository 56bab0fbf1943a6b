// mma_tiles.cuh -- tcgen05 products of 128-row tiles shared by the backward pass and the
// attention over the 8-bit cache.  A tile is 128 rows of D bf16 in shared memory, D / 64 atoms
// of 128 rows x 128 bytes in the 128-byte swizzle that a TMA box {64, 128} writes.
#pragma once

#include "pa_device.cuh"

namespace pa {
namespace tiles {

constexpr int kRows = 128;
constexpr int kAtomBytes = kRows * 128;

template <int D>
constexpr int tile_bytes() { return D / 64 * kAtomBytes; }

// First row of the 128-row box loaded for the tile that starts at `t` of the range [s0, s1).  A
// partial last tile of a range with at least 128 rows is loaded ending at s1 (shifted back over
// rows already processed, which are masked), so no row outside the range is read: a masked row
// has weight 0, and 0 times a non-finite value is NaN in a product.  A shorter range loads
// [s0, s0 + 128), and the rows past s1 are zeroed in shared memory.
__device__ __forceinline__ int box_row(int t, int s0, int s1) {
  return (t + kRows > s1 && s1 - kRows >= s0) ? s1 - kRows : t;
}

// Walks the 128-row tiles of the ranges that group g streams.
template <typename Tables>
struct TileWalk {
  const Tables& t;
  int g, p, s0, s1, at;
  __device__ __forceinline__ TileWalk(const Tables& tab, int group) : t(tab), g(group), p(0), s0(0), s1(0), at(0) {
    advance_range();
  }
  __device__ __forceinline__ void advance_range() {
    p = next_range(t, g, p, s0, s1);
    at = s0;
  }
  __device__ __forceinline__ bool valid() const { return at < s1; }
  __device__ __forceinline__ int row() const { return box_row(at, s0, s1); }        // first row of the box
  __device__ __forceinline__ int first() const { return at - row(); }               // valid rows of the box:
  __device__ __forceinline__ int last() const { return min(at + kRows, s1) - row(); }  // [first, last)
  __device__ __forceinline__ bool is_short() const { return s1 - s0 < kRows; }
  __device__ __forceinline__ void next() {
    at += kRows;
    if (at >= s1) advance_range();
  }
};

template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* m, int row, int bh, uint32_t bar) {
#pragma unroll
  for (int a = 0; a < D / 64; ++a) tma_load_3d(dst + a * kAtomBytes, m, a * 64, row, bh, bar);
}

// Zero rows [from, 128) of a tile (a warp, whose lanes then arrive on the barrier that the issuer of
// the products waits on).  A row of an atom is 128 contiguous bytes whatever the swizzle.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane) {
#pragma unroll 1
  for (int i = from * 8 + lane; i < kRows * 8; i += 32)
#pragma unroll
    for (int a = 0; a < D / 64; ++a) *reinterpret_cast<uint4*>(tile + a * kAtomBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_async_smem();
}

// D[tmem] (+)= A[tmem] * B[smem desc]; A (128 x 16 bf16) is read from 8 TMEM columns.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint64_t kmajor(uint32_t smem) { return smem_desc_sw128(smem, 16, 1024); }
__device__ __forceinline__ uint64_t mnmajor(uint32_t smem) { return smem_desc_sw128(smem, kAtomBytes, 1024); }

// C[128 x 128] = A B^T over D: both tiles K-major.
template <int D>
__device__ __forceinline__ void product_nt(uint32_t c_tmem, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc_bf16(kRows, kRows, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = static_cast<uint32_t>(((kk >> 2) * kAtomBytes + (kk & 3) * 32) >> 4);
    mma_bf16_ss(c_tmem, a + off, b + off, id, kk > 0);
  }
}

// C[128 x D] (+)= W B over 128 rows of B (MN-major).  W is 128 x 128 bf16 in TMEM, its columns
// 0-63 (as pairs) at w_tmem and 64-127 at w_tmem + kSecond.  kSteps: which k-steps of 16 rows, a
// bit each; `first` overwrites C with the first of them.
template <int D, int kSecond, uint32_t kSteps = 0xFF>
__device__ __forceinline__ void product_w(uint32_t c_tmem, uint32_t w_tmem, uint64_t b, bool first) {
  constexpr uint32_t id = idesc_bf16(kRows, D, false, true);
  uint32_t acc = first ? 0u : 1u;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    if (kSteps >> kk & 1) {
      mma_ts(c_tmem, w_tmem + (kk >> 2) * kSecond + (kk & 3) * 8, b + static_cast<uint32_t>((kk * 16 * 128) >> 4), id, acc);
      acc = 1u;
    }
}

// A warp's 32 rows of C fp32 accumulators (one per lane) times `f`, as bf16 to the first `rows` rows of
// `dst` (D channels apart).  They pass through the warp's own 64 C bytes of shared memory, so that a
// store covers whole rows: lanes that write rows of their own touch 32 lines each time (128 x 128
// channels took 3300 cycles that way).
template <int C, int D>
__device__ __forceinline__ void store_rows(uint32_t tmem, uint8_t* stage, __nv_bfloat16* dst, float f, int rows, int lane) {
  constexpr int kChunks = C / 8;           // 16-byte chunks per row
  auto at = [&](int r, int ch) {           // 8 rows of one chunk fall in different banks
    return reinterpret_cast<uint4*>(stage + r * (2 * C) + ((ch ^ (kChunks >= 8 ? r & 7 : (r >> 1) & 3)) << 4));
  };
#pragma unroll
  for (int c = 0; c < C / 32; ++c) {
    uint32_t v[32];
    tmem_ld32(tmem + c * 32, v);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 u;
      u.x = pack_bf16x2(__uint_as_float(v[8 * i + 0]) * f, __uint_as_float(v[8 * i + 1]) * f);
      u.y = pack_bf16x2(__uint_as_float(v[8 * i + 2]) * f, __uint_as_float(v[8 * i + 3]) * f);
      u.z = pack_bf16x2(__uint_as_float(v[8 * i + 4]) * f, __uint_as_float(v[8 * i + 5]) * f);
      u.w = pack_bf16x2(__uint_as_float(v[8 * i + 6]) * f, __uint_as_float(v[8 * i + 7]) * f);
      *at(lane, c * 4 + i) = u;
    }
  }
  __syncwarp();
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 32 / kChunks) {
    const int r = r0 + lane / kChunks, ch = lane % kChunks;
    if (r < rows) *reinterpret_cast<uint4*>(dst + static_cast<size_t>(r) * D + ch * 8) = *at(r, ch);
  }
}

}  // namespace tiles
}  // namespace pa
