// attn_bwd.cu -- backward pass of attention with reuse: the per-row terms, and the gradients of
// fp32 inputs (attn_bwd_tc.cu: bf16).
//
// With the merged outputs (O, LSE) of pa_partition_attn + pa_merge_states, the fresh pairs'
// share of the output is P_ij v_j with P_ij = exp(s_ij - LSE_i), s = scale * q.k: the
// partition weights exp(LSE_p - LSE) and the partition probabilities exp(s - LSE_p) multiply
// to it, so the per-partition states are not needed.  Reused states are constants.  Hence
//   delta_i = dO_i . O_i - dLSE_i,   dS_ij = P_ij (dO_i . v_j - delta_i),
//   dQ_i = scale sum_j dS_ij k_j,    dK_j = scale sum_i dS_ij q_i,    dV_j = sum_i P_ij dO_i
// over the fresh pairs.  P is recomputed from q, k and LSE, never stored.
//
// Blocks own the rows of what they sum and stream the other side: some for dQ (own queries,
// stream keys), some for dK and dV (own keys, stream queries).  Every sum is taken by one block in
// a fixed order, so results do not change from run to run; the price is that s and dO.v are
// computed twice (7 products instead of 5).
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

// ------------------------------------------------------------------ delta
// One group of lanes per row, 16 bytes of O and dO per lane.  Bound by HBM: both read once.
template <typename T, int D>
__global__ void __launch_bounds__(256) delta_kernel(const T* __restrict__ o, const T* __restrict__ dout,
                                                    const float* __restrict__ dlse, float* __restrict__ delta,
                                                    long long rows) {
  constexpr int kLanes = D * sizeof(T) / 16;
  asm volatile("griddepcontrol.launch_dependents;");
  const long long row = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int c = threadIdx.x % kLanes;
  float sum = 0.0f;
  if (row < rows) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(o) + row * kLanes + c);
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(dout) + row * kLanes + c);
    const uint32_t au[4] = {a.x, a.y, a.z, a.w}, bu[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 4) {
        sum = fmaf(__uint_as_float(au[i]), __uint_as_float(bu[i]), sum);
      } else {
        sum = fmaf(__uint_as_float(au[i] << 16), __uint_as_float(bu[i] << 16), sum);
        sum = fmaf(__uint_as_float(au[i] & 0xFFFF0000u), __uint_as_float(bu[i] & 0xFFFF0000u), sum);
      }
    }
  }
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (row < rows && c == 0) delta[row] = sum - (dlse ? dlse[row] : 0.0f);
}

// ------------------------------------------------------------------ fp32 on the tensor cores
// An fp32 value is a sum of three bf16 ones: x = x0 + x1 + x2 with x0 its upper half (cut, so that it
// cannot overflow), x1 the rest rounded and x2 what is left, off by 2^-25 of x.  A product of two values takes
// the six terms x0y0, x0y1, x1y0, x1y1, x0y2, x2y0; the others are below 2^-22 of it, and the sums
// are fp32.  That is six bf16 products for one, at the tensor cores' rate: 24 x 1536 x 128, all
// pairs, takes 1.82 ms (56 fp32 TFLOP/s executed, 334 of bf16), and 2 x 1024 x 64 takes 55 us.  The
// packed multiply-add units took 2.70 ms and 106 us.  Bound by the tensor cores' warp products,
// then by the shared-memory reads of their operands (about 3/4 of the products' time).
//
// A block owns kOwn rows and streams tiles of the other side; its 8 warps are kOwn / 16 groups of
// 16 own rows times kT / 16 groups of 16 streamed rows.  With A the own and B the streamed rows,
//   dK, dV (own K, V; stream Q, dO):  S^T = K Q^T, dP^T = V dO^T, dK += dS^T Q, dV += P^T dO
//   dQ     (own Q, dO; stream K, V):  S = Q K^T, dP = dO V^T, dQ += dS K
// so both are X = A0 B0^T, Y = A1 B1^T, acc0 += dS(X, Y) B0, acc1 += P(X) B1.  X and Y leave the
// products in the layout in which P and dS enter the next ones.  The groups of streamed rows sum
// into accumulators of their own, joined in order at the end.
constexpr int kThreads = 256;

template <int D, int kOwn>
struct Shape {
  static constexpr int kRowGroups = kOwn / 16, kStrGroups = 8 / kRowGroups;
  static constexpr int kT = 16 * kStrGroups;         // streamed rows per tile
  static constexpr int kRow = 2 * D;                 // bytes; 16-byte chunk c of row r lies at chunk c ^ (r & 7)
  static constexpr int kOwnPlane = kOwn * kRow, kStrPlane = kT * kRow;
  static constexpr int kOwnAt = 0;                   // [tensor][plane][row][D] bf16
  static constexpr int kStrAt = kOwnAt + 6 * kOwnPlane;
  static constexpr int kRawBytes = 2 * kT * D * 4, kStatBytes = 2 * kT * 4;
  // two buffers of planes where they fit (all but D = 128 with 64 streamed rows)
  static constexpr int kBuffers = kStrAt + 12 * kStrPlane + kRawBytes + 2 * kStatBytes <= 227 * 1024 ? 2 : 1;
  static constexpr int kRawAt = kStrAt + kBuffers * 6 * kStrPlane;      // the tile after, [tensor][row][D] fp32
  static constexpr int kStatAt = kRawAt + kRawBytes;         // lse, delta by streamed row, per buffer
  static constexpr int kBytes = kStatAt + kBuffers * kStatBytes;
  static_assert((kStrGroups - 1) * 2 * kOwn * D * 4 <= kStatAt - kStrAt, "the join reuses the streamed tiles");
};

__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c0 += a b for columns 0..7 of b, c1 for columns 8..15, and the same for d, x and y: all six terms,
// the smallest first, on four sums in turn (a product takes as long as four take to issue).  The
// tensor cores cut their sums instead of rounding them, which adds up over a long axis (an error of
// 5e-6 of the gradients of 1024 rows; plain fp32 sums 7e-7, these 4e-7): the terms of each 16 summed elements start
// from zero and are added to the running sums in fp32.
__device__ __forceinline__ void mma_terms(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[3][4], const uint32_t (&b)[3][4],
                                          float (&d0)[4], float (&d1)[4], const uint32_t (&x)[3][4], const uint32_t (&y)[3][4]) {
  constexpr int ia[6] = {0, 2, 1, 0, 1, 0}, ib[6] = {2, 0, 1, 1, 0, 0};
  float s[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[i][e] = 0.0f;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    mma(s[0], a[ia[i]], b[ib[i]][0], b[ib[i]][1]);
    mma(s[1], a[ia[i]], b[ib[i]][2], b[ib[i]][3]);
    mma(s[2], x[ia[i]], y[ib[i]][0], y[ib[i]][1]);
    mma(s[3], x[ia[i]], y[ib[i]][2], y[ib[i]][3]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    c0[e] += s[0][e];
    c1[e] += s[1][e];
    d0[e] += s[2][e];
    d1[e] += s[3][e];
  }
}

// The three terms of two values, as bf16 pairs.
__device__ __forceinline__ void split2(float x, float y, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  const uint32_t xu = __float_as_uint(x), yu = __float_as_uint(y);
  t0 = __byte_perm(xu, yu, 0x7632);
  const float x1 = x - __uint_as_float(xu & 0xFFFF0000u), y1 = y - __uint_as_float(yu & 0xFFFF0000u);
  t1 = pack_bf16x2(x1, y1);
  t2 = pack_bf16x2(x1 - __uint_as_float(t1 << 16), y1 - __uint_as_float(t1 & 0xFFFF0000u));
}

// Eight channels of a row into its three planes.
template <int kPlane>
__device__ __forceinline__ void split_store(uint8_t* planes, int row_bytes, int r, int chunk, float4 a, float4 b) {
  uint32_t t[3][4];
  split2(a.x, a.y, t[0][0], t[1][0], t[2][0]);
  split2(a.z, a.w, t[0][1], t[1][1], t[2][1]);
  split2(b.x, b.y, t[0][2], t[1][2], t[2][2]);
  split2(b.z, b.w, t[0][3], t[1][3], t[2][3]);
  uint8_t* at = planes + r * row_bytes + ((chunk ^ (r & 7)) << 4);
#pragma unroll
  for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(at + p * kPlane) = make_uint4(t[p][0], t[p][1], t[p][2], t[p][3]);
}

// kDq: the block owns queries and streams keys; else it owns keys and streams queries.
template <int D, int kOwn, bool kDq>
__device__ __forceinline__ void bwd_unit(const BwdParams& prm, int tile, uint8_t* smem) {
  using S = Shape<D, kOwn>;
  constexpr int kT = S::kT;
  const AttnTables& t = kDq ? prm.tq : prm.tk;
  const int bh = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = warp % S::kRowGroups, sg = warp / S::kRowGroups;
  const int gid = lane >> 2, tig = lane & 3;
  const uint32_t sbase = smem_u32(smem);
  float* stats = reinterpret_cast<float*>(smem + S::kStatAt);
  int g = 0;
  while (g + 1 < t.QG && t.tile_start[g + 1] <= tile) ++g;
  const int own0 = t.qg_row0[g] + (tile - t.tile_start[g]) * kOwn;
  const int own1 = min(own0 + kOwn, t.qg_row0[g + 1]);
  const size_t head = static_cast<size_t>(bh) * prm.N;
  const float* q = static_cast<const float*>(prm.q) + head * D;
  const float* k = static_cast<const float*>(prm.k) + head * D;
  const float* v = static_cast<const float*>(prm.v) + head * D;
  const float* dout = static_cast<const float*>(prm.dout) + head * D;
  const float* own[2] = {kDq ? q : k, kDq ? dout : v};
  const float* str[2] = {kDq ? k : q, kDq ? v : dout};
  // +inf makes every P of the row 0: rows outside the range, and rows without any key
  auto stat_lse = [&](int r, int end) {
    const float l = r < end ? prm.lse[head + r] : INFINITY;
    return l == -INFINITY ? INFINITY : l;
  };

  // Pieces of 8 channels; rows at or past `end` become 0, so that nothing outside the range (which
  // may be non-finite) reaches a product.  A thread splits the pieces it copied.
  constexpr int kPieces = kT * D / 8 / kThreads;
  auto fetch = [&](int r0, int end) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < kPieces; ++n) {
        const int i = n * kThreads + threadIdx.x;
        const int r = r0 + i / (D / 8);
        const bool in = r < end;
        const float* src = str[x] + (in ? static_cast<size_t>(r) * D + i % (D / 8) * 8 : 0);
        const uint32_t dst = sbase + S::kRawAt + (x * kT * D + i * 8) * 4;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16), "l"(src + 4), "r"(in ? 16 : 0) : "memory");
      }
  };
#pragma unroll
  for (int x = 0; x < 2; ++x)
    for (int i = threadIdx.x; i < kOwn * D / 8; i += kThreads) {
      const int r = i / (D / 8), c = i % (D / 8);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      if (own0 + r < own1) {
        const float* src = own[x] + static_cast<size_t>(own0 + r) * D + c * 8;
        a = load4(src);
        b = load4(src + 4);
      }
      split_store<S::kOwnPlane>(smem + S::kOwnAt + x * 3 * S::kOwnPlane, S::kRow, r, c, a, b);
    }
  asm volatile("griddepcontrol.wait;" ::: "memory");           // delta is written
  float lse_own[2] = {INFINITY, INFINITY}, delta_own[2] = {0.0f, 0.0f};    // rows gid, gid + 8 (dQ)
  if (kDq)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = own0 + rg * 16 + gid + 8 * h;
      lse_own[h] = stat_lse(r, own1);
      delta_own[h] = r < own1 ? prm.delta[head + r] : 0.0f;
    }

  float acc0[D / 8][4], acc1[D / 8][4];              // dQ | dK, dV
#pragma unroll
  for (int c = 0; c < D / 8; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc0[c][e] = acc1[c][e] = 0.0f;

  // this lane's row and chunk in the four 8 x 8 matrices of a load: A tiles and transposed B tiles
  // take rows 0..15 of chunk 0, then of chunk 1; B tiles chunks 0, 1 of rows 0..7, then of 8..15
  const int swz = lane & 7;
  const uint32_t rows_first = (swz + ((lane >> 3) & 1) * 8) * S::kRow, rows_last = (swz + (lane >> 4) * 8) * S::kRow;
  const uint32_t xor_first = ((lane >> 4) ^ swz) << 4, xor_last = (((lane >> 3) & 1) ^ swz) << 4;
  const uint32_t a_row = sbase + S::kOwnAt + rg * 16 * S::kRow + rows_first;
  const uint32_t b_row0 = sbase + S::kStrAt + sg * 16 * S::kRow + rows_last;
  const uint32_t w_row0 = sbase + S::kStrAt + sg * 16 * S::kRow + rows_first;

  // Tile i is used while tile i + 1 is split and tile i + 2 copied.  With two buffers, half of the
  // warps (one of each scheduler's two) split first and the others last, so that one splits while
  // the other feeds the tensor cores.
  int s0, s1;
  int p = next_range(t, g, 0, s0, s1);
  int st0 = s0;
  int copied = 0, ready = 0;                         // rows of the copied and of the split tile
  float lse_next = INFINITY, delta_next = 0.0f;      // of row threadIdx.x of the copied tile
  auto copy = [&]() {
    copied = 0;
    if (st0 >= s1) return;
    copied = min(kT, s1 - st0);
    fetch(st0, s1);
    if (!kDq && threadIdx.x < kT) {
      const int r = st0 + threadIdx.x;
      lse_next = stat_lse(r, s1);
      delta_next = r < s1 ? prm.delta[head + r] : 0.0f;
    }
    st0 += kT;
    if (st0 >= s1) {
      p = next_range(t, g, p, s0, s1);
      st0 = s0;
    }
  };
  auto split = [&](int buf) {
    ready = copied;
    if (copied == 0) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < kPieces; ++n) {
        const int i = n * kThreads + threadIdx.x;
        const float4* raw = reinterpret_cast<const float4*>(smem + S::kRawAt + (x * kT * D + i * 8) * 4);
        split_store<S::kStrPlane>(smem + S::kStrAt + (buf * 6 + x * 3) * S::kStrPlane, S::kRow, i / (D / 8), i % (D / 8), raw[0], raw[1]);
      }
    if (!kDq && threadIdx.x < kT) {
      stats[buf * 2 * kT + threadIdx.x] = lse_next;
      stats[buf * 2 * kT + kT + threadIdx.x] = delta_next;
    }
    copy();
  };
  copy();
  split(0);
  __syncthreads();
  for (int buf = 0; ready > 0;) {
    const int n = ready, next = S::kBuffers == 2 ? buf ^ 1 : 0;
    const float* sLse = stats + buf * 2 * kT;
    const float* sDelta = sLse + kT;
    const uint32_t b_row = b_row0 + buf * 6 * S::kStrPlane, w_row = w_row0 + buf * 6 * S::kStrPlane;
    if (S::kBuffers == 2 && warp < 4) split(next);

    float x[2][4], y[2][4];                          // own rows gid, gid + 8; streamed rows 8 h + 2 tig + {0, 1}
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[h][e] = y[h][e] = 0.0f;
#pragma unroll 4
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a0[3][4], b0[3][4], a1[3][4], b1[3][4];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        ldmatrix(a0[i], a_row + i * S::kOwnPlane + ((ks * 32) ^ xor_first));
        ldmatrix(b0[i], b_row + i * S::kStrPlane + ((ks * 32) ^ xor_last));
        ldmatrix(a1[i], a_row + (3 + i) * S::kOwnPlane + ((ks * 32) ^ xor_first));
        ldmatrix(b1[i], b_row + (3 + i) * S::kStrPlane + ((ks * 32) ^ xor_last));
      }
      mma_terms(x[0], x[1], a0, b0, y[0], y[1], a1, b1);
    }
    uint32_t wp[3][4], wd[3][4];                     // P and dS as operands
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float pe[4], de[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = sg * 16 + 8 * h + 2 * tig + (e & 1);
        const float l = kDq ? lse_own[e >> 1] : sLse[c], d = kDq ? delta_own[e >> 1] : sDelta[c];
        pe[e] = c < n ? expf(fmaf(x[h][e], prm.scale, -l)) : 0.0f;
        de[e] = c < n ? pe[e] * (y[h][e] - d) : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (!kDq) split2(pe[2 * e], pe[2 * e + 1], wp[0][2 * h + e], wp[1][2 * h + e], wp[2][2 * h + e]);
        split2(de[2 * e], de[2 * e + 1], wd[0][2 * h + e], wd[1][2 * h + e], wd[2][2 * h + e]);
      }
    }
    // 16 channels of dK and dV at a time, 32 of dQ
#pragma unroll
    for (int c = 0; c < D / 16; c += kDq ? 2 : 1) {
      uint32_t b0[3][4], b1[3][4];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        ldmatrix_trans(b0[i], w_row + i * S::kStrPlane + ((c * 32) ^ xor_first));
        ldmatrix_trans(b1[i], w_row + (kDq ? i : 3 + i) * S::kStrPlane + (((kDq ? c + 1 : c) * 32) ^ xor_first));
      }
      if (kDq)
        mma_terms(acc0[2 * c], acc0[2 * c + 1], wd, b0, acc0[(2 * c + 2) % (D / 8)], acc0[(2 * c + 3) % (D / 8)], wd, b1);
      else
        mma_terms(acc0[2 * c], acc0[2 * c + 1], wd, b0, acc1[2 * c], acc1[2 * c + 1], wp, b1);
    }
    if (S::kBuffers == 1) __syncthreads();
    if (S::kBuffers == 1 || warp >= 4) split(next);
    __syncthreads();
    buf = next;
  }

  // Join of the groups of streamed rows, in order.
  float4* join = reinterpret_cast<float4*>(smem + S::kStrAt);
  auto slot = [&](int group, int x, int c) { return join + ((((group - 1) * 2 + x) * S::kRowGroups + rg) * (D / 8) + c) * 32 + lane; };
  if (sg > 0) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      *slot(sg, 0, c) = make_float4(acc0[c][0], acc0[c][1], acc0[c][2], acc0[c][3]);
      if (!kDq) *slot(sg, 1, c) = make_float4(acc1[c][0], acc1[c][1], acc1[c][2], acc1[c][3]);
    }
  }
  __syncthreads();
  if (sg > 0) return;
  const int r = own0 + rg * 16 + gid;
  auto finish = [&](float* dst, float (&acc)[D / 8][4], int x, float f) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
#pragma unroll
      for (int group = 1; group < S::kStrGroups; ++group) {
        const float4 u = *slot(group, x, c);
        acc[c][0] += u.x;
        acc[c][1] += u.y;
        acc[c][2] += u.z;
        acc[c][3] += u.w;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (r + 8 * h < own1)
          *reinterpret_cast<float2*>(dst + (head + r + 8 * h) * D + c * 8 + 2 * tig) = make_float2(acc[c][2 * h] * f, acc[c][2 * h + 1] * f);
    }
  };
  finish(static_cast<float*>(kDq ? prm.dq : prm.dk), acc0, 0, prm.scale);
  if (!kDq) finish(static_cast<float*>(prm.dv), acc1, 1, 1.0f);
}

// One launch for both: the heavier blocks (dK, dV: four products) first.  At D = 64 two blocks of 64
// rows per SM (24 x 1536 x 64: 0.90 ms with the few spills of 128 registers, 1.03 ms with one).
template <int D, int kOwn>
__global__ void __launch_bounds__(kThreads, D == 64 && kOwn == 64 ? 2 : 1) attn_bwd_f32_kernel(const __grid_constant__ BwdParams prm) {
  extern __shared__ __align__(16) uint8_t smem[];
  if (static_cast<int>(blockIdx.x) < prm.tiles_k)
    bwd_unit<D, kOwn, false>(prm, blockIdx.x, smem);
  else
    bwd_unit<D, kOwn, true>(prm, blockIdx.x - prm.tiles_k, smem);
}

template <int D, int kOwn>
int f32_impl(const BwdParams& prm, cudaStream_t st) {
  constexpr int smem = Shape<D, kOwn>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_bwd_f32_kernel<D, kOwn>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg = {};             // ahead of the end of the delta kernel, which its blocks wait for
  cfg.gridDim = dim3(prm.tiles_k + prm.tiles_q, prm.BH);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, attn_bwd_f32_kernel<D, kOwn>, prm));
}

template <typename T, int D>
int delta_impl(const void* o, const void* dout, const float* dlse, float* delta, long long rows, cudaStream_t st) {
  constexpr int kPerBlock = 256 * 16 / (D * static_cast<int>(sizeof(T)));
  delta_kernel<T, D><<<static_cast<unsigned>((rows + kPerBlock - 1) / kPerBlock), 256, 0, st>>>(
      static_cast<const T*>(o), static_cast<const T*>(dout), dlse, delta, rows);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_delta(const void* o, const void* dout, const float* dlse, float* delta, long long rows, int D, int dtype,
                 cudaStream_t st) {
  if (dtype == PA_BF16)
    return D == 64 ? delta_impl<__nv_bfloat16, 64>(o, dout, dlse, delta, rows, st)
                   : delta_impl<__nv_bfloat16, 128>(o, dout, dlse, delta, rows, st);
  return D == 64 ? delta_impl<float, 64>(o, dout, dlse, delta, rows, st)
                 : delta_impl<float, 128>(o, dout, dlse, delta, rows, st);
}

int launch_attn_bwd_f32(const BwdParams& prm, int own_rows, cudaStream_t st) {
  if (own_rows == 64) return prm.D == 64 ? f32_impl<64, 64>(prm, st) : f32_impl<128, 64>(prm, st);
  return prm.D == 64 ? f32_impl<64, 32>(prm, st) : f32_impl<128, 32>(prm, st);
}

}  // namespace pa
