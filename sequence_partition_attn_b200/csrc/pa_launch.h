// pa_launch.h -- host-side launchers of libpa's kernels (internal; the public ABI is pa.h).
// Each returns a cudaError_t value (0 on success).
#pragma once

#include <cuda_runtime.h>

#include "pa_device.cuh"

namespace pa {

// One CTA per work unit: CTA i takes unit i, or unit ord->unit[i] when `ord` is given.
int launch_attn_tc(const TcParams& prm, const TcUnitOrder* ord, int units, cudaStream_t st);
int attn_tc_tile_rows();

int launch_attn_f32(const F32AttnParams& prm, cudaStream_t st);
int attn_f32_tile_rows();

int launch_merge(const MergeParams& prm, int dtype, cudaStream_t st);
int merge_rows_per_block();
int launch_importance(const ImportanceParams& prm, cudaStream_t st);
int launch_reduce_w(const ReduceWParams& prm, cudaStream_t st);

int compose_rows_per_block();
int launch_compose(const ComposeParams& prm, int dtype, int D, cudaStream_t st);

int launch_wait_selftest(int* status, uint64_t limit_ns, cudaStream_t st);

int drift_rows_per_block();
int launch_drift(const DriftParams& prm, int dtype, int D, cudaStream_t st);
int launch_reduce_pair(const ReducePairParams& prm, cudaStream_t st);

// dst[h][dst_n0 + n - n0][:] = src[n][h][:], n in [n0, n1); dst has dst_N tokens per head.
int launch_relayout(const void* src, void* dst, long long n0, long long n1, long long dst_n0, int dst_N,
                    int H, int row_bytes, int sm_count, cudaStream_t st);

// delta[row] = dout[row] . o[row] - dlse[row] (dlse may be null).
int launch_delta(const void* o, const void* dout, const float* dlse, float* delta, long long rows, int D, int dtype,
                 cudaStream_t st);
int launch_attn_bwd_f32(const BwdParams& prm, int own_rows, cudaStream_t st);     // own_rows 32 or 64

int attn_bwd_tc_tile_rows();
int launch_attn_bwd_tc(const BwdTcParams<32>& prm, int D, cudaStream_t st);
int launch_attn_bwd_tc(const BwdTcParams<PA_MAX_P>& prm, int D, cudaStream_t st);

int launch_cache_store(const CacheStoreParams& prm, unsigned blocks, int dtype, int D, cudaStream_t st);

int cache_attn_rows_tile_rows(int R, int dtype);
int cache_attn_rows_resident(int R, int dtype);     // blocks of threads per SM, each with a share of the work
constexpr int kCacheRowsBox = 16;       // tokens per box of its tensor maps
int launch_cache_attn_rows(const CacheAttnRowsParams& par, int dtype, cudaStream_t st);
int cache_attn_tc_block_rows();
int launch_cache_attn_tc(const CacheAttnTcParams& p, unsigned units, cudaStream_t st);

}  // namespace pa
