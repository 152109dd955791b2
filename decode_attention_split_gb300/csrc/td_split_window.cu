// Attention over a sliding window with sinks: the split kernels' WIN instantiations and their launch.
//
// The query of token t, at position P = L - T + t, attends keys j <= P with j > P - window or j < sinks: for a token
// far into its context min(L, sinks + window) rows of the cache instead of L. The kernels are the plain calls', cutting
// and merging the keys in numbers without the gap between sinks and window (window_span), so chunks, grid and
// workspace follow the window's size, not the context's. What they add per score is two comparisons, and per sequence
// the copies of the stages that hold sinks in boxes of 16 rows, since the rows of one stage then lie apart.
// Measured: one token at 32k keys through a window of 4096 (24 + 8 heads of 128) 9.3 us, latency (16.8 MB, 2.5 us); 32 ragged
// sequences of up to 8k keys through one of 1024 (32 + 8 heads) 27.0 us (127 MB, 4.7 TB/s), instruction fetch and places
// left empty (one chunk a group: 256 on 304 places); six tokens of 8 sequences through 2048 23.8 us (69 MB, 2.9 TB/s), the
// 24-row step; fp32, 4 sequences through 250 (4 + 2 heads of 64) 6.3 us, latency. (Calls among others on a stream; replayed
// from a graph they take up to 5 % longer.) A launch of equal runs with a join after it took 27 us for the first, and 28.5
// instead of 37.5 for 200 sequences through a window of 128.
#include <mutex>

#include "td_internal.h"
#include "td_split_attn.cuh"
#include "td_split_cluster.cuh"
#include "td_split_mma.cuh"

namespace td {

namespace {

constexpr int kMaxDevices = 64;

// Shared-memory (and cluster-size) opt-ins of the instantiations `fns`, once per device.
template <int N>
cudaError_t opt_in(const void *const (&fns)[N], int smem, bool cluster, bool (&done)[kMaxDevices]) {
  static std::mutex mu;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[device]) return cudaSuccess;
  for (const void *fn : fns) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && cluster) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  done[device] = true;
  return cudaSuccess;
}

template <int D, int RP>
cudaError_t launch_f32(const SplitPlan &plan, const SplitParams &p, cudaStream_t stream) {
  if constexpr (SplitCfg<float, D, RP>::kFits) {
    static bool done[kMaxDevices] = {};
    const void *const fns[] = {reinterpret_cast<const void *>(&split_attn_kernel<float, D, RP, 1>)};
    const cudaError_t e = opt_in(fns, plan.smem, false, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(split_attn_kernel<float, D, RP, 1>, dim3(plan.grid), dim3(kThreads), plan.smem, stream, p);
  } else {
    return cudaErrorInvalidValue;
  }
}

template <int D>
cudaError_t launch_mma(const SplitPlan &plan, const SplitParams &p, cudaStream_t stream) {
  constexpr int W = kWindowPad;
  MmaWindowArgs a;
  if (!encode_cache_map(&a.kmap, p.k, p.B, p.Hkv, p.Smax, D) || !encode_cache_map(&a.vmap, p.v, p.B, p.Hkv, p.Smax, D) ||
      !encode_cache_map(&a.kmap16, p.k, p.B, p.Hkv, p.Smax, D, 16) ||
      !encode_cache_map(&a.vmap16, p.v, p.B, p.Hkv, p.Smax, D, 16))
    return cudaErrorInvalidValue;
  a.p = p;
  const int tile = tile_of_rows(p.R);
  if (plan.cluster > 0) {
    static bool done[kMaxDevices] = {};
    const void *const fns[] = {reinterpret_cast<const void *>(&split_attn_cluster_kernel<D, kTileN8, W>),
                               reinterpret_cast<const void *>(&split_attn_cluster_kernel<D, kTileM16, W>),
                               reinterpret_cast<const void *>(&split_attn_cluster_kernel<D, kTileN24, W>)};
    const cudaError_t e = opt_in(fns, cluster_smem<D>(), true, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(D, plan.grid, plan.cluster, stream, attr);
    if (tile == kTileN8) return cudaLaunchKernelEx(&cfg, split_attn_cluster_kernel<D, kTileN8, W>, a);
    if (tile == kTileM16) return cudaLaunchKernelEx(&cfg, split_attn_cluster_kernel<D, kTileM16, W>, a);
    return cudaLaunchKernelEx(&cfg, split_attn_cluster_kernel<D, kTileN24, W>, a);
  }
  static bool done[kMaxDevices] = {};
  const void *const fns[] = {reinterpret_cast<const void *>(&split_attn_mma_kernel<D, true, kTileN8, W>),
                             reinterpret_cast<const void *>(&split_attn_mma_kernel<D, true, kTileM16, W>),
                             reinterpret_cast<const void *>(&split_attn_mma_kernel<D, false, kTileN8, W>),
                             reinterpret_cast<const void *>(&split_attn_mma_kernel<D, false, kTileM16, W>),
                             reinterpret_cast<const void *>(&split_attn_mma_kernel<D, false, kTileN24, W>)};
  const cudaError_t e = opt_in(fns, plan.smem, false, done);
  if (e != cudaSuccess) return e;
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(plan.grid), dim3(kThreads), plan.smem, stream, a);
  };
  // the plan ahead of the wait where the plain calls make it there (launch_mma_tile)
  if (tile == kTileN8) return p.RB == 1 ? go(split_attn_mma_kernel<D, true, kTileN8, W>) : go(split_attn_mma_kernel<D, false, kTileN8, W>);
  if (tile == kTileM16)
    return p.RB == 1 ? go(split_attn_mma_kernel<D, true, kTileM16, W>) : go(split_attn_mma_kernel<D, false, kTileM16, W>);
  return go(split_attn_mma_kernel<D, false, kTileN24, W>);
}

}  // namespace

cudaError_t launch_split_window(td_dtype dtype, int D, const SplitPlan &plan, const SplitParams &p, cudaStream_t stream) {
  if (dtype == TD_BF16) return D == 64 ? launch_mma<64>(plan, p, stream) : launch_mma<128>(plan, p, stream);
  if (D == 64) {
    switch (plan.RP) {
      case 1: return launch_f32<64, 1>(plan, p, stream);
      case 2: return launch_f32<64, 2>(plan, p, stream);
      case 4: return launch_f32<64, 4>(plan, p, stream);
      default: return launch_f32<64, 8>(plan, p, stream);
    }
  }
  return plan.RP == 2 ? launch_f32<128, 2>(plan, p, stream) : launch_f32<128, 4>(plan, p, stream);
}

}  // namespace td
