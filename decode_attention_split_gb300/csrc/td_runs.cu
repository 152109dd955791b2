// Instantiations, plan and launches of the attention in runs (td_runs.cuh).
#include <algorithm>
#include <mutex>

#include "td_runs.cuh"

namespace td {

namespace {

constexpr int kMaxDevices = 64;

template <int D, int NT>
cudaError_t launch_nt(const RunArgs &a, int grid, cudaStream_t stream) {
  constexpr auto kernel = runs_kernel<D, NT, kWindowPad>;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!done[device]) {
      const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 RunCfg<D, kRunStages>::SMEM + (2 * TD_MAX_BATCH + 1) * (int)sizeof(int));
      if (e != cudaSuccess) return e;
      done[device] = true;
    }
  }
  const size_t smem = RunCfg<D, kRunStages>::SMEM + (2 * (size_t)a.p.B + 1) * sizeof(int);
  return launch_pdl(kernel, dim3(grid), dim3(kRunThreads), smem, stream, a);
}

template <int D>
cudaError_t launch_d(const RunArgs &a, int grid, cudaStream_t stream) {
  const int nt = (a.p.R + 7) / 8;
  return nt == 1   ? launch_nt<D, 1>(a, grid, stream)
         : nt == 2 ? launch_nt<D, 2>(a, grid, stream)
                   : launch_nt<D, 3>(a, grid, stream);
}

template <int D, bool PREFIX, int SPLIT>
cudaError_t launch_join_split(const JoinArgs &a, cudaStream_t stream) {
  const long long groups = ((long long)a.B * a.GT + 31) / 32 * a.Hkv;
  return launch_pdl(join_kernel<D, PREFIX, SPLIT>, dim3((unsigned)(groups * (D / 64) * SPLIT)), dim3(kJoinThreads), 0, stream, a);
}

template <int D, bool PREFIX>
cudaError_t launch_join_d(const JoinArgs &a, cudaStream_t stream) {
  // one batch of loads a thread for the prefix's chunks and a few runs, while the CTAs fit the GPU at once
  const long long ctas = ((long long)a.B * a.GT + 31) / 32 * a.Hkv * (D / 64);  // without a split
  int split = 1;
  while (split < 8 && split * 4 < a.chunks + 3 && ctas * split * 2 <= 2 * 152) split *= 2;
  return split == 1   ? launch_join_split<D, PREFIX, 1>(a, stream)
         : split == 2 ? launch_join_split<D, PREFIX, 2>(a, stream)
         : split == 4 ? launch_join_split<D, PREFIX, 4>(a, stream)
                      : launch_join_split<D, PREFIX, 8>(a, stream);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

td_status plan_attn_runs(int B, int Hq, int Hkv, int T, int keys, int D, int per_sm, RunsPlan *plan) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return TD_ERR_CUDA;
  const int sms = device_sm_count(device);
  if (sms <= 0) return TD_ERR_CUDA;
  const long long GT = (long long)(Hq / Hkv) * T, RB = (GT + kMaxTileRows - 1) / kMaxTileRows;
  plan->R = (int)((GT + RB - 1) / RB);
  plan->RB = (int)RB;
  const long long groups = (long long)B * Hkv * RB;
  const long long most = groups * ((keys + kRunKeys - 1) / kRunKeys + kRunGroupUnits);
  if (most >= (1LL << 30)) return TD_ERR_UNSUPPORTED;
  const long long ctas = (most / kRunLeast + kRunWarps) / kRunWarps;
  plan->grid = (int)std::min((long long)per_sm * sms, ctas);
  plan->off_blocks = align256(((size_t)B + 2) * sizeof(int));
  plan->bytes = plan->off_blocks + align256((size_t)(groups + plan->grid * kRunWarps) * run_block_floats(plan->R, D) * sizeof(float));
  return TD_OK;
}

bool fill_runs(RunArgs *a, int D, const RunsPlan &plan, const SplitParams &p, unsigned char *ws) {
  a->p = p;
  a->p.R = plan.R;
  a->p.RB = plan.RB;
  a->p.ws_part = reinterpret_cast<float *>(ws + plan.off_blocks);
  a->plan = reinterpret_cast<int *>(ws);
  return encode_cache_map(&a->kmap, p.k, p.B, p.Hkv, p.Smax, D, kRunKeys) &&
         encode_cache_map(&a->vmap, p.v, p.B, p.Hkv, p.Smax, D, kRunKeys);
}

cudaError_t launch_runs(int D, const RunsPlan &plan, const SplitParams &p, unsigned char *ws, cudaStream_t stream) {
  RunArgs a;
  if (!fill_runs(&a, D, plan, p, ws)) return cudaErrorInvalidValue;
  return D == 64 ? launch_d<64>(a, plan.grid, stream) : launch_d<128>(a, plan.grid, stream);
}

cudaError_t launch_join(int D, const RunsPlan &plan, const SplitParams &p, const unsigned char *ws, const PrefixPart *x,
                        cudaStream_t stream) {
  JoinArgs a = {};
  a.runs = reinterpret_cast<const float *>(ws + plan.off_blocks);
  a.plan = reinterpret_cast<const int *>(ws);
  a.out = p.out, a.lse = p.lse;
  a.B = p.B, a.Hq = p.Hq, a.Hkv = p.Hkv, a.T = p.T, a.GT = p.G * p.T, a.R = plan.R, a.RB = plan.RB;
  if (x != nullptr) a.prefix = x->part, a.prefix_len = x->prefix_len, a.Pmax = x->Pmax, a.tiles = x->tiles, a.chunks = x->chunks;
  if (x != nullptr) return D == 64 ? launch_join_d<64, true>(a, stream) : launch_join_d<128, true>(a, stream);
  return D == 64 ? launch_join_d<64, false>(a, stream) : launch_join_d<128, false>(a, stream);
}

}  // namespace td
