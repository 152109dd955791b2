// Plan of the runs over the sequences' own keys, and the join's launch (td_runs.cuh).
#include <algorithm>

#include "td_runs.cuh"

namespace td {

namespace {

constexpr int kSms = 152;

template <int D, int SPLIT>
cudaError_t launch_join_split(const JoinArgs &a, cudaStream_t stream) {
  constexpr int threads = join_threads(SPLIT), slabs = D / 8 / (threads / 32 / SPLIT);
  constexpr int most = 200 * 1024, own = 40 * threads + 1024;  // a CTA's static shared memory and what the system takes
  const long long ctas = ((long long)a.B * a.GT + 31) / 32 * a.Hkv * slabs;
  const long long per = (ctas + kSms - 1) / kSms;  // an SM's share
  const int spread = per <= kJoinSmThreads / threads ? std::min((int)(224 * 1024 / per) - own, most) / 1024 * 1024 : 0;
  static OptIn opt_in;
  const cudaError_t e = opt_in(reinterpret_cast<const void *>(&join_kernel<D, SPLIT>), most);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_kernel<D, SPLIT>, dim3((unsigned)ctas), dim3(threads), spread, stream, a);
}

template <int D>
cudaError_t launch_join_d(const JoinArgs &a, cudaStream_t stream) {
  // one batch of loads a thread for the prefix's chunks and a few runs, while all rows' threads fit the GPU at once
  const long long threads = ((long long)a.B * a.GT + 31) / 32 * a.Hkv * (D / 8) * 32;  // without a split
  int split = 1;
  while (split < 8 && split * kJoinBatch < a.chunks + 3 && threads * split * 2 <= kJoinSmThreads * kSms) split *= 2;
  return split == 1   ? launch_join_split<D, 1>(a, stream)
         : split == 2 ? launch_join_split<D, 2>(a, stream)
         : split == 4 ? launch_join_split<D, 4>(a, stream)
                      : launch_join_split<D, 8>(a, stream);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

td_status plan_attn_runs(int B, int Hq, int Hkv, int T, int keys, int D, RunsPlan *plan) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return TD_ERR_CUDA;
  const int sms = device_sm_count(device);
  if (sms <= 0) return TD_ERR_CUDA;
  const long long GT = (long long)(Hq / Hkv) * T, RB = (GT + kMaxTileRows - 1) / kMaxTileRows;
  plan->R = (int)((GT + RB - 1) / RB);
  plan->RB = (int)RB;
  const long long groups = (long long)B * Hkv * RB;
  const long long most = groups * ((keys + kRunKeys - 1) / kRunKeys + kRunGroupUnits);
  if (most >= (1LL << 30) || B * GT > (1LL << 26)) return TD_ERR_UNSUPPORTED;  // counted in 32 bits
  const long long ctas = (most / kRunLeast + kRunWarps) / kRunWarps;
  plan->grid = (int)std::min((long long)sms, ctas);
  plan->bytes = align256((size_t)(groups + plan->grid * kRunWarps) * run_block_floats(plan->R, D) * sizeof(float));
  return TD_OK;
}

bool fill_runs(RunArgs *a, int D, const RunsPlan &plan, const SplitParams &p, unsigned char *ws) {
  a->p = p;
  a->p.R = plan.R;
  a->p.RB = plan.RB;
  a->p.ws_part = reinterpret_cast<float *>(ws);
  return encode_cache_map(&a->kmap, p.k, p.B, p.Hkv, p.Smax, D, kRunKeys) &&
         encode_cache_map(&a->vmap, p.v, p.B, p.Hkv, p.Smax, D, kRunKeys);
}

cudaError_t launch_join(int D, const RunsPlan &plan, const SplitParams &p, const unsigned char *ws, const PrefixPart &x,
                        cudaStream_t stream) {
  JoinArgs a = {};
  a.runs = reinterpret_cast<const float *>(ws);
  a.seq_lens = p.seq_lens;
  a.out = p.out, a.lse = p.lse;
  a.B = p.B, a.Hq = p.Hq, a.Hkv = p.Hkv, a.T = p.T, a.GT = p.G * p.T, a.R = plan.R, a.RB = plan.RB;
  a.Smax = p.Smax, a.grid = x.grid;
  a.prefix = x.part, a.prefix_len = x.prefix_len, a.Pmax = x.Pmax, a.tiles = x.tiles, a.chunks = x.chunks;
  return D == 64 ? launch_join_d<64>(a, stream) : launch_join_d<128>(a, stream);
}

}  // namespace td
