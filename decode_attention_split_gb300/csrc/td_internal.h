// Host-side interfaces between the td translation units (not part of the public ABI).
#pragma once

#include <mutex>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "td.h"

namespace td {

struct SplitParams;

// Launch geometry and workspace layout of one split-attention call.
struct SplitPlan {
  bool mma;      // tensor-core kernel (bf16) or CUDA-core kernel
  int RP;        // CUDA-core: padded query rows per CTA (1, 2, 4 or 8); tensor-core: m tiles (1 or 2)
  int R;         // real query rows per CTA
  int RB;        // row blocks per kv head
  int ns_ws;     // partial slots per query row
  int p_target;  // CTAs that fill the GPU once
  bool spare;    // p_target leaves one slot per group for the previous call's merging CTAs
  int grid;      // CTAs launched
  int smem;      // dynamic shared memory per CTA
  int min_chunk; // smallest automatic chunk (keys)
  int warm;      // 64-row units of K and V each CTA warms in L2 before the wait for the previous kernel
  int cluster;   // 0: persistent kernel; else CTAs per cluster of the cluster kernel (grid = groups x cluster)
  int counters_n;  // completion and slice-merge counters before the fused step's read count in the workspace
  bool q8;       // int8 cache (codes + per-row scales): the quantised-cache kernel
  bool f8;       // block-scaled e4m3 cache: its kernel
  bool runs;     // its work cut into equal runs of stages instead of chunks
  bool window;   // windowed attention: the kernels' WIN instantiations
  bool merge_apart;  // its partials merged by a second launch
  long long n_part;  // partial blocks in the workspace
  size_t off_pieces, off_part, bytes;  // workspace layout: counters, pieces (merge_apart), partial blocks
};

// Records a failed CUDA call for td_last_cuda_error (and clears the runtime's last-error slot,
// so a later call does not report it as its own); returns TD_ERR_CUDA.
td_status cuda_fail(cudaError_t e);

// What the caches of an attention call hold: rows of the call's dtype, int8 codes with per-row
// scales, or e4m3 codes with per-block scales (q and out are bf16 for both, dtype TD_BF16).
enum class KvFormat { kRows, kQ8, kF8 };

// Fills *plan for the current device; TD_OK, or an error for unsupported shapes. window > 0: windowed attention
// with so many sinks (both at most Smax).
td_status plan_split(td_dtype dtype, int B, int Hq, int Hkv, int T, int Smax, int D, int split, SplitPlan *plan,
                     KvFormat format = KvFormat::kRows, int window = 0, int sinks = 0);

// The windowed kernels' launch (td_split_window.cu).
cudaError_t launch_split_window(td_dtype dtype, int D, const SplitPlan &plan, const SplitParams &p, cudaStream_t stream);

// The block-scaled kernel for row blocks of R rows: its function (for the occupancy query) and
// dynamic shared memory, and its launch.
const void *f8_kernel(int D, int R, int *smem);
cudaError_t launch_split_f8(int D, const SplitPlan &plan, const SplitParams &p, cudaStream_t stream);

// Appends to the block-scaled 8-bit cache (the rotation is skipped when cos_t is null).
struct AppendF8 {
  const void *q;   // [B, Hq, T, D] or null
  void *q_out;
  const void *k_new, *v_new;  // [B, Hkv, T, D]
  const float *cos_t, *sin_t;
  const int32_t *positions;   // [B, T, A] or null: row L + t
  const int32_t *axes;        // [D / 2] or null: axis 0
  uint8_t *k_codes, *v_codes;  // [B, Hkv, Smax, D]
  float *k_scales, *v_scales;  // [B, Hkv, NB]
  int32_t *seq_lens;
  uint32_t *status;
  int B, Hq, Hkv, T, Smax, NB, block_log2, A, table_rows, advance;
  int per_cta, team;  // tiles kernel: heads of a CTA, threads of a head
};
// Longest chunk of new rows that the warp-per-head kernel takes, and its largest CTA.
constexpr int kF8RowsT = 12;
constexpr int kF8RowsThreads = 1024;
cudaError_t launch_append_f8(size_t elem_bytes, int D, const AppendF8 &p, cudaStream_t stream);

// seq_lens[b] += T for the sequences whose T rows fit, as a launch of its own after their append's.
cudaError_t launch_advance(int32_t *seq_lens, int B, int T, int Smax, cudaStream_t stream);

// Append to a cache of rows with the queries and keys normed and rotated first.
struct NormAppend {
  const void *q;   // [B, Hq, T, D] or null (Hq 0)
  void *q_out;
  const void *k_new, *v_new;  // [B, Hkv, T, D]
  const float *q_weight, *k_weight;  // [D]
  const float *cos_t, *sin_t;        // [table_rows, D / 2]
  const int32_t *positions;   // [B, T, A] or null: row L + t
  const int32_t *axes;        // [D / 2] or null: axis 0
  void *k_cache, *v_cache;    // [B, Hkv, Smax, D]
  int32_t *seq_lens;
  uint32_t *status;
  float eps;
  int B, Hq, Hkv, T, Smax, A, table_rows, advance;
  int per_cta, head_groups;  // a chunk's launch: heads of a CTA, CTAs that share a token tile
};
cudaError_t launch_norm_append(size_t elem_bytes, int D, const NormAppend &p, cudaStream_t stream);

// Read-back of rows start[b] .. start[b] + N - 1 (start null: 0).
struct ReadF8 {
  const uint8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  const int32_t *seq_lens, *start;
  void *k_out, *v_out;  // [B, Hkv, N, D]
  uint32_t *status;
  int B, Hkv, N, Smax, NB, block_log2;
};
cudaError_t launch_read_f8(size_t elem_bytes, int D, const ReadF8 &p, cudaStream_t stream);

// Per-row int8 quantisation (codes + fp32 scales) of `rows` rows of D elements.
cudaError_t launch_quantize_q8(size_t elem_bytes, const void *x, long long rows, int D, int8_t *codes, float *scales,
                               cudaStream_t stream);
// Quantises new rows [B, Hkv, T, D] into an int8 cache at seq_lens (td_kv_append's rules).
cudaError_t launch_append_q8(size_t elem_bytes, const void *k_new, const void *v_new, int8_t *k_codes,
                             float *k_scales, int8_t *v_codes, float *v_scales, int32_t *seq_lens, int B, int Hkv,
                             int T, int Smax, int D, int advance, uint32_t *dev_status, cudaStream_t stream);

cudaError_t launch_split(td_dtype dtype, int D, const SplitPlan &plan, const SplitParams &p, cudaStream_t stream);

cudaError_t launch_merge(const float *m, const float *l, const float *acc, const int32_t *seq_lens, int B, int rows,
                         int NS, int D, int split, td_dtype out_dtype, void *out, float *lse, cudaStream_t stream);

cudaError_t launch_append(size_t elem_bytes, const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                          int32_t *seq_lens, int B, int Hkv, int T, int Smax, int D, int advance,
                          uint32_t *dev_status, cudaStream_t stream);

cudaError_t launch_rope_append(size_t elem_bytes, const void *q, void *q_out, int Hq, const void *k_new,
                               const void *v_new, const float *cos_t, const float *sin_t, void *k_cache,
                               void *v_cache, int32_t *seq_lens, int B, int Hkv, int T, int Smax, int D, int advance,
                               uint32_t *dev_status, cudaStream_t stream);

// Speculative accept/reject: most draft tokens per step, and the launch.
constexpr int kMaxDraft = 16;
constexpr int kMaxCluster = 16;  // CTAs per cluster, at most
int spec_slices(int V);
size_t spec_workspace_bytes(int B, int G, int V);
cudaError_t launch_spec_accept(const float *target, const float *draft, const int32_t *tokens, const float *uniforms,
                               int B, int G, int V, float temperature, int32_t *n_out, int32_t *tok_out,
                               uint32_t *status, void *workspace, cudaStream_t stream);

// Tiled causal prefill attention on the tensor cores (tcgen05); bf16, D 64 or 128. window > 0: over a window with
// so many sinks.
cudaError_t launch_prefill(const void *q, const void *k, const void *v, const int32_t *seq_lens, int B, int Hq, int Hkv,
                           int T, int Smax, int D, float scale, void *out, float *lse, uint32_t *status,
                           cudaStream_t stream, int window = 0, int sinks = 0);

// Attention in runs (td_runs.cuh): the warps that take them leave partial blocks, the join's launch reads them.
struct RunsPlan {
  int R, RB;      // rows of a row block, row blocks of a kv head
  int grid;
  size_t bytes;   // workspace: the blocks (nothing of it needs zeroing)
};
// keys: the most a sequence attends.
td_status plan_attn_runs(int B, int Hq, int Hkv, int T, int keys, int D, RunsPlan *plan);
// The parts over a shared prefix that the join adds (td_prefix.cu).
struct PrefixPart {
  const float *part;
  const int32_t *prefix_len;
  int Pmax, tiles, chunks;
  int grid;  // CTAs whose warps took the runs
};
cudaError_t launch_join(int D, const RunsPlan &plan, const SplitParams &p, const unsigned char *ws, const PrefixPart &x,
                        cudaStream_t stream);

// Attention over a shared prefix and each sequence's own keys (td_prefix.cu).
struct PrefixPlan {
  RunsPlan own;      // over the sequences' own keys
  int tiles, chunks; // 128-row tiles of a kv head, chunks of the prefix
  int grid;
  size_t off_part, bytes;  // workspace: own's, the prefix's partial blocks
};
struct PrefixAttn {
  const void *k, *v;  // [Hkv, Pmax, D]
  const int32_t *prefix_len;
  int Pmax;
};
td_status plan_prefix(int B, int Hq, int Hkv, int T, int Pmax, int Smax, int D, PrefixPlan *plan);
// p: queries, own keys, results.
cudaError_t launch_prefix(int D, const PrefixPlan &plan, const PrefixAttn &x, const SplitParams &p, unsigned char *ws,
                          cudaStream_t stream);

// SM count of the current device (cached per device).
int device_sm_count(int device);

// Launches `kernel` with programmatic dependent launch allowed: its CTAs may be scheduled
// while the previous kernel in the stream drains; every td kernel starts with a
// griddepcontrol.wait, so it still sees all of that kernel's writes.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// One kernel's opt-in to more than 48 KB of dynamic shared memory, made once per device (static at its launch).
class OptIn {
 public:
  cudaError_t operator()(const void *fn, int smem) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[device]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    done_[device] = e == cudaSuccess;
    return e;
  }

 private:
  static constexpr int kMaxDevices = 64;
  std::mutex mu_;
  bool done_[kMaxDevices] = {};
};

}  // namespace td
