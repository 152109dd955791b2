// Attention of a batch whose sequences share a long prefix: its keys and values are read once for all of them.
//
// The row (b, hq, t) attends the prefix's P keys and its sequence's own keys j < L_b - T + t + 1. Softmax sums over
// disjoint key sets join exactly: with (m, l, acc) a part's maximum, sum of 2^(s - m) and sum of 2^(s - m) v,
//   M = max m,  out = sum 2^(m - M) acc / sum 2^(m - M) l,  lse = M + log2 sum 2^(m - M) l   (base 2).
// Three launches, each started while the one before still runs:
//  A. prefix_kernel: of one kv head, the rows of all sequences (B x heads of the group x T tokens) form the M side of
//     tensor-core tiles (tcgen05, 128 rows), so each K/V tile of the prefix serves 128 rows; the prefix is cut into as
//     many chunks as fill the GPU once. Where one sequence at a time reads P keys for G x T rows, this reads them once
//     per 128 rows, and several tiles of rows take the same chunk at the same time, from L2.
//  B. the split kernels over each sequence's own keys (their PART instantiations: fp32 results, alongside A).
//  C. merge_prefix_kernel: joins a row's parts, rounds once.
// A is bound by the tensor cores and the exponentials where many sequences share the prefix, by memory where few do; B
// by memory. A takes one CTA per SM, so that B's CTAs share the SMs with it.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "td_internal.h"
#include "td_split_attn.cuh"
#include "td_split_cluster.cuh"
#include "td_split_mma.cuh"
#include "td_tc.cuh"

namespace td {

namespace {

constexpr int kPxSoftmaxWarps = 4;             // one query row per thread
constexpr int kPxMmaWarp = kPxSoftmaxWarps;    // issues the tensor-core products
constexpr int kPxLoadWarp = kPxSoftmaxWarps + 1;  // issues the TMA copies
constexpr int kPxThreads = 32 * (kPxSoftmaxWarps + 2);
constexpr int kPxRows = 128;                   // query rows per CTA
constexpr int kPxQRegion = kPxRows * 128;      // bytes of one swizzled [128 rows][64 bf16] region
constexpr int kPxKRegion = kPfKeys * 128;      // bytes of one swizzled [64 keys][64 bf16] region
constexpr int kMaxDevices = 64;

template <int D>
struct PxCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int Q_TILE = HALVES * kPxQRegion;
  static constexpr int KV_TILE = HALVES * kPxKRegion;
  static constexpr int K_OFF = Q_TILE;                // two K buffers
  static constexpr int V_OFF = K_OFF + 2 * KV_TILE;   // two V buffers
  static constexpr int SMEM = V_OFF + 2 * KV_TILE + 1024;  // + alignment slack
  static constexpr int TMEM_COLS = 256;               // S (64), two P buffers (32 each), O (D)
};

struct PxArgs {
  CUtensorMap kmap;  // prefix [Hkv][Pmax][D], boxes of 64 rows
  CUtensorMap vmap;
  const void *q;     // [B, Hq, T, D]
  const int32_t *prefix_len;
  float *part;       // [Hkv][tiles][chunks] blocks of part_floats(D)
  uint32_t *status;
  int B, Hq, Hkv, T, GT, Pmax;
  int tiles;         // 128-row tiles of a kv head's B * GT rows
  int chunks;        // chunks the prefix is cut into, at most
  float qscale;      // scale * log2(e)
};

// A chunk's partial block: acc [D / 4][128 rows][4], then m [128] (base 2) and l [128].
__host__ __device__ constexpr int part_floats(int D) { return kPxRows * (D + 2); }

// Prefix length attended, and the keys of a chunk (whole tiles).
__device__ __forceinline__ int prefix_keys(int raw, int Pmax) { return raw < 0 ? 0 : raw > Pmax ? Pmax : raw; }
__device__ __forceinline__ int prefix_chunk(int P, int chunks) {
  const int tiles = (P + kPfKeys - 1) / kPfKeys;
  return (tiles + chunks - 1) / chunks * kPfKeys;
}

template <int D>
__global__ void __launch_bounds__(kPxThreads, 2) prefix_kernel(const __grid_constant__ PxArgs a) {
  using C = PxCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bar_q, bar_k[2], bar_v[2], bar_s[2], bar_sfree, bar_p[2], bar_vfree[2], bar_o,
      bar_fin;
  __shared__ uint32_t s_taddr;
  __shared__ int s_issued[2], s_seen[2];  // wind-down: K / V tiles issued, and seen landed
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  // the tiles of rows that read one chunk are neighbours in the grid
  const int tile = blockIdx.x % a.tiles, kvh = blockIdx.x / a.tiles % a.Hkv, chunk = blockIdx.x / a.tiles / a.Hkv;

  if (tid == 0) {
    mbar_init(smem_u32(&bar_q), kPxSoftmaxWarps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_k[i]), 1);
      mbar_init(smem_u32(&bar_v[i]), 1);
      mbar_init(smem_u32(&bar_s[i]), 1);
      mbar_init(smem_u32(&bar_p[i]), kPxSoftmaxWarps);
      mbar_init(smem_u32(&bar_vfree[i]), 1);
    }
    s_issued[0] = s_issued[1] = 0;
    s_seen[0] = s_seen[1] = 0;
    mbar_init(smem_u32(&bar_sfree), kPxSoftmaxWarps);
    mbar_init(smem_u32(&bar_o), 1);
    mbar_init(smem_u32(&bar_fin), 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_taddr)),
                 "n"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_taddr;
  const uint32_t tS = tmem, tP = tmem + kPfKeys, tO = tmem + 128;

  griddep_wait();
  griddep_launch_dependents();
  const int raw = *a.prefix_len;
  const int P = prefix_keys(raw, a.Pmax);
  if (tid == 0 && blockIdx.x == 0)
    report(a.status, (raw < 0 ? TD_DEV_NEGATIVE_SEQLEN : 0u) | (raw > a.Pmax ? TD_DEV_SEQLEN_CLAMPED : 0u));
  const int S = prefix_chunk(P, a.chunks);
  const int c0 = min(chunk * S, P), c1 = min(c0 + S, P);
  const int nkt = (c1 - c0 + kPfKeys - 1) / kPfKeys;
  const int rows = min(kPxRows, a.B * a.GT - tile * kPxRows);  // rows of this tile that exist
  const float qscale = a.qscale;
  bool ok = true;
  int kq = 0, kw = 0, vq = 0, vw = 0;
  float m_ref = -INFINITY, l = 0.f;  // softmax threads: this row's reference maximum and sum

  if (warp == kPxMmaWarp) {
    if (lane == 0 && nkt > 0) {
      constexpr uint32_t kIdS = mma_idesc(kPxRows, kPfKeys, false);
      constexpr uint32_t kIdO = mma_idesc(kPxRows, D, true);
      const uint64_t dq = smem_desc(sb, 16, 1024);
      const uint64_t dk = smem_desc(sb + C::K_OFF, 16, 1024);
      const uint64_t dv = smem_desc(sb + C::V_OFF, kPxKRegion, 1024);
      auto issue_s = [&](int kt) {
        const uint32_t kb = (uint32_t)(kt & 1) * C::KV_TILE;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)(k & 3) * 32;
          tc_mma(tS, dq + (((uint32_t)(k >> 2) * kPxQRegion + off) >> 4),
                 dk + ((kb + (uint32_t)(k >> 2) * kPxKRegion + off) >> 4), kIdS, k > 0);
        }
        tc_commit(smem_u32(&bar_s[kt & 1]));
      };
      ok = mbar_wait_bounded(smem_u32(&bar_q), 0) && mbar_wait_bounded(smem_u32(&bar_k[0]), 0);
      if (ok) {
        kw = 1;
        issue_s(0);
      }
      for (int kt = 0; ok && kt < nkt; ++kt) {
        const int b0 = kt & 1, b1 = b0 ^ 1;
        if (kt + 1 < nkt) {
          ok = mbar_wait_bounded(smem_u32(&bar_sfree), (uint32_t)kt & 1u);
          ok = ok && mbar_wait_bounded(smem_u32(&bar_k[b1]), (uint32_t)((kt + 1) >> 1) & 1u);
          if (!ok) break;
          kw = kt + 2;
          issue_s(kt + 1);
        }
        ok = mbar_wait_bounded(smem_u32(&bar_p[b0]), (uint32_t)(kt >> 1) & 1u) &&
             mbar_wait_bounded(smem_u32(&bar_v[b0]), (uint32_t)(kt >> 1) & 1u);
        if (!ok) break;
        vw = kt + 1;
        tc_fence_after();
        const uint32_t vb = (uint32_t)b0 * C::KV_TILE;
#pragma unroll
        for (int k = 0; k < kPfKeys / 16; ++k)
          tc_mma_ts(tO, tP + b0 * (kPfKeys / 2) + 8 * k, dv + ((vb + (uint32_t)k * 16 * 128) >> 4), kIdO, kt > 0 || k > 0);
        tc_commit(smem_u32(&bar_o));
        tc_commit(smem_u32(&bar_vfree[b0]));
      }
      s_seen[0] = kw;
      s_seen[1] = vw;
    }
    __syncwarp();
  } else if (warp == kPxLoadWarp) {
    if (lane == 0 && nkt > 0) {
      auto load = [&](bool v, int kt) {
        const int buf = kt & 1;
        const uint32_t bar = smem_u32(v ? &bar_v[buf] : &bar_k[buf]);
        const uint32_t dst = sb + (v ? C::V_OFF : C::K_OFF) + buf * C::KV_TILE;
        mbar_arrive_expect_tx(bar, C::KV_TILE);
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h)
          tma3(dst + h * kPxKRegion, v ? &a.vmap : &a.kmap, 64 * h, c0 + kt * kPfKeys, kvh, bar);
      };
      for (; kq < min(nkt, 2); ++kq) {
        load(false, kq);
        load(true, kq);
      }
      vq = kq;
      for (int j = 2; ok && j < nkt; ++j) {
        const uint32_t ph = (uint32_t)((j - 2) >> 1) & 1u;
        ok = mbar_wait_bounded(smem_u32(&bar_s[j & 1]), ph);
        if (!ok) break;
        load(false, kq++);
        ok = mbar_wait_bounded(smem_u32(&bar_vfree[j & 1]), ph);
        if (!ok) break;
        load(true, vq++);
      }
      s_issued[0] = kq;
      s_issued[1] = vq;
    }
    __syncwarp();
  } else if (nkt > 0) {
    // the tile's query rows, each 16-byte chunk to its place in the swizzled tile (rows that do not exist: zeros)
    for (int idx = tid; idx < kPxRows * (D / 8); idx += 32 * kPxSoftmaxWarps) {
      const int r = idx / (D / 8), c = idx % (D / 8);
      const bool real = r < rows;
      const int row = real ? tile * kPxRows + r : 0;
      const long long at = (long long)(row / a.GT) * a.Hq * a.T + (long long)kvh * a.GT + row % a.GT;
      cp_async_16(sb + tile_chunk(kPxRows, r, c), static_cast<const uint4 *>(a.q) + at * (D / 8) + c, real ? 16u : 0u);
    }
    cp_async_commit();
    cp_async_wait<0>();
    fence_proxy_async_smem();  // read next by the tensor core (asynchronous proxy)
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar_q));
    const int busy = (rows + 31) / 32;  // warps with rows
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    // a warp without rows only keeps the barriers' count: what its lanes of P and O hold reaches no other row
    for (int kt = 0; kt < nkt && warp >= busy; ++kt) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_s[kt & 1]), (uint32_t)(kt >> 1) & 1u))) {
        ok = false;
        break;
      }
      if (lane == 0) {
        mbar_arrive(smem_u32(&bar_sfree));
        mbar_arrive(smem_u32(&bar_p[kt & 1]));
      }
    }
    for (int kt = 0; kt < nkt && warp < busy; ++kt) {
      const int b0 = kt & 1;
      const uint32_t ph = (uint32_t)(kt >> 1) & 1u;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_s[b0]), ph))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int vis = min(kPfKeys, c1 - c0 - kt * kPfKeys);  // keys of the tile (fewer at the prefix's end alone)
      if (vis < kPfKeys) {
        // V rows behind the prefix, once landed: zeroed (a masked p of 0 must not meet a stale value)
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_v[b0]), ph))) {
          ok = false;
          break;
        }
        unsigned char *vt = smem + C::V_OFF + b0 * C::KV_TILE;
        for (int idx = tid; idx < (kPfKeys - vis) * (D / 8); idx += 32 * busy) {
          const int r = vis + idx / (D / 8), c = idx % (D / 8);
          *reinterpret_cast<uint4 *>(vt + tile_chunk(kPfKeys, r, c)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      float sv[kPfKeys];
      tmem_ld64(tS + lane_base, sv);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_sfree));
      if (vis < kPfKeys) {
#pragma unroll
        for (int i = 0; i < kPfKeys; ++i)
          if (i >= vis) sv[i] = qscale >= 0.f ? -INFINITY : INFINITY;
      }
      const float mx = (qscale >= 0.f ? row_extreme<false>(sv) : row_extreme<true>(sv)) * qscale;
      const bool move = mx > m_ref + kRescaleGap || (m_ref == -INFINITY && mx > -INFINITY);
      const float alpha = (move && m_ref != -INFINITY) ? exp2_approx(m_ref - mx) : 1.f;
      if (move) {
        l *= alpha;
        m_ref = mx;
      }
      if (kt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_o), (uint32_t)(kt - 1) & 1u))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tO + lane_base + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= alpha;
          tmem_st32(tO + lane_base + c, o);
        }
      }
      const float nbase = m_ref == -INFINITY ? 0.f : -m_ref;
      const SeenFirst seen{vis};
      uint32_t pk[kPfKeys / 2];
      if (vis == kPfKeys)
        l += p_row<false>(sv, qscale, nbase, seen, pk);
      else
        l += p_row<true>(sv, qscale, nbase, seen, pk);
      if (kt >= 2) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_vfree[b0]), (uint32_t)((kt - 2) >> 1) & 1u))) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      tmem_st32(tP + b0 * (kPfKeys / 2) + lane_base, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_p[b0]));
    }
    if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_o), (uint32_t)(nkt - 1) & 1u))) ok = false;
  }
  ok = __syncthreads_and(ok) != 0;
  if (!ok) {
    // before shared memory and TMEM are released: the products (one commit tracks them all) and the copies in flight
    if (tid == kPxMmaWarp * 32) {
      tc_commit(smem_u32(&bar_fin));
      mbar_wait_bounded(smem_u32(&bar_fin), 0);
    }
    if (tid == kPxLoadWarp * 32) {
      for (int kt = s_seen[0]; kt < s_issued[0]; ++kt)
        mbar_wait_bounded(smem_u32(&bar_k[kt & 1]), (uint32_t)(kt >> 1) & 1u);
      for (int kt = s_seen[1]; kt < s_issued[1]; ++kt)
        mbar_wait_bounded(smem_u32(&bar_v[kt & 1]), (uint32_t)(kt >> 1) & 1u);
      report(a.status, TD_DEV_WAIT_TIMEOUT);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp < kPxSoftmaxWarps && nkt > 0 && warp * 32 < rows) {
    // the partial block: 512 consecutive bytes a warp and store
    float *blk = a.part + (((long long)kvh * a.tiles + tile) * a.chunks + chunk) * part_floats(D);
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
#pragma unroll
    for (int c = 0; c < D; c += 32) {
      float o[32];
      tmem_ld32(tO + lane_base + c, o);
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<float4 *>(blk + ((c + i) / 4 * kPxRows + tid) * 4) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
    blk[kPxRows * D + tid] = m_ref;
    blk[kPxRows * (D + 1) + tid] = ok ? l : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::TMEM_COLS) : "memory");
}

struct MergeArgs {
  const float *part;      // prefix_kernel's blocks
  const float *own, *own_lse;  // [B, Hq, T, D] and [B, Hq, T] (natural log) of the sequences' own keys
  const int32_t *prefix_len;
  void *out;              // [B, Hq, T, D] bf16
  float *lse;             // [B, Hq, T] or null
  int B, Hq, Hkv, T, GT, Pmax, tiles, chunks;
};

// Joins the parts of 32 rows (one tile's), 32 dims: a lane a row, a warp four dims.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) merge_prefix_kernel(const MergeArgs a) {
  const int slab = blockIdx.x % (D / 32), group = blockIdx.x / (D / 32) % (a.tiles * 4), kvh = blockIdx.x / (D / 32) / (a.tiles * 4);
  const int tile = group / 4, lane = threadIdx.x & 31;
  const int r = group % 4 * 32 + lane, row = tile * kPxRows + r;
  const int d4 = slab * 8 + threadIdx.x / 32;
  griddep_wait();
  griddep_launch_dependents();
  if (row >= a.B * a.GT) return;
  const int P = prefix_keys(__ldcg(a.prefix_len), a.Pmax);
  const int S = prefix_chunk(P, a.chunks);
  const int nc = P > 0 ? (P + S - 1) / S : 0;
  const float *blk = a.part + ((long long)kvh * a.tiles + tile) * a.chunks * part_floats(D);
  const long long at = (long long)(row / a.GT) * a.Hq * a.T + (long long)kvh * a.GT + row % a.GT;
  const float own2 = __ldcg(a.own_lse + at) * kLog2e;
  float M = own2, L = own2 == -INFINITY ? 0.f : 1.f;
  float4 A = __ldcg(reinterpret_cast<const float4 *>(a.own + at * D) + d4);
  if (L == 0.f) A = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 8;  // chunks whose loads are in flight at once
  for (int c0 = 0; c0 < nc; c0 += kBatch) {
    float m[kBatch], l[kBatch];
    float4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float *pb = blk + (long long)(c0 + i) * part_floats(D);
      const bool in = c0 + i < nc;
      m[i] = in ? __ldcg(pb + kPxRows * D + r) : -INFINITY;
      l[i] = in ? __ldcg(pb + kPxRows * (D + 1) + r) : 0.f;
      x[i] = in ? __ldcg(reinterpret_cast<const float4 *>(pb) + d4 * kPxRows + r) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float Mn = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (l[i] > 0.f) Mn = fmaxf(Mn, m[i]);
    const float base = Mn == -INFINITY ? 0.f : Mn;
    const float alpha = exp2f(M - base);
    L *= alpha;
    A.x *= alpha, A.y *= alpha, A.z *= alpha, A.w *= alpha;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (l[i] > 0.f) {
        const float f = exp2f(m[i] - base);
        L = fmaf(l[i], f, L);
        A.x = fmaf(x[i].x, f, A.x), A.y = fmaf(x[i].y, f, A.y), A.z = fmaf(x[i].z, f, A.z), A.w = fmaf(x[i].w, f, A.w);
      }
    }
    M = Mn;
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at * D + d4 * 4) =
      make_uint2(pack_bf16x2(A.x * inv, A.y * inv), pack_bf16x2(A.z * inv, A.w * inv));
  if (a.lse != nullptr && d4 == 0) a.lse[at] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

template <int D>
cudaError_t opt_in() {
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[device]) return cudaSuccess;
  constexpr int persistent = MmaCfg<D, kPersistentStages<D>>::RING_BYTES + 1024;
  const struct {
    const void *fn;
    int smem;
    bool cluster;
  } all[] = {{reinterpret_cast<const void *>(&prefix_kernel<D>), PxCfg<D>::SMEM, false},
             {reinterpret_cast<const void *>(&split_attn_mma_kernel<D, false, kTileN8, 0, true>), persistent, false},
             {reinterpret_cast<const void *>(&split_attn_mma_kernel<D, false, kTileM16, 0, true>), persistent, false},
             {reinterpret_cast<const void *>(&split_attn_mma_kernel<D, false, kTileN24, 0, true>), persistent, false},
             {reinterpret_cast<const void *>(&split_attn_cluster_kernel<D, kTileN8, 0, true>), cluster_smem<D>(), true},
             {reinterpret_cast<const void *>(&split_attn_cluster_kernel<D, kTileM16, 0, true>), cluster_smem<D>(), true},
             {reinterpret_cast<const void *>(&split_attn_cluster_kernel<D, kTileN24, 0, true>), cluster_smem<D>(), true}};
  for (const auto &k : all) {
    cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e == cudaSuccess && k.cluster) e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  done[device] = true;
  return cudaSuccess;
}

// The split kernels over the sequences' own keys: fp32 out and lse (p.out, p.lse).
template <int D>
cudaError_t launch_own(const SplitPlan &plan, const SplitParams &p, cudaStream_t stream) {
  MmaArgs a;
  if (!encode_cache_map(&a.kmap, p.k, p.B, p.Hkv, p.Smax, D) || !encode_cache_map(&a.vmap, p.v, p.B, p.Hkv, p.Smax, D))
    return cudaErrorInvalidValue;
  a.p = p;
  const int tile = tile_of_rows(p.R);
  if (plan.cluster > 0) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(D, plan.grid, plan.cluster, stream, attr);
    if (tile == kTileN8) return cudaLaunchKernelEx(&cfg, split_attn_cluster_kernel<D, kTileN8, 0, true>, a);
    if (tile == kTileM16) return cudaLaunchKernelEx(&cfg, split_attn_cluster_kernel<D, kTileM16, 0, true>, a);
    return cudaLaunchKernelEx(&cfg, split_attn_cluster_kernel<D, kTileN24, 0, true>, a);
  }
  const dim3 grid(plan.grid), block(kThreads);
  if (tile == kTileN8) return launch_pdl(split_attn_mma_kernel<D, false, kTileN8, 0, true>, grid, block, plan.smem, stream, a);
  if (tile == kTileM16) return launch_pdl(split_attn_mma_kernel<D, false, kTileM16, 0, true>, grid, block, plan.smem, stream, a);
  return launch_pdl(split_attn_mma_kernel<D, false, kTileN24, 0, true>, grid, block, plan.smem, stream, a);
}

template <int D>
cudaError_t launch_d(const PrefixPlan &plan, const PrefixAttn &x, const SplitParams &own, cudaStream_t stream) {
  cudaError_t e = opt_in<D>();
  if (e != cudaSuccess) return e;
  PxArgs a;
  if (!encode_cache_map(&a.kmap, x.k, 1, own.Hkv, x.Pmax, D) || !encode_cache_map(&a.vmap, x.v, 1, own.Hkv, x.Pmax, D))
    return cudaErrorInvalidValue;
  a.q = own.q;
  a.prefix_len = x.prefix_len;
  a.part = x.part;
  a.status = own.status;
  a.B = own.B, a.Hq = own.Hq, a.Hkv = own.Hkv, a.T = own.T, a.GT = own.G * own.T, a.Pmax = x.Pmax;
  a.tiles = plan.tiles, a.chunks = plan.chunks;
  a.qscale = own.qscale;
  e = launch_pdl(prefix_kernel<D>, dim3((unsigned)(plan.tiles * own.Hkv * plan.chunks)), dim3(kPxThreads), PxCfg<D>::SMEM,
                 stream, a);
  if (e == cudaSuccess) e = launch_own<D>(plan.own, own, stream);
  if (e != cudaSuccess) return e;
  const MergeArgs m{x.part, static_cast<const float *>(own.out), own.lse, x.prefix_len, x.out, x.lse, own.B, own.Hq,
                    own.Hkv, own.T, a.GT, x.Pmax, plan.tiles, plan.chunks};
  return launch_pdl(merge_prefix_kernel<D>, dim3((unsigned)(own.Hkv * plan.tiles * 4 * (D / 32))), dim3(kJoinThreads), 0,
                    stream, m);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

#ifndef TD_PX_PER
#define TD_PX_PER 1
#endif
td_status plan_prefix(int B, int Hq, int Hkv, int T, int Pmax, int Smax, int D, PrefixPlan *plan) {
  const td_status st = plan_split(TD_BF16, B, Hq, Hkv, T, Smax, D, 0, &plan->own);
  if (st != TD_OK) return st;
  if (Pmax < 1) return TD_ERR_INVALID_ARG;
  if (Pmax > (1 << 30)) return TD_ERR_UNSUPPORTED;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return TD_ERR_CUDA;
  const long long rows = (long long)B * (Hq / Hkv) * T;
  const long long tiles = (rows + kPxRows - 1) / kPxRows;
  const long long groups = tiles * Hkv;
  // chunks that fill the GPU once, of at least two tiles of keys
  long long chunks = TD_PX_PER * (long long)device_sm_count(device) / groups;
  chunks = std::min(chunks, ((long long)Pmax + 2 * kPfKeys - 1) / (2 * kPfKeys));
  if (chunks < 1) chunks = 1;
  if (groups * chunks * 16 > 0x7fffffffLL || rows > (1 << 26)) return TD_ERR_UNSUPPORTED;
  plan->tiles = (int)tiles;
  plan->chunks = (int)chunks;
  const size_t out_rows = (size_t)B * Hq * T;
  plan->off_own = align256(plan->own.bytes);
  plan->off_lse = plan->off_own + align256(out_rows * D * sizeof(float));
  plan->off_part = plan->off_lse + align256(out_rows * sizeof(float));
  plan->bytes = plan->off_part + align256((size_t)(groups * chunks) * part_floats(D) * sizeof(float));
  return TD_OK;
}

cudaError_t launch_prefix(int D, const PrefixPlan &plan, const PrefixAttn &x, const SplitParams &own, cudaStream_t stream) {
  const cudaError_t e = D == 64 ? launch_d<64>(plan, x, own, stream) : launch_d<128>(plan, x, own, stream);
  if (e != cudaSuccess) cudaGetLastError();  // reported once, by this call
  return e;
}

}  // namespace td
