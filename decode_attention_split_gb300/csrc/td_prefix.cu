// Attention of a batch whose sequences share a long prefix: its keys and values are read once for all of them.
//
// The row (b, hq, t) attends the prefix's P keys and its sequence's own keys j < L_b - T + t + 1. Softmax sums over
// disjoint key sets join exactly: with (m, l, acc) a part's maximum, sum of 2^(s - m) and sum of 2^(s - m) v,
//   M = max m,  out = sum 2^(m - M) acc / sum 2^(m - M) l,  lse = M + log2 sum 2^(m - M) l   (base 2).
// Two launches. In prefix_kernel, one CTA an SM, three groups of warps work side by side:
//  * softmax warps and the warps that issue products and copies take tiles over the prefix: of one kv head, the rows of
//    all sequences (B x heads of the group x T tokens) form the M side of tensor-core products (tcgen05, 128 rows), so each
//    K/V tile of the prefix serves 128 rows. The prefix is cut into as many chunks as fill the GPU once. Where one sequence
//    at a time reads P keys for G x T rows, this reads them once per 128 rows;
//  * four warps take runs over each sequence's own keys (td_runs.cuh, mma.sync).
// The first is bound by the tensor cores and exponentials where many sequences share the prefix and by memory where few
// do, the second by memory: in one CTA they fill each other's waits, and neither waits for the other's launch.
// join_kernel then joins a row's parts and rounds once.
// Measured (GPU time in a graph, 128 dims): 64 sequences of up to 512 own keys behind 8192 (32 + 8 heads) 27.7 us (102 MB,
// 3.7 TB/s; either part alone 21 us), 16 of up to 1000 behind 32003 (24 + 8 heads) 33.2 us (168 MB, 5.1 TB/s), six tokens of
// 16 sequences behind 4321 24.5 us (48 MB). The fixed part, 7 us with 4 short sequences, is two launches, the lengths and
// queries, one tile, the partial blocks and the join.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "td_internal.h"
#include "td_runs.cuh"
#include "td_tc.cuh"

namespace td {

namespace {

constexpr int kPxSoftmaxWarps = 8;             // warps 0 .. 7: warps w and w + 4 share the rows of TMEM lanes 32 w ..
constexpr int kPxRunWarp = 8;                  // 8 .. 11: runs over the own keys
constexpr int kPxMmaWarp = 12;                 // issues the tensor-core products
constexpr int kPxLoadWarp = 13;                // issues the TMA copies
constexpr int kPxThreads = 512;                // four warpgroups (the last two warps have no work)
constexpr int kPxRows = kPrefixRows;           // query rows per tile
constexpr int kPxKeys = kPrefixKeys;           // keys per tile
constexpr int kPxHalf = kPxKeys / 2;           // of them, one softmax thread's
constexpr int kPxKRegion = kPxKeys * 128;      // bytes of one swizzled [128 keys][64 bf16] region
// The reference of a row moves to kRescaleLead above its maximum: without that lead, and now and then a key of four times
// the others' strength, some row of the 128 moved in nearly every tile (490 cycles of a tile's 3600, 175 with it; a call of 16
// sequences behind 32003 keys 34.1 -> 33.8 us, six tokens of 16 behind 4321 25.2 -> 24.9).
// Registers a thread: launched with 128 (65536 / 512), then split between softmax, run, and product and copy warps. A run
// over row blocks of more than 16 rows needs more than 200, and the softmax warps then keep to what they have.
__host__ __device__ constexpr int px_soft_regs(int NT) { return NT <= 2 ? 136 : 128; }
__host__ __device__ constexpr int px_run_regs(int NT) { return NT <= 2 ? 200 : 216; }
constexpr int kPxIssueRegs = 40;
static_assert(256 * px_soft_regs(1) + 128 * px_run_regs(1) + 128 * kPxIssueRegs <= 512 * 128 &&
                  256 * px_soft_regs(3) + 128 * px_run_regs(3) + 128 * kPxIssueRegs <= 512 * 128,
              "register split within the launch's");

template <int D>
struct PxCfg {
  static constexpr int NST = D == 128 ? 2 : 4;  // buffers of K, and of V
  static constexpr int HALVES = D / 64;
  static constexpr int KV_TILE = HALVES * kPxKRegion;
  static constexpr int V_OFF = NST * KV_TILE;         // the K buffers come first
  static constexpr int RUN_OFF = V_OFF + NST * KV_TILE;  // then the rings of the run warps
  using Run = RunCfg<D, 2>;
  static constexpr int LEN_OFF = RUN_OFF + kRunWarps * Run::RING;  // then two ints a sequence and one
  static constexpr int SMEM = LEN_OFF + 1024;         // + alignment slack
  static constexpr int O_COL = 256, Q_COL = O_COL + D;  // columns: S (128), two P buffers (64 each), O (D), Q (D / 2)
  static constexpr int TMEM_COLS = 512;
  static_assert(SMEM + (2 * TD_MAX_BATCH + 1) * 4 + 1024 <= 227 * 1024, "shared memory");
};

struct PxArgs {
  RunArgs own;       // the sequences' own keys; its p holds the queries too
  CUtensorMap kmap;  // prefix [Hkv][Pmax][D], boxes of 128 rows
  CUtensorMap vmap;
  const int32_t *prefix_len;
  float *part;       // [Hkv][tiles][chunks] blocks of prefix_block_floats(D) (td_runs.cuh)
  int GT, Pmax;
  int tiles;         // 128-row tiles of a kv head's B * GT rows
  int chunks;        // chunks the prefix is cut into, at most
};

// A tile's work: a kv head's rows [tile * 128, + rows) over keys [c0, c0 + 128 nkt), the last tile cut at c1.
struct PxItem {
  int tile, kvh, chunk, rows, c0, c1, nkt;
};
__device__ __forceinline__ PxItem px_item(const PxArgs &a, int item, int P) {
  PxItem w;
  const PrefixItem at = prefix_item(item, a.tiles, a.own.p.Hkv);
  w.tile = at.tile, w.kvh = at.kvh, w.chunk = at.chunk;
  w.rows = min(kPxRows, a.own.p.B * a.GT - w.tile * kPxRows);
  const int S = prefix_chunk(P, a.chunks);
  w.c0 = min(w.chunk * S, P);
  w.c1 = min(w.c0 + S, P);
  w.nkt = (w.c1 - w.c0 + kPxKeys - 1) / kPxKeys;
  return w;
}

// NT: 8-row tiles of a run's row block. Buffers and barriers go round over all of a CTA's key tiles: tile g (counted over
// its items) uses K / V buffer g % NST and S and P buffers g % 2.
template <int D, int NT>
__global__ void __launch_bounds__(kPxThreads, 1) prefix_kernel(const __grid_constant__ PxArgs a) {
  using C = PxCfg<D>;
  const SplitParams &p = a.own.p;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bar_q, bar_k[C::NST], bar_v[C::NST], bar_s[2], bar_sfree, bar_p[2], bar_kfree[C::NST],
      bar_vfree[C::NST], bar_pfree[2], bar_fin, run_bars[kRunWarps][C::Run::STAGES];
  __shared__ uint32_t s_taddr;
  __shared__ int s_issued[2], s_seen[2];  // wind-down: K / V tiles issued, and seen landed
  __shared__ int s_red[kRunWarps];
  __shared__ float s_max[2][2][kPxRows];  // by tile's parity and half: a row's maximum over the half's keys, then its sum
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);

  if (tid == 0) {
    mbar_init(smem_u32(&bar_q), kPxSoftmaxWarps);
#pragma unroll
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(smem_u32(&bar_k[i]), 1);
      mbar_init(smem_u32(&bar_v[i]), 1);
      mbar_init(smem_u32(&bar_kfree[i]), 1);
      mbar_init(smem_u32(&bar_vfree[i]), 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_s[i]), 1);
      mbar_init(smem_u32(&bar_p[i]), kPxSoftmaxWarps);
      mbar_init(smem_u32(&bar_pfree[i]), 1);
    }
    s_issued[0] = s_issued[1] = 0;
    s_seen[0] = s_seen[1] = 0;
    mbar_init(smem_u32(&bar_sfree), kPxSoftmaxWarps);
    mbar_init(smem_u32(&bar_fin), 1);
    fence_mbar_init();
  }
  if (warp >= kPxRunWarp && warp < kPxRunWarp + kRunWarps && lane == 0) init_ring<C::Run::STAGES>(run_bars[warp - kPxRunWarp]);
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
  const uint32_t tS = tmem, tP = tmem + kPxKeys, tO = tmem + C::O_COL, tQ = tmem + C::Q_COL;

  bool ok = true;
  if (warp >= kPxRunWarp && warp < kPxRunWarp + kRunWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(px_run_regs(NT)));
    int *s_len = reinterpret_cast<int *>(smem + C::LEN_OFF);  // [B]
    int *s_prefix = s_len + p.B;                              // [B + 1]
    const int rt = tid - 32 * kPxRunWarp, rw = warp - kPxRunWarp, run = blockIdx.x * kRunWarps + rw;
    // planned on the lengths as they read ahead of the wait for the launches before, and again should they read otherwise
    // after it
    RunCursor start;
    int u1;
#pragma unroll 1
    for (bool waited = false;;) {
      const int S = plan_runs<1>(p, rt, s_len, s_prefix, s_red);
      start = run_start(p, s_len, s_prefix, S, run, u1);
      if (waited) break;
      griddep_wait();
      griddep_launch_dependents();
      waited = true;
      if (lens_stand<1>(p, rt, s_len)) break;
    }
    run_warp<D, NT, 2>(p, a.own.kmap, a.own.vmap, s_len, start, u1, run, smem + C::RUN_OFF + rw * C::Run::RING,
                       run_bars[rw]);
  } else if (warp >= kPxMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPxIssueRegs));
    griddep_wait();
    griddep_launch_dependents();
    const int P = prefix_keys(*a.prefix_len, a.Pmax);
    const int items = P > 0 ? a.tiles * p.Hkv * a.chunks : 0;
    if (warp == kPxMmaWarp) {
      if (lane == 0) {
        constexpr uint32_t kIdS = mma_idesc(kPxRows, kPxKeys, false);
        constexpr uint32_t kIdO = mma_idesc(kPxRows, D, true);
        const uint64_t dk = smem_desc(sb, 16, 1024);
        const uint64_t dv = smem_desc(sb + C::V_OFF, kPxKRegion, 1024);
        int kw = 0, vw = 0;  // K and V tiles seen landed
        // S of tile g into the S columns, once every softmax warp has read the S before it and K has landed
        auto issue_s = [&](int g) {
          ok = (g == 0 || mbar_wait_bounded(smem_u32(&bar_sfree), (uint32_t)(g - 1) & 1u)) &&
               mbar_wait_bounded(smem_u32(&bar_k[g % C::NST]), (uint32_t)(g / C::NST) & 1u);
          if (!ok) return;
          kw = g + 1;
          const uint32_t kb = (uint32_t)(g % C::NST) * C::KV_TILE;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (uint32_t)(k & 3) * 32;
            tc_mma_ts(tS, tQ + 8 * k, dk + ((kb + (uint32_t)(k >> 2) * kPxKRegion + off) >> 4), kIdS, k > 0);
          }
          tc_commit(smem_u32(&bar_s[g & 1]));
          tc_commit(smem_u32(&bar_kfree[g % C::NST]));
        };
        int g = 0, it = 0;
        for (int item = blockIdx.x; ok && item < items; item += gridDim.x, ++it) {
          const PxItem w = px_item(a, item, P);
          if (w.nkt == 0) break;  // later items are of the same or a later chunk
          ok = mbar_wait_bounded(smem_u32(&bar_q), (uint32_t)it & 1u);
          if (ok) issue_s(g);
          for (int kt = 0; ok && kt < w.nkt; ++kt, ++g) {
            const int b0 = g & 1, buf = g % C::NST;
            if (kt + 1 < w.nkt) issue_s(g + 1);
            // O += P V once the softmax warps have left P of g and V has landed
            ok = ok && mbar_wait_bounded(smem_u32(&bar_p[b0]), (uint32_t)(g >> 1) & 1u) &&
                 mbar_wait_bounded(smem_u32(&bar_v[buf]), (uint32_t)(g / C::NST) & 1u);
            if (!ok) break;
            vw = g + 1;
            tc_fence_after();
            const uint32_t vb = (uint32_t)buf * C::KV_TILE;
#pragma unroll
            for (int k = 0; k < kPxKeys / 16; ++k)
              tc_mma_ts(tO, tP + b0 * (kPxKeys / 2) + 8 * k, dv + ((vb + (uint32_t)k * 16 * 128) >> 4), kIdO,
                        kt > 0 || k > 0);
            tc_commit(smem_u32(&bar_pfree[b0]));
            tc_commit(smem_u32(&bar_vfree[buf]));
          }
        }
        s_seen[0] = kw;
        s_seen[1] = vw;
      }
      __syncwarp();
    } else if (warp == kPxLoadWarp) {
      if (lane == 0) {
        const uint64_t policy = l2_evict_first_policy();
        int g = 0;
        for (int item = blockIdx.x; ok && item < items; item += gridDim.x) {
          const PxItem w = px_item(a, item, P);
          if (w.nkt == 0) break;
          for (int kt = 0; kt < w.nkt; ++kt, ++g) {
            const int buf = g % C::NST;
            const uint32_t ph = (uint32_t)(g / C::NST - 1) & 1u;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              // each buffer once the product that read its previous tile is complete
              ok = g < C::NST || mbar_wait_bounded(smem_u32(v ? &bar_vfree[buf] : &bar_kfree[buf]), ph);
              if (!ok) break;
              const uint32_t bar = smem_u32(v ? &bar_v[buf] : &bar_k[buf]);
              const uint32_t dst = sb + (v ? C::V_OFF : 0) + buf * C::KV_TILE;
              mbar_arrive_expect_tx(bar, C::KV_TILE);
#pragma unroll
              for (int h = 0; h < C::HALVES; ++h)
                tma_load_3d(dst + h * kPxKRegion, v ? &a.vmap : &a.kmap, 64 * h, w.c0 + kt * kPxKeys, w.kvh, bar, policy);
              s_issued[v] = g + 1;
            }
            if (!ok) break;
          }
        }
      }
      __syncwarp();
    }
  } else {
    if constexpr (px_soft_regs(NT) > 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(px_soft_regs(NT)));
    griddep_wait();
    griddep_launch_dependents();
    // thread `row` of half `half` (0: warps 0 .. 3) takes keys 64 half .. of the row's 128 a tile, and dims D / 2 half ..
    // of its output; the two of a row meet in s_max
    const int quarter = warp & 3, half = warp >> 2, row = tid & (kPxRows - 1);
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const float qscale = p.qscale;
    const int nrows = p.B * a.GT;
    auto meet = [&]() {  // the two warps of a quarter's rows
      asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory");
    };
    // this thread's half of its query row, asked for ahead of the prefix's length (past the last item: a row in vain)
    uint4 qv[D / 16];
    auto fetch_q = [&](int item) {
      const int at = item % a.tiles * kPxRows + row, kvh = item / a.tiles % p.Hkv;
      const bool real = at < nrows;
      const uint4 *qrow = static_cast<const uint4 *>(p.q) + half * (D / 16) +
                          (real ? (long long)(at / a.GT) * p.Hq * p.T + (long long)kvh * a.GT + at % a.GT : 0) * (D / 8);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) qv[i] = real ? qrow[i] : make_uint4(0u, 0u, 0u, 0u);
    };
    fetch_q(blockIdx.x);
    const int raw = *a.prefix_len;
    const int P = prefix_keys(raw, a.Pmax);
    if (tid == 0 && blockIdx.x == 0)
      report(p.status, (raw < 0 ? TD_DEV_NEGATIVE_SEQLEN : 0u) | (raw > a.Pmax ? TD_DEV_SEQLEN_CLAMPED : 0u));
    const int items = P > 0 ? a.tiles * p.Hkv * a.chunks : 0;
    int g = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x, fetch_q(item)) {
      const PxItem w = px_item(a, item, P);
      if (w.nkt == 0) break;
      const int busy = (w.rows + 31) / 32;  // quarters with rows
      // the query row into its TMEM lane, a column per pair of dims (rows that do not exist: zeros)
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint32_t x[16] = {qv[4 * c].x,     qv[4 * c].y,     qv[4 * c].z,     qv[4 * c].w,
                                qv[4 * c + 1].x, qv[4 * c + 1].y, qv[4 * c + 1].z, qv[4 * c + 1].w,
                                qv[4 * c + 2].x, qv[4 * c + 2].y, qv[4 * c + 2].z, qv[4 * c + 2].w,
                                qv[4 * c + 3].x, qv[4 * c + 3].y, qv[4 * c + 3].z, qv[4 * c + 3].w};
        tmem_st16(tQ + lane_base + half * (D / 4) + 16 * c, x);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(smem_u32(&bar_q));
      // a warp without rows only keeps the barriers' count: what its lanes of P and O hold reaches no other row
      const int g0 = g;
      g += w.nkt;
      for (int k = g0; ok && k < g && quarter >= busy; ++k) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_s[k & 1]), (uint32_t)(k >> 1) & 1u));
        if (ok && lane == 0) {
          mbar_arrive(smem_u32(&bar_sfree));
          mbar_arrive(smem_u32(&bar_p[k & 1]));
        }
      }
      if (quarter >= busy) continue;
      // (a warp whose wait gave up takes part in nothing but the meetings from then on, which the other warp counts on)
      float m_ref = -INFINITY, l = 0.f;  // this row's reference maximum, and its sum over this thread's keys
      for (int k = g0; k < g; ++k) {
        const int b0 = k & 1;
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_s[b0]), (uint32_t)(k >> 1) & 1u));
        tc_fence_after();
        // keys of the tile (fewer at the prefix's end alone), and of this half of it
        const int left = w.c1 - w.c0 - (k - g0) * kPxKeys, vis = min(kPxHalf, left - half * kPxHalf);
        if (ok && left < kPxKeys) {
          // V rows behind the prefix, once landed: zeroed (a masked p of 0 must not meet a stale value)
          const int buf = k % C::NST;
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_v[buf]), (uint32_t)(k / C::NST) & 1u));
          unsigned char *vt = smem + C::V_OFF + buf * C::KV_TILE;
          for (int idx = 32 * (quarter + half * busy) + lane; ok && idx < (kPxKeys - left) * (D / 8); idx += 64 * busy) {
            const int r = left + idx / (D / 8), c = idx % (D / 8);
            *reinterpret_cast<uint4 *>(vt + tile_chunk(kPxKeys, r, c)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // read next by the tensor core (asynchronous proxy)
        }
        float sv[kPxHalf];
        float mx = -INFINITY;
        if (ok) {
          tmem_ld64(tS + lane_base + half * kPxHalf, sv);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_sfree));
          if (left < kPxKeys) {
#pragma unroll
            for (int i = 0; i < kPxHalf; ++i)
              if (i >= vis) sv[i] = qscale >= 0.f ? -INFINITY : INFINITY;
          }
          if (vis > 0) mx = (qscale >= 0.f ? row_extreme<false>(sv) : row_extreme<true>(sv)) * qscale;
        }
        // the row's maximum over both halves
        s_max[b0][half][row] = mx;
        meet();
        mx = fmaxf(mx, s_max[b0][half ^ 1][row]);
        if (!ok) continue;
        // the reference moves only when the row's maximum rises more than kRescaleGap above it (a row's first scores
        // always move it); only then are O and l rescaled, once the previous product is complete
        const bool move = mx > m_ref + kRescaleGap || (m_ref == -INFINITY && mx > -INFINITY);
        const float m_new = mx + kRescaleLead;
        const float alpha = (move && m_ref != -INFINITY) ? exp2_approx(m_ref - m_new) : 1.f;
        if (move) {
          l *= alpha;
          m_ref = m_new;
        }
        if (k > g0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          // (the product of k - 2 may still run: S of k is issued before the product of k - 1. Each of the two barriers'
          // phase before is known complete, so neither wait can pass a phase early)
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_pfree[b0 ^ 1]), (uint32_t)((k - 1) >> 1) & 1u));
          if (!ok) continue;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 16) {  // (16 at a time: the scores are held meanwhile)
            uint32_t o[16];
            tmem_ld16(tO + lane_base + half * (D / 2) + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(tO + lane_base + half * (D / 2) + c, o);
          }
        }
        const float nbase = m_ref == -INFINITY ? 0.f : -m_ref;
        // P of this half into P buffer b0, once the product of tile k - 2 has read it
        if (k >= 2) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_pfree[b0]), (uint32_t)((k - 2) >> 1) & 1u));
          if (!ok) continue;
          tc_fence_after();
        }
#pragma unroll
        for (int c = 0; c < kPxHalf; c += 32) {
          const SeenFirst seen{vis - c};
          uint32_t pk[16];
          const float(&part)[32] = reinterpret_cast<const float(&)[32]>(sv[c]);
          if (left >= kPxKeys || qscale != 0.f)  // (a masked score times a scale other than 0 is -inf: probability 0)
            l += p_row<false>(part, qscale, nbase, seen, pk);
          else
            l += p_row<true>(part, qscale, nbase, seen, pk);
          tmem_st16(tP + b0 * (kPxKeys / 2) + half * (kPxHalf / 2) + c / 2 + lane_base, pk);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_p[b0]));
      }
      s_max[g & 1][half][row] = l;
      meet();
      l += s_max[g & 1][half ^ 1][row];
      // the partial block, once the last product is complete: 512 consecutive bytes a warp and store
      ok = ok && __all_sync(0xffffffffu,
                            mbar_wait_bounded(smem_u32(&bar_pfree[(g - 1) & 1]), (uint32_t)((g - 1) >> 1) & 1u));
      if (!ok) continue;
      tc_fence_after();
      const PxItem here = px_item(a, item, P);  // (again: its numbers are not held over the tiles)
      float *blk = a.part + prefix_block(here.kvh, here.tile, here.chunk, a.tiles, a.chunks) * prefix_block_floats(D);
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        const int d0 = half * (D / 2) + c;
        tmem_ld32_waited(tO + lane_base + d0, o);
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4 *>(blk + ((d0 + i) / 4 * kPxRows + row) * 4) =
              make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      }
      if (half == 0) {
        blk[kPxRows * D + row] = m_ref;
        blk[kPxRows * (D + 1) + row] = l;
      }
    }
  }
  ok = __syncthreads_and(ok) != 0;
  if (!ok) {
    // before shared memory and TMEM are released: the products (one commit tracks them all) and the copies in flight
    if (tid == kPxMmaWarp * 32) {
      tc_commit(smem_u32(&bar_fin));
      mbar_wait_bounded(smem_u32(&bar_fin), 0);
    }
    if (tid == kPxLoadWarp * 32) {
      for (int g = s_seen[0]; g < s_issued[0]; ++g)
        mbar_wait_bounded(smem_u32(&bar_k[g % C::NST]), (uint32_t)(g / C::NST) & 1u);
      for (int g = s_seen[1]; g < s_issued[1]; ++g)
        mbar_wait_bounded(smem_u32(&bar_v[g % C::NST]), (uint32_t)(g / C::NST) & 1u);
      report(p.status, TD_DEV_WAIT_TIMEOUT);
    }
    if (tid < kPxRows)
      drop_items<D>(a.part, prefix_keys(*a.prefix_len, a.Pmax), a.tiles, p.Hkv, a.chunks, blockIdx.x, gridDim.x, tid, kPxRows);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::TMEM_COLS) : "memory");
}

template <int D, int NT>
cudaError_t launch_nt(const PxArgs &a, int grid, cudaStream_t stream) {
  static OptIn opt_in;
  const cudaError_t e = opt_in(reinterpret_cast<const void *>(&prefix_kernel<D, NT>),
                               PxCfg<D>::SMEM + (2 * TD_MAX_BATCH + 1) * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  const size_t smem = PxCfg<D>::SMEM + (2 * (size_t)a.own.p.B + 1) * sizeof(int);
  return launch_pdl(prefix_kernel<D, NT>, dim3(grid), dim3(kPxThreads), smem, stream, a);
}

template <int D>
cudaError_t launch_d(const PrefixPlan &plan, const PrefixAttn &x, const SplitParams &p, unsigned char *ws, float *part,
                     cudaStream_t stream) {
  PxArgs a;
  if (!fill_runs(&a.own, D, plan.own, p, ws) || !encode_cache_map(&a.kmap, x.k, 1, p.Hkv, x.Pmax, D, kPxKeys) ||
      !encode_cache_map(&a.vmap, x.v, 1, p.Hkv, x.Pmax, D, kPxKeys))
    return cudaErrorInvalidValue;
  a.prefix_len = x.prefix_len;
  a.part = part;
  a.GT = p.G * p.T, a.Pmax = x.Pmax;
  a.tiles = plan.tiles, a.chunks = plan.chunks;
  const int nt = (plan.own.R + 7) / 8;
  return nt == 1   ? launch_nt<D, 1>(a, plan.grid, stream)
         : nt == 2 ? launch_nt<D, 2>(a, plan.grid, stream)
                   : launch_nt<D, 3>(a, plan.grid, stream);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

td_status plan_prefix(int B, int Hq, int Hkv, int T, int Pmax, int Smax, int D, PrefixPlan *plan) {
  if (D != 64 && D != 128) return TD_ERR_UNSUPPORTED;
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || Smax < 1 || Pmax < 1 || Hq % Hkv != 0) return TD_ERR_INVALID_ARG;
  if (B > TD_MAX_BATCH || Smax > (1 << 30) || Pmax > (1 << 30) || T > Smax) return TD_ERR_UNSUPPORTED;
  const td_status st = plan_attn_runs(B, Hq, Hkv, T, Smax, D, &plan->own);
  if (st != TD_OK) return st;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return TD_ERR_CUDA;
  const long long rows = (long long)B * (Hq / Hkv) * T;
  const long long tiles = (rows + kPxRows - 1) / kPxRows;
  const long long groups = tiles * Hkv;
  const int sms = device_sm_count(device);
  // chunks that fill the GPU once
  long long chunks = sms / groups;
  chunks = std::min(chunks, ((long long)Pmax + kPxKeys - 1) / kPxKeys);
  if (chunks < 1) chunks = 1;
  if (groups * chunks * 16 > 0x7fffffffLL) return TD_ERR_UNSUPPORTED;
  plan->tiles = (int)tiles;
  plan->chunks = (int)chunks;
  plan->grid = (int)std::min((long long)sms, std::max((long long)plan->own.grid, groups * chunks));
  plan->off_part = align256(plan->own.bytes);
  plan->bytes = plan->off_part + align256((size_t)(groups * chunks) * prefix_block_floats(D) * sizeof(float));
  return TD_OK;
}

cudaError_t launch_prefix(int D, const PrefixPlan &plan, const PrefixAttn &x, const SplitParams &p, unsigned char *ws,
                          cudaStream_t stream) {
  float *part = reinterpret_cast<float *>(ws + plan.off_part);
  // another thread's call on this stream and workspace comes before or after both launches, not between them
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  cudaError_t e = D == 64 ? launch_d<64>(plan, x, p, ws, part, stream) : launch_d<128>(plan, x, p, ws, part, stream);
  const PrefixPart joined{part, x.prefix_len, x.Pmax, plan.tiles, plan.chunks, plan.grid};
  if (e == cudaSuccess) e = launch_join(D, plan.own, p, ws, joined, stream);
  return e;
}

}  // namespace td
