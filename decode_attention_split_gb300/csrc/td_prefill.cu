// Tiled causal prefill attention on the fifth-generation tensor cores (tcgen05, TMEM, TMA).
//
// Method ("tinydecode": prefill is the causal attention path over the prompt; "llm-decode-cuda"
// names "a tiled FlashAttention-style kernel" as its next step for prefill): for every query
// row t of a chunk of T tokens on top of the cache (seq_lens[b] = L counting them), the exact
// softmax attention over keys j < L - T + t + 1, the same result td_verify_attn defines,
// computed tile by tile with an online softmax.
//
// GB300 design: one CTA per tile of 128 query rows of one query head, two CTAs per SM. Q, K
// and V tiles cross by TMA with the 128-byte swizzle (K and V double-buffered with their own
// barriers, 64 keys per tile). A fifth warp issues the tensor-core products and a sixth the
// copies (a copy waits for its buffer's previous product, which must not hold up the next
// product's issue); the accumulators live in TMEM (256 columns: S in [0, 64), P buffers in
// [64, 96) and [96, 128), O from column 128):
//   S[128 x 64] = Q K^T     (A = Q, B = K, both K-major in shared memory)  -> S columns
//   O[128 x D] += P V       (A = P in TMEM, B = V MN-major in shared memory) -> O
// Each softmax thread owns one query row (its TMEM lane): it reads its 64 scores once and at
// once releases the S columns (an "S free" barrier, one arrival per warp), so the product S of
// tile kt+1 runs while the four softmax warps work on tile kt. It masks the scores causally
// (only in tiles that reach the diagonal or the sequence's end) and writes P = 2^(s - m) as
// bf16 pairs into P buffer kt % 2 once the P V product of tile kt-2 has read it; the P V
// product reads P as its A operand (lane = row, one column per pair of keys). A softmax warp
// hands its rows over through an mbarrier (one arrival per warp), so the warps do not wait
// for one another within a tile. The reference maximum m moves only when a row's maximum
// rises more than 8 (base 2) above it, and only then are that row's O and l rescaled (after
// the previous P V product is complete); otherwise P stays below 2^8 and O / l, kept against
// the same m, need no correction. Query tiles are launched longest first (causal rows late in
// the prompt see the most keys). Every wait is bounded; a timeout sets TD_DEV_WAIT_TIMEOUT,
// and the CTA waits (bounded) for its copies and products in flight before it frees TMEM.
// Measured, 24 + 8 heads of 128: a prompt of 4096 tokens 90 us (1144 TFLOP/s), of 8192 302 to 313 (1364 to 1319; 320 in long
// runs, the power cap); 8000 tokens through a window of 1024 with 4 sinks 120.1 us (798 TFLOP/s of visible work, 1000
// with the masked parts of its tiles).
#include <cudaTypedefs.h>
#include <math.h>

#include <mutex>

#include "td_device.cuh"
#include "td_internal.h"
#include "td_mma.cuh"
#include "td_tc.cuh"

namespace td {

namespace {

constexpr int kPfSoftmaxWarps = 4;                         // one query row per thread
constexpr int kPfMmaWarp = kPfSoftmaxWarps;                  // issues the tensor-core products
constexpr int kPfLoadWarp = kPfSoftmaxWarps + 1;             // issues the TMA copies
constexpr int kPfThreads = 32 * (kPfSoftmaxWarps + 2);
constexpr int kPfRows = 128;   // query rows per CTA
constexpr int kQRegion = kPfRows * 128;  // bytes of one swizzled [128 rows][64 bf16] region
constexpr int kKRegion = kPfKeys * 128;  // bytes of one swizzled [64 rows][64 bf16] region

template <int D>
struct PfCfg {
  static constexpr int HALVES = D / 64;                 // 64-column regions per row tile
  static constexpr int Q_TILE = HALVES * kQRegion;
  static constexpr int KV_TILE = HALVES * kKRegion;     // one K or V tile
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_TILE;                  // two K buffers
  static constexpr int V_OFF = K_OFF + 2 * KV_TILE;     // two V buffers
  static constexpr int SMEM = V_OFF + 2 * KV_TILE + 1024;  // + alignment slack
  static constexpr int TMEM_COLS = 256;                 // S (64), two P buffers (32 each), O (D): a power of two
  static_assert(2 * (SMEM + 1024 + 128) <= 228 * 1024, "two CTAs per SM");
};

struct PfArgs {
  CUtensorMap qmap;  // q [B*Hq][T][D]
  CUtensorMap kmap;  // caches [B*Hkv][Smax][D], boxes of 64 rows
  CUtensorMap vmap;
  const int32_t *seq_lens;
  void *out;         // [B, Hq, T, D] bf16
  float *lse;        // [B, Hq, T] or null
  uint32_t *status;
  int B, Hq, Hkv, T, Smax;
  float qscale;      // scale * log2(e)
  int window, sinks; // the WIN instantiation: keys j <= P with j > P - window or j < sinks
};

// What a row that sees keys below `lim` sees of the tile of keys from j0 on.
template <bool WIN>
__device__ __forceinline__ auto seen_of(const PfArgs &a, int j0, int lim) {
  if constexpr (WIN) {
    const int end = lim - j0, start = end - a.window, first = min(a.sinks, lim) - j0;
    SeenBits s;
    s.lo = (low_bits(end) & ~low_bits(start)) | low_bits(first);
    s.hi = (low_bits(end - 32) & ~low_bits(start - 32)) | low_bits(first - 32);
    return s;
  } else {
    return SeenFirst{min(kPfKeys, max(0, lim - j0))};
  }
}

// WIN: attention over a sliding window with sinks. The key tiles are then those of the sinks and those from the first
// row's window on; tiles that every row sees whole need no mask, as without a window.
template <int D, bool WIN>
__global__ void __launch_bounds__(kPfThreads, 2) prefill_kernel(const __grid_constant__ PfArgs a) {
  using C = PfCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bar_q, bar_k[2], bar_v[2], bar_s[2], bar_sfree, bar_p[2], bar_vfree[2], bar_fin;
  __shared__ uint32_t s_taddr;
  __shared__ int s_issued[2], s_seen[3];  // wind-down: K / V tiles issued; K / V tiles, Q seen landed
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  // blocks start in index order, x fastest: every head's tile late in the prompt (most keys)
  // comes before any shorter one
  const int qt = gridDim.y - 1 - blockIdx.y;
  const int hq = blockIdx.x % a.Hq, b = blockIdx.x / a.Hq;
  const int G = a.Hq / a.Hkv, kvh = hq / G;
  const int t0 = qt * kPfRows;

  if (tid == 0) {
    mbar_init(smem_u32(&bar_q), 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar_k[i]), 1);
      mbar_init(smem_u32(&bar_v[i]), 1);
      mbar_init(smem_u32(&bar_s[i]), 1);
      mbar_init(smem_u32(&bar_p[i]), kPfSoftmaxWarps);
      mbar_init(smem_u32(&bar_vfree[i]), 1);
    }
    s_issued[0] = s_issued[1] = 0;
    s_seen[0] = s_seen[1] = 0;
    s_seen[2] = 1;
    mbar_init(smem_u32(&bar_sfree), kPfSoftmaxWarps);
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
  // S of the current tile in columns [0, 64), P of tile kt in P buffer kt % 2 (columns 64 + 32 (kt % 2),
  // bf16 pairs), O in [128, 128 + D)
  const uint32_t tS = tmem, tP = tmem + kPfKeys, tO = tmem + 128;

  griddep_wait();
  griddep_launch_dependents();
  const int32_t raw = a.seq_lens[b];
  const int L = raw < 0 ? 0 : (raw > a.Smax ? a.Smax : raw);
  const int last_t = min(t0 + kPfRows, a.T) - 1;
  const int kend = max(0, min(L, L - a.T + last_t + 1));  // keys any row of the tile sees
  const int kall = max(0, min(L, L - a.T + t0 + 1));      // keys every row of the tile sees
  // tile i holds the keys from tile_key(i) on
  const int ends = (kend + kPfKeys - 1) / kPfKeys;
  const int head = WIN ? min((min(a.sinks, kend) + kPfKeys - 1) / kPfKeys, ends) : 0;  // tiles with sinks
  const int win0 = WIN ? max(0, L - a.T + t0 - a.window + 1) : 0;  // first key in the first row's window
  const int skip = WIN ? max(0, min(win0 / kPfKeys, ends) - head) : 0;  // tiles between the sinks and the window
  const int nkt = ends - skip;
  auto tile_key = [&](int i) { return (WIN && i >= head ? i + skip : i) * kPfKeys; };
  if (tid == 0 && qt == 0 && hq == 0) {
    uint32_t bits = 0;
    if (raw < 0) bits |= TD_DEV_NEGATIVE_SEQLEN;
    if (raw > a.Smax) bits |= TD_DEV_SEQLEN_CLAMPED;
    if (a.T > 1 && L < a.T) bits |= TD_DEV_VERIFY_SHORT;
    report(a.status, bits);
  }
  const float qscale = a.qscale;
  bool ok = true;
  // copy / tensor-core thread: tiles of K and V issued and seen landed (for the wind-down)
  int kq = 0, kw = 0, vq = 0, vw = 0;
  bool q_seen = false;
  float m_ref = -INFINITY, l = 0.f;  // softmax threads: this row's reference maximum and sum

  if (warp == kPfMmaWarp) {
    if (lane == 0 && nkt > 0) {
      constexpr uint32_t kIdS = mma_idesc(kPfRows, kPfKeys, false);
      constexpr uint32_t kIdO = mma_idesc(kPfRows, D, true);
      // shared-memory descriptors of Q and of K / V buffer 0; any other tile, buffer or k
      // step differs only in its start address (descriptor field in 16-byte units)
      const uint64_t dq = smem_desc(sb + C::Q_OFF, 16, 1024);
      const uint64_t dk = smem_desc(sb + C::K_OFF, 16, 1024);
      const uint64_t dv = smem_desc(sb + C::V_OFF, kKRegion, 1024);
      // S of tile kt into the S columns (K tile kt has landed; its completion is signalled on
      // the barrier of K buffer kt % 2): over D in steps of 16 (32 bytes along a swizzled row;
      // the next 64 columns are the next region)
      auto issue_s = [&](int kt) {
        const uint32_t kb = (uint32_t)(kt & 1) * C::KV_TILE;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)(k & 3) * 32;
          tc_mma(tS, dq + (((uint32_t)(k >> 2) * kQRegion + off) >> 4),
                 dk + ((kb + (uint32_t)(k >> 2) * kKRegion + off) >> 4), kIdS, k > 0);
        }
        tc_commit(smem_u32(&bar_s[kt & 1]));
      };
      q_seen = mbar_wait_bounded(smem_u32(&bar_q), 0);
      ok = q_seen && mbar_wait_bounded(smem_u32(&bar_k[0]), 0);
      if (ok) {
        kw = 1;
        issue_s(0);
      }
      for (int kt = 0; ok && kt < nkt; ++kt) {
        const int b0 = kt & 1, b1 = b0 ^ 1;
        if (kt + 1 < nkt) {
          // the S columns are free once every softmax warp has read S of kt
          ok = mbar_wait_bounded(smem_u32(&bar_sfree), (uint32_t)kt & 1u);
          ok = ok && mbar_wait_bounded(smem_u32(&bar_k[b1]), (uint32_t)((kt + 1) >> 1) & 1u);
          if (!ok) break;
          kw = kt + 2;
          issue_s(kt + 1);
        }
        // P of kt is in P buffer b0 (all four softmax warps) and V of kt has landed: O += P V
        // over 64 keys in steps of 16 (A: 8 TMEM columns per step; B: MN-major, 16 rows of 128
        // bytes per step, the next 64 columns in the next region)
        ok = mbar_wait_bounded(smem_u32(&bar_p[b0]), (uint32_t)(kt >> 1) & 1u) &&
             mbar_wait_bounded(smem_u32(&bar_v[b0]), (uint32_t)(kt >> 1) & 1u);
        if (!ok) break;
        vw = kt + 1;
        tc_fence_after();
        const uint32_t vb = (uint32_t)b0 * C::KV_TILE;
#pragma unroll
        for (int k = 0; k < kPfKeys / 16; ++k)
          tc_mma_ts(tO, tP + b0 * (kPfKeys / 2) + 8 * k, dv + ((vb + (uint32_t)k * 16 * 128) >> 4), kIdO, kt > 0 || k > 0);
        tc_commit(smem_u32(&bar_vfree[b0]));  // V buffer b0 may be refilled, P buffer b0 rewritten, O of kt read
      }
      s_seen[0] = kw;
      s_seen[1] = vw;
      s_seen[2] = q_seen;
    }
    __syncwarp();
  } else if (warp == kPfLoadWarp) {
    if (lane == 0 && nkt > 0) {
      const int zq = b * a.Hq + hq, zk = b * a.Hkv + kvh;
      auto load = [&](bool v, int kt) {  // K or V tile kt into buffer kt % 2
        const int buf = kt & 1;
        const uint32_t bar = smem_u32(v ? &bar_v[buf] : &bar_k[buf]);
        const uint32_t dst = sb + (v ? C::V_OFF : C::K_OFF) + buf * C::KV_TILE;
        mbar_arrive_expect_tx(bar, C::KV_TILE);
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h) tma3(dst + h * kKRegion, v ? &a.vmap : &a.kmap, 64 * h, tile_key(kt), zk, bar);
      };
      {
        const uint32_t bar = smem_u32(&bar_q);
        mbar_arrive_expect_tx(bar, C::Q_TILE);
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h) tma3(sb + C::Q_OFF + h * kQRegion, &a.qmap, 64 * h, t0, zq, bar);
      }
      for (; kq < min(nkt, 2); ++kq) {
        load(false, kq);
        load(true, kq);
      }
      vq = kq;
      // tile j (j >= 2) goes to buffer j % 2 once its previous user, tile j-2, is done with
      // it: K after the product S of j-2, V after the P V product of j-2. Each buffer's next
      // product needs the copy issued here, so its barrier cannot run a phase ahead.
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
    // softmax warps: thread `row` owns query t = t0 + row, which sees keys j < L - T + t + 1
    const int row = tid;
    const int t = t0 + row;
    const int lim = t < a.T ? max(0, min(L, L - a.T + t + 1)) : 0;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    for (int kt = 0; kt < nkt; ++kt) {
      const int b0 = kt & 1;
      const uint32_t ph = (uint32_t)(kt >> 1) & 1u;
      // S of kt is complete (the TMEM accesses below are warp-wide: one decision per warp)
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_s[b0]), ph))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int j0 = tile_key(kt);
      // V rows at or past the sequence's length (with a window: rows that none of the tile's
      // queries sees), once landed: zeroed (a masked p of 0 must not meet a stale value)
      const int vrows = min(kPfKeys, (WIN ? kend : L) - j0);
      const int g0 = WIN ? max(a.sinks - j0, 0) : 0, g1 = WIN ? min(win0 - j0, kPfKeys) : 0;  // and [g0, g1)
      if (vrows < kPfKeys || g0 < g1) {
        // (the product of kt-2 first: until then the buffer's barrier may be in kt-2's phase, whose
        // predecessor has the parity of kt's)
        const bool before = kt < 2 || mbar_wait_bounded(smem_u32(&bar_vfree[b0]), (uint32_t)((kt - 2) >> 1) & 1u);
        if (!__all_sync(0xffffffffu, before && mbar_wait_bounded(smem_u32(&bar_v[b0]), ph))) {
          ok = false;
          break;
        }
        unsigned char *vt = smem + C::V_OFF + b0 * C::KV_TILE;
        for (int idx = tid; idx < (kPfKeys - vrows) * (D / 8); idx += 32 * kPfSoftmaxWarps) {
          const int r = vrows + idx / (D / 8), c = idx % (D / 8);
          *reinterpret_cast<uint4 *>(vt + tile_chunk(kPfKeys, r, c)) = make_uint4(0u, 0u, 0u, 0u);
        }
        for (int idx = tid; WIN && idx < (g1 - g0) * (D / 8); idx += 32 * kPfSoftmaxWarps) {
          const int r = g0 + idx / (D / 8), c = idx % (D / 8);
          *reinterpret_cast<uint4 *>(vt + tile_chunk(kPfKeys, r, c)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();  // read next by the tensor core (asynchronous proxy)
      }
      // this row's 64 scores, read once; then the S columns are released for the next tile
      float sv[kPfKeys];
      tmem_ld64(tS + lane_base, sv);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_sfree));
      // tiles short of every row's diagonal and of the sequence's end need no mask; in the
      // others, keys from `vis` on are masked (this row's visible keys of the tile)
      const bool full = j0 + kPfKeys <= kall && (!WIN || j0 + kPfKeys <= a.sinks || j0 >= kend - a.window);
      const auto seen = seen_of<WIN>(a, j0, lim);
      if (!full) {
#pragma unroll
        for (int i = 0; i < kPfKeys; ++i)
          if (!seen(i)) sv[i] = qscale >= 0.f ? -INFINITY : INFINITY;
      }
      // the row maximum, scaled to base 2 (the scale's sign decides which extreme): eight
      // independent chains of three-input steps
      const float ext = qscale >= 0.f ? row_extreme<false>(sv) : row_extreme<true>(sv);
      const float mx = full || seen.any() ? ext * qscale : -INFINITY;
      const bool move = mx > m_ref + kRescaleGap || (m_ref == -INFINITY && mx > -INFINITY);
      const float m_new = WIN ? mx + kRescaleLead : mx;  // (the 8000-token prompt: 127.2 -> 120.1 us)
      const float alpha = (move && m_ref != -INFINITY) ? exp2_approx(m_ref - m_new) : 1.f;
      if (move) {
        l *= alpha;
        m_ref = m_new;
      }
      // a warp rescales its rows of O when any of them must, once the previous P V product
      // is complete (TMEM loads and stores are warp-wide). The product of kt-2 may still be
      // running here (S of kt is issued before the product of kt-1), so the wait is on a barrier
      // whose last phase but one, kt-3, is known complete (P of kt-1 waited for it): a barrier
      // that every product arrives on could still be in the phase of kt-2, whose parity lets a wait for
      // kt-1 pass at once
      if (kt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_vfree[b0 ^ 1]), (uint32_t)((kt - 1) >> 1) & 1u))) {
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
      // P = 2^(s - m) as bf16 pairs into P buffer b0, once the P V product of kt-2 has read it
      const float nbase = m_ref == -INFINITY ? 0.f : -m_ref;
      uint32_t pk[kPfKeys / 2];
      // (a masked score times a scale other than 0 is -inf, whose probability is 0 without a second mask)
      if (full || (WIN && qscale != 0.f))
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
    // the last P V product is complete before O is read
    if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bar_vfree[(nkt - 1) & 1]), (uint32_t)((nkt - 1) >> 1) & 1u)))
      ok = false;
  }
  ok = __syncthreads_and(ok) != 0;
  if (!ok) {
    // before shared memory and TMEM are released: the tensor-core products (one commit
    // tracks them all) and the copies issued but never seen landed
    if (tid == kPfMmaWarp * 32) {
      tc_commit(smem_u32(&bar_fin));
      mbar_wait_bounded(smem_u32(&bar_fin), 0);
    }
    if (tid == kPfLoadWarp * 32) {
      if (nkt > 0 && !s_seen[2]) mbar_wait_bounded(smem_u32(&bar_q), 0);
      for (int kt = s_seen[0]; kt < s_issued[0]; ++kt)
        mbar_wait_bounded(smem_u32(&bar_k[kt & 1]), (uint32_t)(kt >> 1) & 1u);
      for (int kt = s_seen[1]; kt < s_issued[1]; ++kt)
        mbar_wait_bounded(smem_u32(&bar_v[kt & 1]), (uint32_t)(kt >> 1) & 1u);
      report(a.status, TD_DEV_WAIT_TIMEOUT);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp < kPfSoftmaxWarps) {
    // epilogue: O / l for this row, lse = m + log2(l) (natural-log units); the TMEM loads are
    // warp-wide, so every thread takes part and only the stores depend on the row
    const int row = tid, t = t0 + row;
    const bool row_valid = t < a.T;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const float inv = (ok && l != 0.f) ? 1.f / l : 0.f;
    __nv_bfloat16 *orow =
        static_cast<__nv_bfloat16 *>(a.out) + (((size_t)b * a.Hq + hq) * a.T + (row_valid ? t : 0)) * D;
#pragma unroll
    for (int c = 0; c < D; c += 32) {
      float o[32];
      if (nkt > 0) {
        tmem_ld32(tO + lane_base + c, o);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0.f;
      }
      if (row_valid) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) pk[i / 2] = pack_bf16x2(o[i] * inv, o[i + 1] * inv);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<uint4 *>(orow + c)[q] = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
      }
    }
    if (row_valid && a.lse != nullptr)
      a.lse[((size_t)b * a.Hq + hq) * a.T + t] = (ok && l != 0.f) ? (m_ref + log2f(l)) * kLn2 : -INFINITY;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::TMEM_COLS) : "memory");
}

PFN_cuTensorMapEncodeTiled_v12000 pf_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// 3-D map over [planes][rows][D] bf16, boxes of 64 columns x box_rows rows, 128-byte swizzle.
bool pf_map(CUtensorMap *m, const void *base, long long planes, int rows, int D, int box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = pf_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)rows * D * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool WIN>
cudaError_t launch_prefill_d(PfArgs &a, const void *q, const void *k, const void *v, cudaStream_t stream) {
  if (!pf_map(&a.qmap, q, (long long)a.B * a.Hq, a.T, D, kPfRows) ||
      !pf_map(&a.kmap, k, (long long)a.B * a.Hkv, a.Smax, D, kPfKeys) ||
      !pf_map(&a.vmap, v, (long long)a.B * a.Hkv, a.Smax, D, kPfKeys))
    return cudaErrorInvalidValue;
  static OptIn opt_in;
  const cudaError_t attr = opt_in(reinterpret_cast<const void *>(&prefill_kernel<D, WIN>), PfCfg<D>::SMEM);
  if (attr != cudaSuccess) return attr;
  const dim3 grid((unsigned)(a.B * a.Hq), (unsigned)((a.T + kPfRows - 1) / kPfRows));
  return launch_pdl(prefill_kernel<D, WIN>, grid, dim3(kPfThreads), PfCfg<D>::SMEM, stream, a);
}

}  // namespace

cudaError_t launch_prefill(const void *q, const void *k, const void *v, const int32_t *seq_lens, int B, int Hq, int Hkv,
                           int T, int Smax, int D, float scale, void *out, float *lse, uint32_t *status,
                           cudaStream_t stream, int window, int sinks) {
  PfArgs a;
  a.seq_lens = seq_lens;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.T = T;
  a.Smax = Smax;
  a.qscale = scale * kLog2e;
  a.window = window;
  a.sinks = sinks;
  if (window > 0)
    return D == 64 ? launch_prefill_d<64, true>(a, q, k, v, stream) : launch_prefill_d<128, true>(a, q, k, v, stream);
  return D == 64 ? launch_prefill_d<64, false>(a, q, k, v, stream) : launch_prefill_d<128, false>(a, q, k, v, stream);
}

}  // namespace td
