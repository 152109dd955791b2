// Split attention in equal runs of 16-key steps, a run a warp, for bf16 caches; the parts of a row meet in a launch
// of their own (join_kernel).
//
// The keys of every group (sequence, kv head, row block of at most 24 rows) are cut into steps of 16, one group after
// another, and the steps into equal runs. Each warp takes one run on its own: lane 0 keeps its ring of stages (16 keys of
// K and V each, TMA) full across the ends of groups, so a warp that finishes one group and starts the next has
// copies in flight all the time, and no barrier ties the warps of a CTA together once the runs are planned. Where
// a CTA's warps share a chunk instead (split_attn_mma_kernel), starting and finishing a chunk costs a CTA as much as a few
// stages of 64 keys, and chunks of one size leave CTAs idle: many short sequences pay both.
// A warp leaves each group it met as one partial block, so a row has as many parts as runs touch its group.
#pragma once

#include "td_internal.h"
#include "td_split_mma.cuh"

namespace td {

constexpr int kRunWarps = 4;
constexpr int kRunThreads = 32 * kRunWarps;
constexpr int kRunKeys = 16;  // keys of a step and stage

// ST: stages of a warp's ring at D = 128 (twice as many at 64).
template <int D, int ST>
struct RunCfg {
  static constexpr int STAGES = D == 128 ? ST : 2 * ST;
  static constexpr int HALVES = D / 64;
  static constexpr int BOX = kRunKeys * 128;             // 16 rows x 128 bytes
  static constexpr int TILE = HALVES * BOX;              // K or V of a stage
  static constexpr int RING = STAGES * 2 * TILE;
};

struct RunArgs {
  CUtensorMap kmap;  // caches [B*Hkv][Smax][D], boxes of 16 rows
  CUtensorMap vmap;
  SplitParams p;
};
bool fill_runs(RunArgs *a, int D, const RunsPlan &plan, const SplitParams &p, unsigned char *ws);

// A partial block: acc [D / 4][R][4] (sums of 2^(s - m) v), then m [R] (base 2) and l [R]; whole 16-byte units, so that
// every block's sums can be read four at a time.
__host__ __device__ constexpr int run_block_floats(int R, int D) { return (R * (D + 2) + 3) / 4 * 4; }

// Units of a group of `keys` keys: its steps, and as many units as starting and finishing it costs, ahead of its own.
constexpr int kRunGroupUnits = 1;
constexpr int kRunLeast = 2;  // units of the shortest run
__host__ __device__ __forceinline__ int run_steps(int keys) { return (keys + kRunKeys - 1) / kRunKeys; }
__host__ __device__ __forceinline__ int run_units(int keys) { return keys > 0 ? run_steps(keys) + kRunGroupUnits : 0; }
// The block of group g's keys in run r: runs and groups advance together, so every (group, run) that meet have their own.
__host__ __device__ __forceinline__ long long run_block(long long g, int r) { return g + r; }
// The runs, S units long, that hold steps of a group of `units` units behind `base` others: n of them from the first on.
struct RunSpan {
  int first, n;
};
__host__ __device__ __forceinline__ RunSpan runs_of(int base, int units, int S) {
  const int first = (base + kRunGroupUnits) / S;
  return {first, units > 0 ? (base + units - 1) / S + 1 - first : 0};
}

// A barrier of the kRunThreads threads that take runs.
template <int ID>
__device__ __forceinline__ void run_barrier() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(kRunThreads) : "memory");
}

// Units of a run, of W in all dealt to `grid` CTAs.
__host__ __device__ __forceinline__ int run_length(int W, int grid) {
  const int runs = grid * kRunWarps;
  return max((W + runs - 1) / runs, kRunLeast);
}

// Fills s_len (attended lengths, as they read now) and s_prefix (units before each sequence; their total at [B]); returns
// the units of a run. By kRunThreads threads, `tid` theirs, meeting at barrier BAR. Ends with a barrier.
template <int BAR>
__device__ int plan_runs(const SplitParams &p, int tid, int *s_len, int *s_prefix, int *s_red) {
  const int lane = tid & 31, warp = tid >> 5;
  const int U = p.Hkv * p.RB, per = (p.B + kRunThreads - 1) / kRunThreads, b0 = tid * per;
  int seg = 0;
  uint32_t bits = 0;
  for (int b = b0; b < min(b0 + per, p.B); ++b) {
    const int L = attended_len(p, ld_relaxed(p.seq_lens + b), bits);
    s_len[b] = L;
    seg += run_units(L) * U;
  }
  int incl = seg;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_red[warp] = incl;
  run_barrier<BAR>();
  int W = 0, before = incl - seg;
#pragma unroll
  for (int w = 0; w < kRunWarps; ++w) {
    if (w < warp) before += s_red[w];
    W += s_red[w];
  }
  for (int b = b0; b < min(b0 + per, p.B); ++b) {
    s_prefix[b] = before;
    before += run_units(s_len[b]) * U;
  }
  if (tid == 0) s_prefix[p.B] = W;
  run_barrier<BAR>();
  return run_length(W, gridDim.x);
}

// Where a warp is in its run: group `ug` of sequence b, steps [s, e) of it left in this run.
struct RunCursor {
  int b, ug, s, e;
  int base;  // units before this group
};

// Moves the cursor to the next group with steps in units [.., u1); e = s where none is left.
__host__ __device__ __forceinline__ void next_group(const SplitParams &p, const int *s_len, int u1, RunCursor &c) {
  const int U = p.Hkv * p.RB;
  c.s = c.e = 0;
  c.base += run_units(s_len[c.b]);
  if (++c.ug == U) {
    c.ug = 0;
    do {
      if (++c.b >= p.B) return;
    } while (s_len[c.b] == 0);
  }
  if (c.base + kRunGroupUnits < u1) c.e = min(run_steps(s_len[c.b]), u1 - c.base - kRunGroupUnits);
}

// Whether the lengths still read as a plan_runs of these threads found them; reports the status bits that they raise.
template <int BAR>
__device__ __forceinline__ bool lens_stand(const SplitParams &p, int tid, const int *s_len) {
  const int per = (p.B + kRunThreads - 1) / kRunThreads, b0 = tid * per;
  uint32_t bits = 0, same = 1;
  for (int b = b0; b < min(b0 + per, p.B); ++b) same &= attended_len(p, ld_relaxed(p.seq_lens + b), bits) == s_len[b];
  if (blockIdx.x == 0) report(p.status, bits);
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %0, 0;\nbarrier.cta.red.and.pred q, %1, %2, p;\nselp.u32 %0, 1, 0, q;\n}"
      : "+r"(same)
      : "n"(BAR), "n"(kRunThreads)
      : "memory");
  return same != 0;
}

// Where run number `run`, S units long, starts; u1 receives where it ends.
__host__ __device__ __forceinline__ RunCursor run_start(const SplitParams &p, const int *s_len, const int *s_prefix, int S,
                                                        int run, int &u1) {
  const int W = s_prefix[p.B], u0 = (int)min((long long)run * S, (long long)W);
  u1 = (int)min((long long)u0 + S, (long long)W);
  RunCursor c{};
  if (u0 < u1) {
    int lo = 0, hi = p.B - 1;  // the last sequence whose units start at or before u0 (those without keys have none)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_prefix[mid] <= u0) lo = mid; else hi = mid - 1;
    }
    const int n = run_units(s_len[lo]);
    c.b = lo;
    c.ug = (u0 - s_prefix[lo]) / n;
    c.base = s_prefix[lo] + c.ug * n;
    c.s = max(u0 - c.base - kRunGroupUnits, 0);
    c.e = max(min(n, u1 - c.base) - kRunGroupUnits, 0);
    if (c.s >= c.e) next_group(p, s_len, u1, c);
  }
  return c;
}

// A run that gave up in the group at c: the groups behind it, which the join reads as well, are left without keys (l = 0;
// their blocks may hold an earlier call's). By threads lane, lane + lanes, ...
template <int D>
__host__ __device__ inline void drop_rest_of_run(const SplitParams &p, const int *s_len, RunCursor c, int u1, int run, int lane,
                                                 int lanes) {
  for (next_group(p, s_len, u1, c); c.s < c.e; next_group(p, s_len, u1, c)) {
    float *blk = p.ws_part + run_block((long long)c.b * p.Hkv * p.RB + c.ug, run) * run_block_floats(p.R, D);
    for (int r = lane; r < p.R; r += lanes) blk[p.R * (D + 1) + r] = 0.f;
  }
}

// A warp's ring: its barriers, by one thread.
template <int STAGES>
__device__ __forceinline__ void init_ring(uint64_t *bars) {
#pragma unroll
  for (int i = 0; i < STAGES; ++i) mbar_init(smem_u32(&bars[i]), 1);
  fence_mbar_init();
}

// One warp's run, number `run`, from c on to unit u1. The warp's ring (1024-byte aligned) and its barriers (initialised, one
// arrival).
template <int D, int NT, int ST>
__device__ __forceinline__ void run_warp(const SplitParams &p, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                         const int *s_len, RunCursor c, int u1, int run, unsigned char *ring_p,
                                         uint64_t *bars) {
  using C = RunCfg<D, ST>;
  constexpr int KSD = D / 16, NL = 2 * NT;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const uint32_t ring = smem_u32(ring_p);
  const int GT = p.G * p.T;
  const uint64_t policy = l2_evict_first_policy();

  RunCursor ahead = c;  // the next step to be fetched
  int fetched = 0, used = 0;
  auto fetch = [&]() {  // lane 0 of a warp whose ring has room
    const int buf = fetched % C::STAGES;
    const uint32_t bar = smem_u32(&bars[buf]);
    const uint32_t kdst = ring + buf * 2 * C::TILE, vdst = kdst + C::TILE;
    const int key = ahead.s * kRunKeys, z = ahead.b * p.Hkv + ahead.ug / p.RB;
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(bar, 2 * C::TILE);
#pragma unroll
    for (int h = 0; h < C::HALVES; ++h) {
      tma_load_3d(kdst + h * C::BOX, &kmap, 64 * h, key, z, bar, policy);
      tma_load_3d(vdst + h * C::BOX, &vmap, 64 * h, key, z, bar, policy);
    }
  };
  auto step_ahead = [&]() {  // the cursor is the warp's, whichever lane issues
    if (ahead.s >= ahead.e) return;
    if (lane == 0) fetch();
    ++fetched;
    if (++ahead.s == ahead.e) next_group(p, s_len, u1, ahead);
  };
#pragma unroll 1
  for (int i = 0; i < C::STAGES; ++i) step_ahead();

  bool ok = true;
  while (ok && c.s < c.e) {
    // one group: its query rows as B fragments of each n tile
    const int rb = c.ug % p.RB, kvh = c.ug / p.RB, L = s_len[c.b];
    uint32_t qb[NT][KSD][2];
    int lim[NL];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + gid, gr = rb * p.R + r;
      const bool there = r < p.R && gr < GT;
      const uint32_t *qrow = static_cast<const uint32_t *>(p.q) +
                             ((long long)c.b * p.Hq * p.T + (long long)kvh * GT + (there ? gr : 0)) * (D / 2) + tig;
#pragma unroll
      for (int j = 0; j < KSD; ++j) {
        qb[nt][j][0] = there ? __ldcg(qrow + 8 * j) : 0u;
        qb[nt][j][1] = there ? __ldcg(qrow + 8 * j + 4) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rl = 8 * nt + 2 * tig + e, gl = rb * p.R + rl;
        lim[2 * nt + e] = rl < p.R && gl < GT ? max(L - p.T + gl % p.T + 1, 0) : 0;
      }
    }
    float o[NT][KSD][4], m_run[NL], l_run[NL];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < KSD; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
    for (int h = 0; h < NL; ++h) m_run[h] = -INFINITY, l_run[h] = 0.f;
#pragma unroll 1
    for (; c.s < c.e; ++c.s) {
      const int buf = used % C::STAGES;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&bars[buf]), (uint32_t)(used / C::STAGES) & 1u))) {
        ok = false;
        break;
      }
      const uint32_t kt = ring + buf * 2 * C::TILE, vt = kt + C::TILE;
      const int key0 = c.s * kRunKeys;
      // V rows behind the sequence's end: zeroed, so that a masked probability meets no stale value
      const int z0 = L - key0;
      if (z0 < kRunKeys) {
        unsigned char *vrow = ring_p + buf * 2 * C::TILE + C::TILE;
        for (int i = lane; i < (kRunKeys - z0) * (D / 8); i += 32)
          *reinterpret_cast<uint4 *>(vrow + tma_swz<kRunKeys>(z0 + i / (D / 8), i % (D / 8))) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();  // precedes the stage's next refill by the TMA unit
        __syncwarp();
      }
      if constexpr (NT == 1)
        warp_keys16_n8<D, 0, kRunKeys>(qb[0], kt, vt, 0, key0, lim, p.qscale, o[0], m_run, l_run);
      else
        warp_keys16_nt<D, 0, NT, kRunKeys>(qb, kt, vt, 0, key0, lim, p.qscale, o, m_run, l_run);
      ++used;
      __syncwarp();  // every lane has read the stage
      step_ahead();
    }
    // this run's part of the group
    float *blk = p.ws_part + run_block(((long long)c.b * p.Hkv + kvh) * p.RB + rb, run) * run_block_floats(p.R, D);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_run[2 * nt + e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int r = 8 * nt + 2 * tig + e;
        if (r >= p.R) continue;
        float *row = blk + 4 * r + (gid & 3);
#pragma unroll
        for (int dt = 0; dt < KSD; ++dt) {
          row[(4 * dt + gid / 4) * 4 * p.R] = o[nt][dt][e];
          row[(4 * dt + 2 + gid / 4) * 4 * p.R] = o[nt][dt][2 + e];
        }
        if (gid == 0) {
          blk[p.R * D + r] = m_run[2 * nt + e];
          blk[p.R * (D + 1) + r] = ok ? l : 0.f;
        }
      }
    if (ok) next_group(p, s_len, u1, c);
  }
  if (!ok) {
    // a copy never completed: the others in flight are waited for (bounded) before the ring goes
    if (lane == 0) {
      for (int i = used; i < fetched; ++i)
        mbar_wait_bounded(smem_u32(&bars[i % C::STAGES]), (uint32_t)(i / C::STAGES) & 1u);
      report(p.status, TD_DEV_WAIT_TIMEOUT);
    }
    drop_rest_of_run<D>(p, s_len, c, u1, run, lane, 32);
  }
}

// Prefix length attended, and the keys of a chunk of it (whole tiles).
constexpr int kPrefixKeys = 128;
__host__ __device__ __forceinline__ int prefix_keys(int raw, int Pmax) { return raw < 0 ? 0 : raw > Pmax ? Pmax : raw; }
__host__ __device__ __forceinline__ int prefix_chunk(int P, int chunks) {
  return ((P + kPrefixKeys - 1) / kPrefixKeys + chunks - 1) / chunks * kPrefixKeys;
}
// Chunks of it that hold keys.
__host__ __device__ __forceinline__ int prefix_parts(int P, int chunks) {
  const int C = prefix_chunk(P, chunks);
  return P > 0 ? (P + C - 1) / C : 0;
}
constexpr int kPrefixRows = 128;  // query rows of a tile over the prefix
__host__ __device__ constexpr int prefix_block_floats(int D) { return kPrefixRows * (D + 2); }
// The block of chunk `chunk` for tile `tile` of kv head kvh.
__host__ __device__ __forceinline__ long long prefix_block(int kvh, int tile, int chunk, int tiles, int chunks) {
  return ((long long)kvh * tiles + tile) * chunks + chunk;
}

// Work over the prefix, item by item: a tile of a kv head's rows over a chunk. The tiles that read one chunk are neighbours.
struct PrefixItem {
  int tile, kvh, chunk;
};
__host__ __device__ __forceinline__ PrefixItem prefix_item(int item, int tiles, int Hkv) {
  return {item % tiles, item / tiles % Hkv, item / tiles / Hkv};
}
// A CTA that gave up: the blocks of its items (`item` and every grid-th behind it), which the join reads as well, are left
// without keys (they may hold an earlier call's). By threads lane, lane + lanes, ...
template <int D>
__host__ __device__ inline void drop_items(float *part, int P, int tiles, int Hkv, int chunks, int item, int grid, int lane,
                                           int lanes) {
  const int items = tiles * Hkv * prefix_parts(P, chunks);
  for (; item < items; item += grid) {
    const PrefixItem w = prefix_item(item, tiles, Hkv);
    float *blk = part + prefix_block(w.kvh, w.tile, w.chunk, tiles, chunks) * prefix_block_floats(D);
    for (int r = lane; r < kPrefixRows; r += lanes) blk[kPrefixRows * (D + 1) + r] = 0.f;
  }
}

// Joins the parts of a row: those that the runs left of its own keys and one per chunk of the shared
// prefix (blocks acc [D / 4][128 rows][4], m [128], l [128] of 128-row tiles).
struct JoinArgs {
  const float *runs;      // blocks of the runs that `grid` CTAs took
  const int32_t *seq_lens;
  const float *prefix;    // [Hkv][tiles][chunks] blocks
  const int32_t *prefix_len;
  void *out;              // [B, Hq, T, D] bf16
  float *lse;             // [B, Hq, T] or null
  int B, Hq, Hkv, T, GT, R, RB, Smax, Pmax, tiles, chunks, grid;
};

// Grid: kv heads x 32-row groups of their B * GT rows x slabs of dims. A lane has a row, a warp eight dims and every
// SPLIT-th of the row's parts (its runs', then the prefix's); the warps of a row's dims meet in shared memory. What bounds it
// is its chain of loads (a part's m and l and sums, one batch after another) behind the launch, so a batch is asked for at
// once, where rows are few their parts are spread over SPLIT warps, and each warp finds its rows' parts before it waits
// for the launch that leaves them. (It may read the lengths then: every CTA of that launch, which lets this one start, has
// waited for the launches before it.)
//
// CTAs of four warps (SPLIT's, if those are more), so that a few hundred of them spread evenly, and no more registers than
// let an SM hold 768 threads. The launch asks for so much shared memory that no SM takes more than its share of the CTAs:
// they start while SMs fall free one by one, and would share the first while others stay idle. Measured in us of a
// call: six tokens of 16 sequences behind 4321 keys 26.5 -> 25.0, single tokens of 48 behind 8192 26.5 -> 25.5, of 64
// unchanged at 28.0, of 16 behind 1000 (5 heads of 64) 10.6 -> 8.7. Without the spreading, 3 CTAs of 256 threads an SM lose 1 us.
constexpr int kJoinBatch = 4;         // parts of a row in flight at once (6 and 8: no gain, 2.5 us lost at 25 parts)
constexpr int kJoinSmThreads = 768;
__host__ __device__ constexpr int join_threads(int split) { return split > 4 ? 32 * split : 128; }
template <int D, int SPLIT>
__global__ void __launch_bounds__(join_threads(SPLIT), kJoinSmThreads / join_threads(SPLIT)) join_kernel(const JoinArgs a) {
  constexpr int THREADS = join_threads(SPLIT), COLS = THREADS / 32 / SPLIT;  // warps side by side, eight dims each
  constexpr int SLABS = D / 8 / COLS;
  const int rows = a.B * a.GT, groups = (rows + 31) / 32;
  const int slab = blockIdx.x % SLABS, group = blockIdx.x / SLABS % groups, kvh = blockIdx.x / SLABS / groups;
  const int warp = threadIdx.x / 32, part0 = warp / COLS, d8 = slab * COLS + warp % COLS;
  const int row = min(group * 32 + (int)(threadIdx.x & 31), rows - 1);  // (the last group's lanes repeat a row)
  const int b = row / a.GT, gt = row % a.GT, rb = gt / a.R, r = gt % a.R;
  // the runs that hold steps of this row's group, and the chunks of the prefix
  const int P = prefix_keys(__ldcg(a.prefix_len), a.Pmax), U = a.Hkv * a.RB, lane = threadIdx.x & 31;
  int first = 0, units = 0, W = 0;  // units before the row's sequence, of one of its groups, and in all
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int mine = b0 + lane < a.B ? run_units(min(max(__ldcg(a.seq_lens + b0 + lane), 0), a.Smax)) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int own = __shfl_sync(0xffffffffu, mine, b & 31), upto = __shfl_sync(0xffffffffu, incl, b & 31);
    if (b >= b0 && b < b0 + 32) first = W + (upto - own) * U, units = own;
    W += __shfl_sync(0xffffffffu, incl, 31) * U;
  }
  const int S = run_length(W, a.grid), base = first + (kvh * a.RB + rb) * units;
  const RunSpan span = runs_of(base, units, S);
  const int n_runs = span.n, n = n_runs + prefix_parts(P, a.chunks);
  const int BF = run_block_floats(a.R, D);
  const float *runs = a.runs + run_block(((long long)b * a.Hkv + kvh) * a.RB + rb, span.first) * BF;
  const float *chunks = a.prefix + prefix_block(kvh, row / kPrefixRows, 0, a.tiles, a.chunks) * prefix_block_floats(D);
  float M = -INFINITY, L = 0.f, A[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) A[k] = 0.f;
  griddep_wait();
  griddep_launch_dependents();
  for (int p0 = part0; p0 < n; p0 += SPLIT * kJoinBatch) {
    float m[kJoinBatch], l[kJoinBatch];
    float4 x[kJoinBatch], y[kJoinBatch];
    float Mn = M;
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      const int p = p0 + i * SPLIT;
      const bool own = p < n_runs;
      const float *pb = own ? runs + (long long)p * BF : chunks + (long long)(p - n_runs) * prefix_block_floats(D);
      const int R = own ? a.R : kPrefixRows, at = own ? r : row % kPrefixRows;
      m[i] = -INFINITY, l[i] = 0.f;
      if (p < n) {
        m[i] = __ldcg(pb + R * D + at);
        l[i] = __ldcg(pb + R * (D + 1) + at);
        x[i] = __ldcg(reinterpret_cast<const float4 *>(pb) + 2 * d8 * R + at);
        y[i] = __ldcg(reinterpret_cast<const float4 *>(pb) + (2 * d8 + 1) * R + at);
      }
    }
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i)
      if (l[i] != 0.f) Mn = fmaxf(Mn, m[i]);  // a part without keys (l = 0) counts nothing; a NaN stays one
    const float ref = Mn == -INFINITY ? 0.f : Mn;
    const float alpha = exp2f(M - ref);
    L *= alpha;
#pragma unroll
    for (int k = 0; k < 8; ++k) A[k] *= alpha;
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      if (l[i] != 0.f) {
        const float f = exp2f(m[i] - ref);
        L = fmaf(l[i], f, L);
        A[0] = fmaf(x[i].x, f, A[0]), A[1] = fmaf(x[i].y, f, A[1]), A[2] = fmaf(x[i].z, f, A[2]), A[3] = fmaf(x[i].w, f, A[3]);
        A[4] = fmaf(y[i].x, f, A[4]), A[5] = fmaf(y[i].y, f, A[5]), A[6] = fmaf(y[i].z, f, A[6]), A[7] = fmaf(y[i].w, f, A[7]);
      }
    }
    M = Mn;
  }
  if constexpr (SPLIT > 1) {
    __shared__ float s_acc[8][THREADS];
    __shared__ float2 s_ml[THREADS];
#pragma unroll
    for (int k = 0; k < 8; ++k) s_acc[k][threadIdx.x] = A[k];
    s_ml[threadIdx.x] = make_float2(M, L);
    __syncthreads();
    if (part0 != 0) return;
    float2 ml[SPLIT];
    M = -INFINITY, L = 0.f;
#pragma unroll
    for (int j = 0; j < SPLIT; ++j) {
      ml[j] = s_ml[threadIdx.x + 32 * COLS * j];
      if (ml[j].y != 0.f) M = fmaxf(M, ml[j].x);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) A[k] = 0.f;
#pragma unroll
    for (int j = 0; j < SPLIT; ++j) {
      if (ml[j].y != 0.f) {
        const float f = exp2f(ml[j].x - (M == -INFINITY ? 0.f : M));
        L = fmaf(ml[j].y, f, L);
#pragma unroll
        for (int k = 0; k < 8; ++k) A[k] = fmaf(s_acc[k][threadIdx.x + 32 * COLS * j], f, A[k]);
      }
    }
  }
  if (group * 32 + (int)(threadIdx.x & 31) >= rows) return;
  const long long at = (long long)b * a.Hq * a.T + (long long)kvh * a.GT + gt;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + at * D + d8 * 8) =
      make_uint4(pack_bf16x2(A[0] * inv, A[1] * inv), pack_bf16x2(A[2] * inv, A[3] * inv),
                 pack_bf16x2(A[4] * inv, A[5] * inv), pack_bf16x2(A[6] * inv, A[7] * inv));
  if (a.lse != nullptr && d8 == 0) a.lse[at] = L != 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
}

}  // namespace td
