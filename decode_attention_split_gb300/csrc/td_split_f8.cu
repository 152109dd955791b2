// Split-KV attention over the block-scaled 8-bit cache (e4m3 codes, one fp32 scale per block of
// tokens and kv head).
//
//   out = sum_j p_j vs_j v_j / sum_j p_j,   p_j = 2^(scale log2(e) ks_j (q . k_j) - m)
// with codes k_j, v_j and the scales ks_j, vs_j of the blocks that hold row j. The method is the
// split attention of split_attn_mma_kernel, with the L2 warm-up before the wait for the previous
// kernel, the partial blocks and the fused merge of that kernel and a plan of its own.
//
// Bound by the codes' bytes at few query rows, and by the warps' latency at many. Measured (GPU time
// in a graph, inputs past L2): 3B-style layer, 32k keys, batch of 8, 79 us, 6.8 TB/s; ragged batch
// of 32 (277 MB) 48 us; verify chunk of six over 16k keys, batch of 8 (24 rows), 62 us, 4.3 TB/s; one
// sequence of 32k keys 15.1 us, of 4096 keys in the 360M-style layer 7.6 us (calls this short are a
// chain of launch, lengths, first stage, ticket and merge).
//
// Design:
//  * Stages of 128 rows of K and V cross by TMA as code tiles (128-byte swizzle for D = 128,
//    64-byte for D = 64); each of the 4 warps takes 32 keys of a stage. Half the bytes of bf16, so
//    the register work of a key counts: the tensor-core operands are taken from the code tiles by
//    ldmatrix (16-bit words, two codes), and one conversion turns two codes into the exact fp16
//    pair of their values (e4m3's range and precision lie inside fp16's).
//  * Keys lie on the m side of the products and the query rows of a row block on 1, 2 or 3 8-wide
//    n tiles, so a converted K or V fragment serves up to 24 rows (a verify chunk of 6 tokens of 4
//    grouped heads reads the cache once).
//  * A block holds at least 16 rows and a chunk starts at a multiple of 16, so the scales are
//    uniform over each 16-key half of a warp's step: the key scale multiplies the half's scores,
//    the value scale its p V product, in fp32, on the way into the running sums. Nothing of a
//    scale reaches the fp16 operands, so any scale is as good as another.
//  * The CTA that finishes a group's last segment merges its partials (finish_item); blocks of more
//    than 8 rows are merged by a second launch. Either way no CTA waits for another, so calls on
//    several streams cannot block one another.
//  * fp16 has 11 significant bits but a short range: a query row is first brought to a largest
//    element in [2^14, 2^15) by a power of two (undone with the scores' scale), and probabilities
//    are kept 2^7 above their usual place (at most 2^15). So fewer bits than fp32 are left to query
//    elements below 2^-28 of their row's largest, and to probabilities: 11 significant bits down to
//    2^-21 of the row's reference, an absolute 2^-32 of it below. The sum of a row's probabilities
//    is taken before that rounding. Outputs are as far from the exact ones as a formula in fp32's,
//    whose last rounding into bf16 is the coarser.
//  * A code may be NaN (a stored NaN or infinity; any byte behind a sequence's end). A step that
//    reaches a row's limit or the sequence's end zeroes the value codes past the end, and a NaN
//    value code that only some rows see is taken out of the tile and put into those rows' sums.
#include <algorithm>
#include <cfloat>
#include <mutex>

#include "td_f8.cuh"
#include "td_internal.h"
#include "td_split_mma.cuh"

namespace td {

namespace {

template <int D>
struct F8Cfg {
  static constexpr int NST = D == 128 ? 3 : 6;  // ring stages: two CTAs per SM
  static constexpr int TK = 128;                // keys per stage, 32 per warp
  static constexpr int CODE_BYTES = TK * D;     // one code tile
  static constexpr int STAGE_BYTES = 2 * CODE_BYTES;
  static constexpr int RING_BYTES = NST * STAGE_BYTES;
  static constexpr int Q_BYTES = kMaxTileRows * D * 2;  // query fragments of two or three n tiles
  static constexpr int SMEM_BYTES = RING_BYTES + Q_BYTES + 1024;  // + alignment slack
  static_assert(CODE_BYTES % 1024 == 0, "code tiles keep the swizzle's 1024-byte alignment");
  static_assert(kWarps * kMaxTileRows * (D + 6) * 4 + (2 + kWarps) * kMaxTileRows * 4 <= RING_BYTES, "combine area fits");
  static_assert((merge_fixed_floats<D, kMaxTileRows>() + part_block_floats(kMaxTileRows, D)) * 4 <= RING_BYTES,
                "merge stages at least one chunk");
  static_assert(SMEM_BYTES + 8704 <= 227 * 1024, "shared memory of a CTA");
};

// Powers of two that the probabilities are kept above their usual place by, for fp16's sake alone: the
// value scales take them off again, so the fp32 sums of p V hold values as large as the bf16 kernel's do
// (a value of 3e38 seen alone is the output), and the sums of p as they leave the CTA.
constexpr float kPShift = 7.f, kPUnit = 1.f / 128;

// Byte offset of 16-byte chunk `ch` of row `row` in a code tile of D-byte rows as the TMA unit
// writes it (128- or 64-byte swizzle): the 8 rows one ldmatrix reads fall in 8 bank groups.
template <int D>
__device__ __forceinline__ uint32_t code_swz(int row, int ch) {
  if constexpr (D == 128) {
    return (uint32_t)(row * 128 + ((ch ^ (row & 7)) << 4));
  } else {
    return (uint32_t)(row * 64 + ((ch ^ ((row >> 1) & 3)) << 4));
  }
}

struct F8Args {
  CUtensorMap kmap, vmap;  // codes [B*Hkv][Smax][D]
  SplitParams p;
};

__device__ __forceinline__ uint32_t lo_pair(uint32_t w) { return e4m3x2_f16x2((uint16_t)w); }
__device__ __forceinline__ uint32_t hi_pair(uint32_t w) { return e4m3x2_f16x2((uint16_t)(w >> 16)); }

// The bytes of w that are NaN codes (0x7f or 0xff), as 0x80 each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

__device__ __forceinline__ void add_scaled(float (&o)[4], const float (&x)[4], float s) {
  const float2 a = ffma2(make_float2(x[0], x[1]), make_float2(s, s), make_float2(o[0], o[1]));
  const float2 b = ffma2(make_float2(x[2], x[3]), make_float2(s, s), make_float2(o[2], o[3]));
  o[0] = a.x, o[1] = a.y, o[2] = b.x, o[3] = b.y;
}

// One warp's step over 32 keys (rows kr .. kr+31 of the code tiles kt / vt; keys key0 ..) for the
// NT * 8 query rows of the block. Fragment orders (mma m16n8k16, g = lane / 4, c = lane % 4):
//  - scores S^T = K Q^T: ldmatrix gives thread (g, c) codes 4c .. 4c+3 of a 16-dim block of keys g
//    and g + 8; they fill k slots 2c, 2c+1, 2c+8, 2c+9 of the A fragment, and the query fragments
//    qn hold the same dims in the same slots. sc[nt][hf] holds keys g, g + 8 of 16-key half hf
//    for rows 8 nt + 2c, + 1;
//  - O^T += V^T P^T: the transposed ldmatrix gives thread (g, c) dims 2g, 2g+1 of keys 2c, 2c+1;
//    with the middle bytes swapped the two conversions give dim 2g's pair (tile o[2i]) and dim
//    2g+1's (tile o[2i+1]). o[nt][2i] holds dims 32i + 2g and 32i + 16 + 2g of rows 8 nt + 2c, + 1,
//    o[nt][2i+1] the dims after them.
// Query fragments: qn in registers for one n tile; of more, q_mem in shared memory (8 bytes per tile,
// k step and lane), which leaves the registers to fragments in flight.
// ksc / vsc: the halves' scales (the values' times kPUnit); qs: the rows' score scale (base 2); lim: the rows' visible keys
// (index 2 nt + e). masked: some key lies past a row's limit; the values that it must not see whatever
// they are have gone by then (clear_tail, mark_nans).
template <int D, int NT>
__device__ __forceinline__ void warp_keys32_f8(const uint32_t (&qn)[1][D / 16][2], const uint2 *q_mem,
                                               uint32_t kt, uint32_t vt, int kr,
                                               int key0, bool masked, const int (&lim)[2 * NT], const float (&qs)[2 * NT],
                                               const float (&ksc)[2], const float (&vsc)[2],
                                               float (&o)[NT][D / 16][4], float (&m_run)[2 * NT],
                                               float (&l_run)[2 * NT]) {
  constexpr int NX = D / 32;  // ldmatrix.x4 per 16 keys: 16 keys x 32 dims
  const int lane = threadIdx.x & 31, gid = lane >> 2;
  const int lrow = kr + (lane & 7) + ((lane >> 3) & 1) * 8, lch = lane >> 4;
  float sc[NT][2][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) sc[nt][hf][0] = sc[nt][hf][1] = sc[nt][hf][2] = sc[nt][hf][3] = 0.f;
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    uint32_t qf[NT][2][2];  // the query fragments of dims 32i .. 32i+31
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        if constexpr (NT == 1) {
          qf[nt][blk][0] = qn[nt][2 * i + blk][0], qf[nt][blk][1] = qn[nt][2 * i + blk][1];
        } else {
          const uint2 w = q_mem[(nt * (D / 16) + 2 * i + blk) * 32 + lane];
          qf[nt][blk][0] = w.x, qf[nt][blk][1] = w.y;
        }
      }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t r[4];  // keys 0-7 / 8-15 of dims 32i .. 32i+15, then of dims 32i+16 .. 32i+31
      ldmatrix_x4(r, kt + code_swz<D>(lrow + 16 * hf, 2 * i + lch));
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint32_t ak[4] = {lo_pair(r[2 * blk]), lo_pair(r[2 * blk + 1]), hi_pair(r[2 * blk]),
                                hi_pair(r[2 * blk + 1])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(sc[nt][hf], ak, qf[nt][blk][0], qf[nt][blk][1]);
      }
    }
  }
  // Online softmax with a lazy reference maximum (see warp_keys16): it moves when some key of the
  // warp rises more than kMaxGap above its row's, which one vote finds; only then are the rows'
  // maxima reduced over their 8 lanes and the sums rescaled. The score scales are not negative.
  float kss[2 * NT][2], top[2 * NT];
#pragma unroll
  for (int ri = 0; ri < 2 * NT; ++ri) kss[ri][0] = ksc[0] * qs[ri], kss[ri][1] = ksc[1] * qs[ri];
  if (masked) {
#pragma unroll
    for (int ri = 0; ri < 2 * NT; ++ri)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        // a normal number, so that -inf times it stays -inf; of a score it leaves nothing
        if (kss[ri][hf] < FLT_MIN) kss[ri][hf] = FLT_MIN;
#pragma unroll
        for (int hk = 0; hk < 2; ++hk)
          if (key0 + 16 * hf + 8 * hk + gid >= lim[ri]) sc[ri / 2][hf][2 * hk + (ri & 1)] = -INFINITY;
      }
  }
  bool over = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int ri = 2 * nt + e;
      float half_top[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) half_top[hf] = fmaxf(sc[nt][hf][e], sc[nt][hf][2 + e]) * kss[ri][hf];
      top[ri] = fmaxf(half_top[0], half_top[1]);
      over |= top[ri] > m_run[ri] + kMaxGap;
    }
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int ri = 2 * nt + e;
        float mx = fmaxf(top[ri], __shfl_xor_sync(0xffffffffu, top[ri], 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const bool move = mx > m_run[ri] + kMaxGap;
        alpha[e] = move ? exp2_approx(m_run[ri] - mx) : 1.f;
        if (move) m_run[ri] = mx;
        l_run[ri] *= alpha[e];
      }
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        o[nt][t][0] *= alpha[0];
        o[nt][t][1] *= alpha[1];
        o[nt][t][2] *= alpha[0];
        o[nt][t][3] *= alpha[1];
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int ri = 2 * nt + e;
      const float base = m_run[ri] == -INFINITY ? 0.f : m_run[ri] - kPShift;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int hk = 0; hk < 2; ++hk) {
          float &x = sc[nt][hf][2 * hk + e];
          x = exp2_approx(fmaf(x, kss[ri][hf], -base));
        }
      // this thread's keys; lanes summed at the end
      l_run[ri] += (sc[nt][0][e] + sc[nt][0][2 + e]) + (sc[nt][1][e] + sc[nt][1][2 + e]);
    }
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    // P^T as B operands: keys 2c, 2c+1 (+8) of row 8 nt + g
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      pb[nt][0] = movmatrix_trans(pack_f16x2(sc[nt][hf][0], sc[nt][hf][1]));
      pb[nt][1] = movmatrix_trans(pack_f16x2(sc[nt][hf][2], sc[nt][hf][3]));
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      uint32_t r[4];  // transposed: keys 0-7 / 8-15 of dims 32i .. 32i+15, then of 32i+16 ..
      ldmatrix_x4_trans(r, vt + code_swz<D>(lrow + 16 * hf, 2 * i + lch));
#pragma unroll
      for (int x = 0; x < 4; ++x) r[x] = __byte_perm(r[x], 0u, 0x3120);  // the middle bytes swapped
      const uint32_t ae[4] = {lo_pair(r[0]), lo_pair(r[2]), lo_pair(r[1]), lo_pair(r[3])};
      const uint32_t ao[4] = {hi_pair(r[0]), hi_pair(r[2]), hi_pair(r[1]), hi_pair(r[3])};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float te[4] = {0.f, 0.f, 0.f, 0.f}, to[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16_16816(te, ae, pb[nt][0], pb[nt][1]);
        mma_f16_16816(to, ao, pb[nt][0], pb[nt][1]);
        add_scaled(o[nt][2 * i], te, vsc[hf]);
        add_scaled(o[nt][2 * i + 1], to, vsc[hf]);
      }
    }
  }
}

// One warp's values of a step that some row does not see whole (rows kr .. kr+31 of the tile vt, keys
// key0 ..): zeros in place of the rows from key c1 on, whose bytes may be anything. True if a value
// that some rows see and others do not, of keys [lim_all, c1), holds a NaN code, for mark_nans.
// The step itself is one for whole and cut tiles: with one of its own for cut tiles the first CTA of
// an SM that came to one waited for its instructions (one sequence, 8 kv heads, D = 128: 500 keys 7.6
// -> 6.4 us, 4060 keys 8.7 -> 7.7; verify of six after 300, 14.4 -> 11.7).
template <int D>
__device__ __forceinline__ bool clear_tail(uint32_t vt, int kr, int key0, int lim_all, int c1) {
  constexpr int CH = D / 16;  // 16-byte chunks of a row, in some order
  const int lane = threadIdx.x & 31;
  bool nan = false;
#pragma unroll 1
  for (int r = max(lim_all - key0, 0) + lane / CH; r < 32; r += 32 / CH) {
    const uint32_t at = vt + (kr + r) * D + (lane % CH) * 16;
    uint4 w;
    if (key0 + r >= c1) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
    } else {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
      nan |= (nan_bytes(w.x) | nan_bytes(w.y) | nan_bytes(w.z) | nan_bytes(w.w)) != 0u;
    }
  }
  nan = __any_sync(0xffffffffu, nan);
  __syncwarp();
  return nan;
}

// The NaN codes among the values of keys [lim_all, c1) of a step: NaN in the sums of the rows that see
// them, and zeros in their place for the rows that do not.
template <int D, int NT>
__device__ __forceinline__ void mark_nans(uint32_t vt, int kr, int key0, int lim_all, int c1, const int (&lim)[2 * NT],
                                          float (&o)[NT][D / 16][4]) {
  const int lane = threadIdx.x & 31, gid = lane >> 2;
#pragma unroll 1
  for (int r = max(lim_all - key0, 0); r < min(c1 - key0, 32); ++r) {
    // this thread's dims 32 i + 16 h + 2 g, + 1: those of its o
    uint16_t w[D / 16];
#pragma unroll
    for (int x = 0; x < D / 16; ++x)
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w[x]) : "r"(vt + code_swz<D>(kr + r, x) + 2 * gid) : "memory");
    __syncwarp();
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      const uint32_t n = nan_bytes(w[x]);
      if ((n & 0x8080u) == 0u) continue;
#pragma unroll
      for (int ri = 0; ri < 2 * NT; ++ri)
        if (key0 + r < lim[ri]) {
          if (n & 0x80u) o[ri / 2][x & ~1][2 * (x & 1) + (ri & 1)] = __uint_as_float(0x7fffffffu);
          if (n & 0x8000u) o[ri / 2][x | 1][2 * (x & 1) + (ri & 1)] = __uint_as_float(0x7fffffffu);
        }
      const uint16_t kept = (uint16_t)(w[x] & ~((n >> 7) * 0xffu));
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(vt + code_swz<D>(kr + r, x) + 2 * gid), "h"(kept) : "memory");
    }
  }
  fence_proxy_async_smem();  // the stage may not be the last of its buffer
  __syncwarp();
}

// Streams keys [c0, c1) of (b, kvh) for row block rb, as stream_chunk does for bf16 caches,
// leaving the same combine area (at the start of `smem`), 8 NT rows per warp. c0 is a multiple of
// 16. False, CTA-uniformly, if a copy never completed.
template <int D, int NT>
__device__ bool stream_chunk_f8(const F8Args &a, unsigned char *smem, uint64_t *s_bars, uint32_t &seq, int b, int kvh,
                                int rb, int L, int c0, int c1) {
  using C = F8Cfg<D>;
  constexpr int NST = C::NST, TR = 8 * NT;
  const SplitParams &p = a.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const uint32_t sbase = smem_u32(smem);
  const int GT = p.G * p.T;
  const int nstages = (c1 - c0 + C::TK - 1) / C::TK;
  const int zc = b * p.Hkv + kvh;
  const uint64_t policy = l2_evict_first_policy();

  auto issue = [&](int sidx) {
    const int buf = (seq + sidx) % NST;
    const uint32_t bar = smem_u32(&s_bars[buf]);
    const uint32_t dst = sbase + buf * C::STAGE_BYTES;
    const int y = c0 + sidx * C::TK;
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
    tma_load_3d(dst, &a.kmap, 0, y, zc, bar, policy);
    tma_load_3d(dst + C::CODE_BYTES, &a.vmap, 0, y, zc, bar, policy);
  };
  // this thread's share of query rows 8 nt + g, asked for ahead of the stages: behind them, in a full
  // memory system, they took 5 us to come
  uint2 q[NT][D / 16];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + gid, gr = rb * p.R + r;
    const bool valid = r < p.R && gr < GT;
    const int hq = kvh * p.G + (valid ? gr / p.T : 0), t = valid ? gr % p.T : 0;
    const uint2 *qrow = reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.q) +
                                                        (((size_t)b * p.Hq + hq) * p.T + t) * D);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) q[nt][ks] = valid ? qrow[ks * 4 + tig] : make_uint2(0u, 0u);
  }
  if (tid == 0) {
    for (int s2 = 0; s2 < min(NST - 1, nstages); ++s2) issue(s2);
  }
  // lanes 0 .. 3 fetch the scales of this warp's two 16-key halves of a stage (K, then V), one
  // stage ahead of their use; a half past the chunk's end reads none
  const float *scales = (lane & 2 ? p.v_scales : p.k_scales) + (size_t)zc * p.n_blocks;
  auto load_scale = [&](int st) -> float {
    const int key = c0 + st * C::TK + warp * 32 + (lane & 1) * 16;
    return lane < 4 && st < nstages && key < c1 ? __ldcg(scales + (key >> p.block_log2)) : 0.f;
  };
  float s_next = load_scale(0);

  // query row 8 nt + g of this block as fp16 B fragments (slots 2c, 2c+1 <- dims 4c, 4c+1; slots
  // 2c+8, 2c+9 <- dims 4c+2, 4c+3), brought to a largest element in [2^14, 2^15); the limits and
  // score scales of rows 8 nt + 2c, + 1
  uint32_t qn[1][D / 16][2];
  uint2 *q_mem = reinterpret_cast<uint2 *>(smem + C::RING_BYTES);
  int lim[2 * NT];
  float qs[2 * NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t top = 0;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint2 w = q[nt][ks];
      top = max(max(top, w.x & 0x7fffu), (w.x >> 16) & 0x7fffu);
      top = max(max(top, w.y & 0x7fffu), (w.y >> 16) & 0x7fffu);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // exponent of the row's largest element (a bf16's 8 exponent bits); rows of zeros and rows
    // with an infinity or NaN stay as they are
    const int ex = (int)(top >> 7);
    const int k = top == 0u || ex == 255 ? 0 : min(14 - (ex - 127), 126);
    // (the sign of the scale goes with the query, so the scores' scales are not negative)
    const float up = copysignf(__uint_as_float((uint32_t)(127 + k) << 23), p.qscale);
    const float down = __uint_as_float((uint32_t)(127 - k) << 23);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      float f[4];
      widen_bf16x2(q[nt][ks].x, f[0], f[1]);
      widen_bf16x2(q[nt][ks].y, f[2], f[3]);
      const uint2 w2 = make_uint2(pack_f16x2(f[0] * up, f[1] * up), pack_f16x2(f[2] * up, f[3] * up));
      if constexpr (NT == 1)
        qn[nt][ks][0] = w2.x, qn[nt][ks][1] = w2.y;
      else if (warp == ks % kWarps)
        q_mem[(nt * (D / 16) + ks) * 32 + lane] = w2;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      qs[2 * nt + e] = fabsf(p.qscale) * __shfl_sync(0xffffffffu, down, 4 * (2 * tig + e));
      const int lr = 8 * nt + 2 * tig + e, lgr = rb * p.R + lr;
      lim[2 * nt + e] = lr < p.R && lgr < GT ? min(max(L - p.T + lgr % p.T + 1, 0), c1) : 0;
    }
  }
  // keys every row of the block sees: the limit of its first token (token 0 if the rows wrap)
  const int first = (rb * p.R) % p.T, rows = min(p.R, GT - rb * p.R);
  const int lim_all = min(c1, max(L - p.T + (first + rows > p.T ? 0 : first) + 1, 0));
  float o[NT][D / 16][4];
  float m_run[2 * NT], l_run[2 * NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[nt][t][0] = o[nt][t][1] = o[nt][t][2] = o[nt][t][3] = 0.f;
#pragma unroll
  for (int h = 0; h < 2 * NT; ++h) m_run[h] = -INFINITY, l_run[h] = 0.f;

  int consumed = 0;
  bool ok = true;
  for (int st = 0; st < nstages; ++st) {
    const float s_mine = s_next;
    s_next = load_scale(st + 1);
    const int buf = (seq + st) % NST;
    const bool landed = mbar_wait_bounded(smem_u32(&s_bars[buf]), ((seq + st) / NST) & 1u);
    // every warp has finished the previous stage, whose buffer is refilled next; one decision
    // for the whole CTA
    if (!__syncthreads_and(landed)) {
      ok = false;
      break;
    }
    if (tid == 0 && st + NST - 1 < nstages) issue(st + NST - 1);
    const int kr = warp * 32, key0 = c0 + st * C::TK + kr;
    if (key0 < c1) {
      const uint32_t kt = sbase + buf * C::STAGE_BYTES, vt = kt + C::CODE_BYTES;
      const float ksc[2] = {__shfl_sync(0xffffffffu, s_mine, 0), __shfl_sync(0xffffffffu, s_mine, 1)};
      const float vsc[2] = {kPUnit * __shfl_sync(0xffffffffu, s_mine, 2), kPUnit * __shfl_sync(0xffffffffu, s_mine, 3)};
      const bool masked = key0 + 32 > lim_all;
      if (masked && clear_tail<D>(vt, kr, key0, lim_all, c1))
        mark_nans<D, NT>(vt, kr, key0, lim_all, c1, lim, o);
      warp_keys32_f8<D, NT>(qn, q_mem, kt, vt, kr, key0, masked, lim, qs, ksc, vsc, o, m_run, l_run);
    }
    consumed = st + 1;
  }
  if (!ok) {
    const int issued = min(nstages, consumed + NST - 1);
    for (int st = consumed; st < issued; ++st)
      mbar_wait_bounded(smem_u32(&s_bars[(seq + st) % NST]), ((seq + st) / NST) & 1u);
    if (tid == 0) report(p.status, TD_DEV_WAIT_TIMEOUT);
#pragma unroll
    for (int h = 0; h < 2 * NT; ++h) m_run[h] = -INFINITY, l_run[h] = 0.f;
  }
  seq += nstages;
#pragma unroll
  for (int h = 0; h < 2 * NT; ++h) {
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 4);
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 8);
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 16);
  }
  __syncthreads();  // ring idle: reuse it as the combine area
  float *cm = reinterpret_cast<float *>(smem);
  float *cl = cm + kWarps * TR;
  float *ca = cm + 2 * kWarps * TR;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * tig + e, ri = 2 * nt + e;
      if (gid == 0) {
        // a row that saw a NaN key: the merges drop partials whose sum is not positive, so it is
        // given a sum and a maximum that outweigh every other partial's
        const bool bad = isnan(l_run[ri]);
        cm[warp * TR + r] = bad ? 3e38f : m_run[ri];
        cl[warp * TR + r] = bad ? INFINITY : l_run[ri] * kPUnit;
      }
      float *row = &ca[(warp * TR + r) * combine_stride<D>()];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        *reinterpret_cast<float2 *>(&row[32 * i + 2 * gid]) = make_float2(o[nt][2 * i][e], o[nt][2 * i + 1][e]);
        *reinterpret_cast<float2 *>(&row[32 * i + 16 + 2 * gid]) =
            make_float2(o[nt][2 * i][2 + e], o[nt][2 * i + 1][2 + e]);
      }
    }
  __syncthreads();
  return ok;
}

// Four dims of an output row and, with its first, the row's lse.
template <int D>
__device__ __forceinline__ void store_row_f8(const SplitParams &p, long long row, int d, float4 A, float M, float Ls) {
  const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
  __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + row * D + d;
  *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(A.x * inv, A.y * inv), pack_bf16x2(A.z * inv, A.w * inv));
  if (d == 0 && p.lse != nullptr) p.lse[row] = Ls > 0.f ? (M + log2f(Ls)) * kLn2 : -INFINITY;
}

// Leaves a segment's result: the four warps' partials combined, to out and lse if it is its group's
// only one, else as the group's partial block c (the first is `first`) for merge_f8_kernel. Segment 0
// also leaves the group's entry of p.pieces, whatever their number. Ends with a barrier.
template <int D, int ROWS>
__device__ void publish_f8(const SplitParams &p, const float *combine, int b, int kvh, int rb, int c, int NC,
                           long long first) {
  constexpr int D4 = D / 4, RF = part_row_floats(D), CAS = combine_stride<D>();
  const float *cm = combine, *cl = combine + kWarps * ROWS, *ca = combine + 2 * kWarps * ROWS;
  const int nv = min(p.R, p.G * p.T - rb * p.R);  // rows of this block that exist
  const long long g = ((long long)b * p.Hkv + kvh) * p.RB + rb;
  float *blk = p.ws_part + (first + c) * (long long)part_block_floats(p.R, D);
  if (c == 0 && threadIdx.x == 0) p.pieces[g] = make_int2((int)first, NC);
#pragma unroll 1
  for (int idx = threadIdx.x; idx < nv * D4; idx += kThreads) {
    const int r = idx / D4, d = (idx % D4) * 4;
    float M = -INFINITY, Ls = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, cm[w * ROWS + r]);
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = cm[w * ROWS + r];
      const float f = mw == -INFINITY ? 0.f : exp2f(mw - M);
      const float4 v = *reinterpret_cast<const float4 *>(ca + (w * ROWS + r) * CAS + d);
      Ls = fmaf(cl[w * ROWS + r], f, Ls);
      A.x = fmaf(v.x, f, A.x), A.y = fmaf(v.y, f, A.y), A.z = fmaf(v.z, f, A.z), A.w = fmaf(v.w, f, A.w);
    }
    if (NC == 1) {
      store_row_f8<D>(p, out_row_of(p, b, kvh, rb, r), d, A, M, Ls);
    } else {
      *reinterpret_cast<float4 *>(blk + r * RF + d) = A;
      if (d == 0) *reinterpret_cast<float2 *>(blk + r * RF + D) = make_float2(Ls > 0.f ? M : -INFINITY, Ls);
    }
  }
  __syncthreads();
}

// Log-sum-exp merge of the partial blocks that publish_f8 left, one warp per query row of every
// group of more than one: its lanes hold the blocks' maxima and sums (32 a pass), then four dims of
// the weighted sum. Launched after the attention for row blocks of more than 8 rows: the CTA that
// finished such a group last would merge it alone, row after row, while the others have ended
// (24 rows: 4 us of 5 blocks, 8 of 13, 25 of 38). No CTA waits for another.
constexpr int kMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32, 4) merge_f8_kernel(const SplitParams p) {
  constexpr int RF = part_row_floats(D), PER = D / 32;  // PER: dims of a lane
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int g = blockIdx.x, rb = g % p.RB, kvh = g / p.RB % p.Hkv, b = g / p.RB / p.Hkv;
  if (r >= min(p.R, p.G * p.T - rb * p.R)) return;
  const int BF = part_block_floats(p.R, D);
  uint32_t bits = 0;
  const int L = attended_len(p, p.seq_lens[b], bits);
  // this call's if the sequence has keys and no copy timed out, which leaves a group unpublished
  const int2 piece = __ldcg(p.pieces + g);
  const int first = min(max(piece.x, 0), p.n_part), NC = min(max(piece.y, 0), p.n_part - first);
  if (L == 0 || NC == 1) return;
  const float *row = p.ws_part + (long long)first * BF + r * RF;
  float M = -INFINITY, Ls = 0.f;
  float acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int c0 = 0; c0 < NC; c0 += 32) {
    const int nb = min(32, NC - c0);
    const float *src = row + (long long)c0 * BF;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < nb) ml = __ldcg(reinterpret_cast<const float2 *>(src + (long long)lane * BF + D));
    const bool some = ml.y > 0.f;
    float Mn = some ? fmaxf(M, ml.x) : M;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
    const float base = Mn == -INFINITY ? 0.f : Mn;
    const float f = some ? exp2f(ml.x - base) : 0.f, a = exp2f(M - base);
    float ls = some ? ml.y * f : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
    Ls = Ls * a + ls;
    M = Mn;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= a;
#pragma unroll 8
    for (int c = 0; c < nb; ++c) {
      const float w = __shfl_sync(0xffffffffu, f, c);
      const float *v = src + (long long)c * BF + lane * PER;
      if constexpr (PER == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(v));
        acc[0] = fmaf(x.x, w, acc[0]), acc[1] = fmaf(x.y, w, acc[1]);
        acc[2] = fmaf(x.z, w, acc[2]), acc[3] = fmaf(x.w, w, acc[3]);
      } else {
        const float2 x = __ldcg(reinterpret_cast<const float2 *>(v));
        acc[0] = fmaf(x.x, w, acc[0]), acc[1] = fmaf(x.y, w, acc[1]);
      }
    }
  }
  const long long orow = out_row_of(p, b, kvh, rb, r);
  const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + orow * D + lane * PER;
  if constexpr (PER == 4)
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[orow] = Ls > 0.f ? (M + log2f(Ls)) * kLn2 : -INFINITY;
}

// How work is cut. A split the caller chose: chunks of that size, an item per chunk (plan_items).
// Else whole groups (see kMergeStages) or runs: the stages of 128 keys of every group (sequence, kv head, row block), one group after
// another, cut into equal runs, one per CTA, whatever the lengths. Starting and finishing a segment
// of a group takes a CTA about as long as kSegmentStages stages, so each group counts that many
// units more, ahead of its own. Measured, ragged batch of 32 (256 groups of 1 to 8192 keys,
// D = 128): plan_items' automatic chunks 68 us; runs without those units 68 (the CTAs that hold
// several short groups end last), with 1, 2, 3, 4 of them 63, 57, 56, 56; 48 once the runs' plan,
// one pass over the lengths, was made ahead of the wait for the previous kernel (plan_items' rounds
// took 5 us after it). One sequence of 16384 keys and 8 kv heads: chunks 11.6 us, runs 11.1.
constexpr int kSegmentStages = 3;

// A run that ends inside a group costs the merge of its pieces, about kMergeStages stages; and of long
// runs memory is the bound, which four fifths of the CTAs reach as well as all. So each CTA takes whole
// groups while the longest is at most an equal run and kMergeStages, and in one round of CTAs a
// quarter of a run more (in more than two rounds never: 1024 groups of 1024 keys took 52.5 us whole
// and 49.2 in runs). Measured, runs / whole groups, D =
// 128, 8 kv heads: one sequence of 256 keys 7.0 / 5.2 us, of 512 7.1 / 6.5, of 768 7.1 / 8.1; 32
// sequences of 512 keys 15.9 / 11.6, of 2048 27.9 / 25.3, of 8192 83.2 / 79.9; 8 of 1024 11.0 / 12.2;
// 20 of 4096 33.1 / 34.8. 5 kv heads, D = 64: 64 sequences (two rounds) of 256 12.5 / 10.8, of 512
// 15.1 / 14.3; 56 of 32768 190.5 / 183.2.
// Blocks of more than 8 rows are always cut: their stages take longer, their merge is spread over the GPU
// by its own launch, and the same rule would lose more than it gains (runs / whole groups, verify of six,
// 32 query and 8 kv heads, D = 128: one sequence of 256 keys 11.4 / 13.0 us, of 500 12.2 / 15.1; 8 of 512
// 16.1 / 18.2; 32 of 512 25.3 / 21.2, of 2048 41.1 / 38.8, of 8192 101 / 109).
constexpr int kMergeStages = 7;

// Units of a group of L keys.
__device__ __forceinline__ int group_units(int L) {
  constexpr int TK = F8Cfg<128>::TK;
  return L > 0 ? (L + TK - 1) / TK + kSegmentStages : 0;
}

// Units of a run, or 0 for whole groups: W units in all, the longest group Kmax.
__device__ __forceinline__ int run_units(const SplitParams &p, int W, int Kmax) {
  const unsigned S = max((W + (int)gridDim.x - 1) / (int)gridDim.x, 1), rounds = p.rounds;
  return rounds != 0 && rounds * Kmax <= S + kMergeStages + (rounds == 1 ? S / 4 : 0) ? 0 : (int)S;
}

// Fills s_len (attended lengths) and s_prefix (units, or whole groups, before each sequence; their
// total at [B]) and returns the units of a run, 0 for whole groups. report_bits as for plan_items.
// Ends with a barrier.
__device__ int plan_runs(const SplitParams &p, int *s_len, int *s_prefix, int *s_red, bool report_bits) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int U = p.Hkv * p.RB, per = (p.B + kThreads - 1) / kThreads, b0 = tid * per;
  int seg = 0, top = 0;
  uint32_t bits = 0;
  for (int b = b0; b < min(b0 + per, p.B); ++b) {
    const int L = attended_len(p, report_bits ? p.seq_lens[b] : ld_relaxed(p.seq_lens + b), bits);
    s_len[b] = L;
    seg += group_units(L) * U;
    top = max(top, group_units(L));
  }
  if (report_bits && blockIdx.x == 0) report(p.status, bits);
  int incl = seg;
  top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // s_red may still be read by an earlier plan
  if (lane == 31) s_red[warp] = incl, s_red[kWarps + warp] = top;
  __syncthreads();
  int W = 0, before = incl - seg;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_red[w];
    W += s_red[w];
    top = max(top, s_red[kWarps + w]);
  }
  const int S = run_units(p, W, top);
  for (int b = b0; b < min(b0 + per, p.B); ++b) {
    s_prefix[b] = S > 0 ? before : b * U;
    before += group_units(s_len[b]) * U;
  }
  if (tid == 0) s_prefix[p.B] = S > 0 ? W : p.B * U;
  __syncthreads();
  return S;
}

// Run by one thread before the wait for the previous kernel: warms L2 with the start of this CTA's
// run, as prefetch_first_item does for chunks, on a guess of the lengths. Batches of up to 8.
template <int D>
__device__ void prefetch_first_run(const SplitParams &p) {
  constexpr int TK = F8Cfg<D>::TK;
  if (p.B > 8) return;
  const int U = p.Hkv * p.RB;
  int len[8], W = 0, top = 0;
  uint32_t bits = 0;
#pragma unroll
  for (int b = 0; b < 8; ++b) len[b] = b < p.B ? attended_len(p, ld_relaxed(p.seq_lens + b), bits) : 0;
#pragma unroll
  for (int b = 0; b < 8; ++b) W += group_units(len[b]) * U, top = max(top, group_units(len[b]));
  const int run = run_units(p, W, top);
  if (run == 0) {
    const int b = blockIdx.x / U, L = b < p.B ? attended_len(p, ld_relaxed(p.seq_lens + b), bits) : 0;
    if (L > 0) prefetch_chunk_l2<D, kWarmF8>(p, b, blockIdx.x % U / p.RB, 0, L, prefetch_stages(p));
    return;
  }
  int at = min(blockIdx.x * (long long)run, (long long)W);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const int K = group_units(len[b]);
    if (at >= 0 && at < K * U) {
      const int st = max(at % K - kSegmentStages, 0), kvh = at / K / p.RB;
      prefetch_chunk_l2<D, kWarmF8>(p, b, kvh, st * TK, min((st + run) * TK, len[b]), prefetch_stages(p));
    }
    at -= K * U;
  }
}

// The last sequence b with s_prefix[b] <= at.
__device__ __forceinline__ int sequence_of(const int *s_prefix, int B, int at) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_prefix[mid] <= at) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// First partial block of group g, which has some. A caller's split: [B, Hkv, RB][ns_ws]. Runs: a group's
// segment c lies in run f + c, f the run of its first stage, and starts at block f + min(f, g) + c. A group
// that is cut has two segments or more, so for the next one cut f has grown by at least one less than
// their number and min(f, g) by at least one: no block is shared, and grid + min(grid, groups) hold all
// (64 sequences, 8 kv heads, 24 rows: 7.7 MB, where ns_ws for every group took 253).
__device__ __forceinline__ long long first_block(const SplitParams &p, bool runs, int g, int c) {
  const int f = (int)blockIdx.x - c;
  return runs ? f + min(f, g) : (long long)g * p.ns_ws;
}

// Persistent kernel over a block-scaled cache: the items, chunks and fused merge of
// split_attn_mma_kernel, or runs.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 2) split_attn_f8_kernel(const __grid_constant__ F8Args a) {
  using C = F8Cfg<D>;
  using E = __nv_bfloat16;
  constexpr int NST = C::NST, TR = 8 * NT;
  const SplitParams &p = a.p;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ int s_len[TD_MAX_BATCH];
  __shared__ int s_prefix[TD_MAX_BATCH + 1];
  __shared__ long long s_red[2 * kWarps];
  __shared__ int s_chunk, s_last, s_sum[2 * kWarps];
  __shared__ __align__(8) uint64_t s_merge_bar;
  __shared__ __align__(8) uint64_t s_bars[NST];

  const int tid = threadIdx.x;
  unsigned char *smem = align1024(smem_raw);
  float *combine = reinterpret_cast<float *>(smem);
  if (tid == 0) {
    mbar_init(smem_u32(&s_merge_bar), 1);
#pragma unroll
    for (int i = 0; i < NST; ++i) mbar_init(smem_u32(&s_bars[i]), 1);
    fence_mbar_init();
  }
  uint32_t merge_phase = 0;
  uint32_t seq = 0;
  if (tid == 0) {
    if (p.runs)
      prefetch_first_run<D>(p);
    else
      prefetch_first_item<D, kWarmF8>(p, prefetch_stages(p), blockIdx.x);
  }
  // the plan is made before the wait for the previous kernel, on the lengths as they read then, and
  // kept if they read the same after it
  int S = 0;  // keys of a chunk, or units of a run
  if (p.runs)
    S = plan_runs(p, s_len, s_prefix, s_sum, false);
  else
    plan_items(p, s_len, s_prefix, &s_chunk, s_red, false);
  griddep_wait();  // inputs may come from the previous kernel in the stream
  griddep_launch_dependents();
  if (!lengths_unchanged(p, s_len)) {
    if (p.runs)
      S = plan_runs(p, s_len, s_prefix, s_sum, true);
    else
      plan_items(p, s_len, s_prefix, &s_chunk, s_red);
  }
  const bool runs = S > 0;
  if (!runs) S = p.runs ? p.Smax : s_chunk;  // a whole group is a chunk that holds every key
  const int W = s_prefix[p.B];
  const int rows = p.Hq * p.T;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (s_len[b] != 0) continue;
    for (long long idx = tid; idx < (long long)rows * D; idx += kThreads)
      store_elem<E>(static_cast<E *>(p.out) + (long long)b * rows * D + idx, 0.f);
    if (p.lse != nullptr)
      for (int r = tid; r < rows; r += kThreads) p.lse[(long long)b * rows + r] = -INFINITY;
  }
  // chunks: items blockIdx.x, + gridDim.x, ...; runs: segments of stages [at, end)
  int at = runs ? min((long long)blockIdx.x * S, (long long)W) : blockIdx.x;
  const int end = runs ? min((long long)at + S, (long long)W) : W;
  while (at < end) {
    const int b = sequence_of(s_prefix, p.B, at);
    const int L = s_len[b];
    const int local = at - s_prefix[b];
    int unit, c, NC, c0, c1;
    if (runs) {
      const int K = group_units(L);
      unit = local / K;
      const int in = local % K, n = min(end - at, K - in);
      const int first = at - in + kSegmentStages, last = at - in + K - 1;  // units of the group's stages
      at += n;
      if (in + n <= kSegmentStages) continue;  // the run ends ahead of the group's first stage
      c = (int)blockIdx.x - first / S;
      NC = last / S - first / S + 1;
      c0 = max(in - kSegmentStages, 0) * C::TK;
      c1 = min((in + n - kSegmentStages) * C::TK, L);
    } else {
      if (L == 0) {  // only whole groups are counted for an empty sequence
        at += gridDim.x;
        continue;
      }
      NC = (L + S - 1) / S;
      unit = local / NC;
      c = local % NC;
      c0 = c * S;
      c1 = min(c0 + S, L);
      at += gridDim.x;
    }
    const int rb = unit % p.RB, kvh = unit / p.RB;
    const bool ok = stream_chunk_f8<D, NT>(a, smem, s_bars, seq, b, kvh, rb, L, c0, c1);
    const long long first = NC > 1 ? first_block(p, runs, b * p.Hkv * p.RB + unit, c) : 0;
    if (p.merge_apart)
      publish_f8<D, TR>(p, combine, b, kvh, rb, c, NC, first);
    else
      finish_item<E, D, TR, kWarps, combine_stride<D>()>(p, combine, C::RING_BYTES / 4, &s_merge_bar, merge_phase, b, kvh,
                                                         rb, c, NC, &s_last, false, first);
    fence_proxy_async_smem();
    __syncthreads();
    if (!ok) break;
  }
}

template <int D>
const void *kernel_of(int nt) {
  return nt == 1   ? reinterpret_cast<const void *>(&split_attn_f8_kernel<D, 1>)
         : nt == 2 ? reinterpret_cast<const void *>(&split_attn_f8_kernel<D, 2>)
                   : reinterpret_cast<const void *>(&split_attn_f8_kernel<D, 3>);
}

bool encode_code_map(CUtensorMap *m, const void *base, const SplitParams &p, int D) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint32_t estr[3] = {1, 1, 1};
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.Smax, (cuuint64_t)p.B * p.Hkv};
  const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)p.Smax * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)F8Cfg<128>::TK, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const SplitPlan &plan, const SplitParams &p, cudaStream_t stream) {
  constexpr int kMaxDevices = 64;
  F8Args a;
  if (!encode_code_map(&a.kmap, p.k, p, D) || !encode_code_map(&a.vmap, p.v, p, D)) return cudaErrorInvalidValue;
  a.p = p;
  a.p.runs = plan.runs;
  a.p.merge_apart = plan.merge_apart;
  const long long rounds = ((long long)p.B * p.Hkv * p.RB + plan.grid - 1) / plan.grid;
  a.p.rounds = plan.merge_apart || rounds > 2 ? 0 : (int)rounds;
  {
    // every instantiation's shared-memory opt-in, once per device
    static std::mutex mu;
    static bool done[kMaxDevices] = {};
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[device]) {
      for (int nt = 1; nt <= 3; ++nt) {
        const cudaError_t e = cudaFuncSetAttribute(kernel_of<D>(nt), cudaFuncAttributeMaxDynamicSharedMemorySize, plan.smem);
        if (e != cudaSuccess) return e;
      }
      done[device] = true;
    }
  }
  const dim3 grid(plan.grid), block(kThreads);
  cudaError_t e;
  if (p.R <= 8)
    e = launch_pdl(split_attn_f8_kernel<D, 1>, grid, block, plan.smem, stream, a);
  else if (p.R <= 16)
    e = launch_pdl(split_attn_f8_kernel<D, 2>, grid, block, plan.smem, stream, a);
  else
    e = launch_pdl(split_attn_f8_kernel<D, 3>, grid, block, plan.smem, stream, a);
  if (e == cudaSuccess && a.p.merge_apart)
    e = launch_pdl(merge_f8_kernel<D>, dim3((unsigned)(p.B * p.Hkv * p.RB), (p.R + kMergeWarps - 1) / kMergeWarps),
                   dim3(kMergeWarps * 32), 0, stream, a.p);
  return e;
}

}  // namespace

const void *f8_kernel(int D, int R, int *smem) {
  const int nt = (R + 7) / 8;
  *smem = D == 64 ? F8Cfg<64>::SMEM_BYTES : F8Cfg<128>::SMEM_BYTES;
  return D == 64 ? kernel_of<64>(nt) : kernel_of<128>(nt);
}

cudaError_t launch_split_f8(int D, const SplitPlan &plan, const SplitParams &p, cudaStream_t stream) {
  return D == 64 ? launch<64>(plan, p, stream) : launch<128>(plan, p, stream);
}

}  // namespace td
