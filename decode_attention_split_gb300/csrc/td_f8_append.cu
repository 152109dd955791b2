// Cache append into the block-scaled 8-bit cache, and the same with a rotation first.
//
// For every (sequence b, kv head h, cache block j) that new rows L .. L+T-1 touch, K and V apart:
//   amax = the largest finite |x| of the block's new rows, c = 2^k, k the least with amax <= 448 c
//   s    = max(s_old, c) if the block already holds rows below L, else c
//   older codes of the block: code * (s_old / s), rounded, if s > s_old
//   new codes: x * (1 / s), rounded to nearest even (NaN and infinities: NaN)
// The rotation is quantised directly from fp32 (one rounding into e4m3, none into bf16 before it).
// Pair i of token t turns by the table row L + t, or by positions[b, t, axes[i]].
//
// Two kernels share the arithmetic. Both are bound by memory: a long chunk by its bytes, a
// token's rows by the chain of dependent loads (length, then scale and table row).
//  * rows (a few rows a sequence, see takes_rows): a warp per (head, block) or query row; where one CTA holds a sequence's
//    warps, it also advances the length once they have read it;
//  * tiles: a team of warps per (block, head) with the block's rows held in registers between the
//    maximum and the conversion (128 bytes a thread in flight), so the rows cross once. Plain appends take one team per
//    CTA. A rotation's CTA gathers the block's table rows into shared memory once and turns several
//    heads by them, fetching each head's rows a round ahead. Measured (GPU time in a graph):
//    a 4096-token chunk of 8 heads of 128, bf16, 6.0 us (25.2 MB, 4.2 TB/s); an 8000-token chunk
//    rotated with 24 query heads 29 us (150 MB, 5.1 TB/s), where rotating from the tables in L1,
//    head by head, took 39; three position axes, 4 x 1531 tokens, 30 us (83).
#include <math.h>

#include "td_f8.cuh"
#include "td_internal.h"
#include "td_rope.cuh"

namespace td {

namespace {

// Table offset of the row that pair i of token t of sequence b turns by, or -1 for a position or axis out of range (the pair is then not
// turned).
template <int D>
__device__ __forceinline__ long long table_row(const AppendF8 &p, int b, int t, int L, int i) {
  if (p.positions == nullptr) return (long long)(L + t) * (D / 2);
  const int a = p.axes == nullptr ? 0 : p.axes[i];
  if (a < 0 || a >= p.A) return -1;
  const int pos = p.positions[((long long)b * p.T + t) * p.A + a];
  if (pos < 0 || pos >= p.table_rows) return -1;
  return (long long)pos * (D / 2);
}

// cos and sin of N consecutive pairs from i (i and N multiples of 4 when N > 2) of token t.
template <int D, int N>
__device__ __forceinline__ void load_turn(const AppendF8 &p, int b, int t, int L, int i, float (&c)[N], float (&s)[N]) {
  bool one = true;  // all N pairs turn by the same table row
  if (p.axes != nullptr) {
    const int a0 = p.axes[i];
#pragma unroll
    for (int e = 1; e < N; ++e) one = one && p.axes[i + e] == a0;
  }
  if (one) {
    const long long row = table_row<D>(p, b, t, L, i);
    if (row < 0) report(p.status, TD_DEV_BAD_POSITION);
    const float *cp = p.cos_t + row + i, *sp = p.sin_t + row + i;
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 cv = row < 0 ? make_float4(1.f, 1.f, 1.f, 1.f) : *reinterpret_cast<const float4 *>(cp + e);
        const float4 sv = row < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4 *>(sp + e);
        c[e] = cv.x, c[e + 1] = cv.y, c[e + 2] = cv.z, c[e + 3] = cv.w;
        s[e] = sv.x, s[e + 1] = sv.y, s[e + 2] = sv.z, s[e + 3] = sv.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        c[e] = row < 0 ? 1.f : cp[e];
        s[e] = row < 0 ? 0.f : sp[e];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const long long row = table_row<D>(p, b, t, L, i + e);
      if (row < 0) report(p.status, TD_DEV_BAD_POSITION);
      c[e] = row < 0 ? 1.f : p.cos_t[row + i + e];
      s[e] = row < 0 ? 0.f : p.sin_t[row + i + e];
    }
  }
}

// N consecutive elements (N * sizeof(E) is 2, 4, 8 or 16 bytes, so aligned) widened, and back.
template <typename E, int N>
__device__ __forceinline__ void load_n(const E *x, float (&f)[N]) {
  if constexpr (N * sizeof(E) >= 4 && !(sizeof(E) == 4 && N == 1)) {
    load_widen<E, N>(x, f);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = widen_elem(x[e]);
  }
}
template <typename E, int N>
__device__ __forceinline__ void store_n(E *y, const float (&f)[N]) {
  if constexpr (N == 8) {
    *reinterpret_cast<uint4 *>(y) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                               pack_bf16x2(f[6], f[7]));
  } else if constexpr (N == 4) {
    *reinterpret_cast<float4 *>(y) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) store_elem<E>(y + i, f[i]);
  }
}
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *c, const float (&f)[N], float inv) {
  if constexpr (N == 1) {
    c[0] = (uint8_t)quant2_e4m3(make_float2(f[0], 0.f), inv);
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint16_t *>(c) = quant2_e4m3(make_float2(f[0], f[1]), inv);
  } else {
    uint32_t w[N / 4];
#pragma unroll
    for (int e = 0; e < N; e += 4)
      w[e / 4] = (uint32_t)quant2_e4m3(make_float2(f[e], f[e + 1]), inv) |
                 ((uint32_t)quant2_e4m3(make_float2(f[e + 2], f[e + 3]), inv) << 16);
    if constexpr (N == 8)
      *reinterpret_cast<uint2 *>(c) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t *>(c) = w[0];
  }
}
// rope_pair's products on two pairs at a time (the same operations, so the same bits).
template <int N>
__device__ __forceinline__ void rotate(float (&lo)[N], float (&hi)[N], const float (&c)[N], const float (&s)[N]) {
  if constexpr (N == 1) {
    const float a = lo[0], b = hi[0];
    rope_pair(a, b, c[0], s[0], lo[0], hi[0]);
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 a = make_float2(lo[e], lo[e + 1]), b = make_float2(hi[e], hi[e + 1]);
      const float2 cc = make_float2(c[e], c[e + 1]), ss = make_float2(s[e], s[e + 1]);
      const float2 y = ffma2(a, cc, fmul2(b, make_float2(-s[e], -s[e + 1]))), z = ffma2(b, cc, fmul2(a, ss));
      lo[e] = y.x, lo[e + 1] = y.y, hi[e] = z.x, hi[e + 1] = z.y;
    }
  }
}
// The keys' rotation: y = x0 c - x1 s, z = x1 c + x0 s with every product and sum rounded by itself, so
// the codes are those of the plain formula in fp32, bit for bit, whoever evaluates it. The products
// are the scalar intrinsic's, which is never joined into a fused operation: packed products and sums
// in inline PTX were, although each names its rounding, and moved about one code in a million. The
// sums are packed: all scalar, the bf16 tiles spill (8000 tokens 30.3 us, packed sums 29.4).
template <int N>
__device__ __forceinline__ void rotate_keys(float (&lo)[N], float (&hi)[N], const float (&c)[N], const float (&s)[N]) {
  if constexpr (N == 1) {
    const float a = lo[0], b = hi[0];
    lo[0] = __fadd_rn(__fmul_rn(a, c[0]), -__fmul_rn(b, s[0]));
    hi[0] = __fadd_rn(__fmul_rn(b, c[0]), __fmul_rn(a, s[0]));
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 a = make_float2(lo[e], lo[e + 1]), b = make_float2(hi[e], hi[e + 1]);
      const float2 ac = make_float2(__fmul_rn(a.x, c[e]), __fmul_rn(a.y, c[e + 1]));
      const float2 bs = make_float2(__fmul_rn(b.x, -s[e]), __fmul_rn(b.y, -s[e + 1]));
      const float2 bc = make_float2(__fmul_rn(b.x, c[e]), __fmul_rn(b.y, c[e + 1]));
      const float2 as = make_float2(__fmul_rn(a.x, s[e]), __fmul_rn(a.y, s[e + 1]));
      const float2 y = fadd2(ac, bs), z = fadd2(bc, as);
      lo[e] = y.x, lo[e + 1] = y.y, hi[e] = z.x, hi[e + 1] = z.y;
    }
  }
}
// The larger of amax and the finite |f|.
template <int N>
__device__ __forceinline__ float finite_max(float amax, const float (&f)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const float2 z = finite_or_nan(make_float2(f[e], N == 1 ? 0.f : f[e + (N > 1)]));
    amax = fmaxf(amax, fabsf(z.x));
    if (N > 1) amax = fmaxf(amax, fabsf(z.y));
  }
  return amax;
}
// The largest of a warp's amax (not negative, so its bits order as its values).
__device__ __forceinline__ uint32_t warp_amax(float amax) { return __reduce_max_sync(0xffffffffu, __float_as_uint(amax)); }

// The scale a block takes: its new rows' own, or the older rows' if that is larger.
__device__ __forceinline__ float block_scale(uint32_t amax, bool held, float s_old) {
  const float c = pow2_scale(amax);
  return held ? fmaxf(s_old, c) : c;
}

// ---- a few rows -------------------------------------------------------------------------

// Lane l of a warp holds dims l*N .. and D/2 + l*N .. of a row (N = D/64): the pairs of a rotation
// lie in one lane, and a row's codes go out as two runs of D/2 bytes.
template <typename E, int D, bool ROPE>
__global__ void __launch_bounds__(kF8RowsThreads) append_f8_rows_kernel(const AppendF8 p) {
  constexpr int N = D / 64, H = D / 2;
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int warp = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5), warps = gridDim.y * (blockDim.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  const long long L64 = p.seq_lens[b];
  const bool fits = L64 >= 0 && L64 + p.T <= p.Smax;
  const int L = (int)L64, T = p.T;
  if (!fits) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(p.status, TD_DEV_APPEND_OVERFLOW);
    return;
  }
  const int j0 = L >> p.block_log2, nblk = ((L + T - 1) >> p.block_log2) - j0 + 1;
  const int kv_units = 2 * p.Hkv * nblk;
  const int units = kv_units + (ROPE && p.q != nullptr ? p.Hq * T : 0);
  for (int u = warp; u < units; u += warps) {
    if (ROPE && u >= kv_units) {
      const int t = (u - kv_units) % T;
      const long long row = ((long long)b * p.Hq * T + (u - kv_units)) * D + lane * N;
      const E *x = static_cast<const E *>(p.q) + row;
      E *y = static_cast<E *>(p.q_out) + row;
      float lo[N], hi[N], c[N], s[N];
      load_n<E, N>(x, lo);
      load_n<E, N>(x + H, hi);
      load_turn<D, N>(p, b, t, L, lane * N, c, s);
      rotate<N>(lo, hi, c, s);
      store_n<E, N>(y, lo);
      store_n<E, N>(y + H, hi);
      continue;
    }
    const int j = j0 + u % nblk, h = (u / nblk) % p.Hkv;
    const bool isv = u >= p.Hkv * nblk;
    const int base = j << p.block_log2;
    const int r0 = max(L, base), r1 = min(L + T, base + (1 << p.block_log2));
    const long long head = (long long)b * p.Hkv + h;
    const E *x = static_cast<const E *>(isv ? p.v_new : p.k_new) + (head * T + (r0 - L)) * D + lane * N;
    uint8_t *codes = (isv ? p.v_codes : p.k_codes) + (head * p.Smax + base) * D;
    float *scale = (isv ? p.v_scales : p.k_scales) + head * p.NB + j;
    const bool held = r0 > base;
    const float s_old = held ? *scale : 0.f;
    float lo[N], hi[N];
    auto load_row = [&](int r) {
      load_n<E, N>(x + (long long)(r - r0) * D, lo);
      load_n<E, N>(x + (long long)(r - r0) * D + H, hi);
      if (ROPE && !isv) {
        float c[N], s[N];
        load_turn<D, N>(p, b, r - L, L, lane * N, c, s);
        rotate_keys<N>(lo, hi, c, s);
      }
    };
    float big = 0.f;
    for (int r = r0; r < r1; ++r) {
      load_row(r);
      big = finite_max<N>(finite_max<N>(big, lo), hi);
    }
    const uint32_t amax = warp_amax(big);
    const float sn = block_scale(amax, held, s_old);
    const float inv = __fdiv_rn(1.f, sn);
    if (held && sn > s_old) {
      const float ratio = __fdiv_rn(s_old, sn);
      uint32_t *w = reinterpret_cast<uint32_t *>(codes);
      for (int i = lane; i < (r0 - base) * (D / 4); i += 32) w[i] = rescale4_e4m3(w[i], ratio);
    }
    for (int r = r0; r < r1; ++r) {
      if (r1 - r0 > 1) load_row(r);  // one row is still in registers
      uint8_t *dst = codes + (long long)(r - base) * D + lane * N;
      store_codes<N>(dst, lo, inv);
      store_codes<N>(dst + H, hi, inv);
    }
    __syncwarp();  // every lane holds the old scale
    if (lane == 0) *scale = sn;
  }
  if (p.advance) {
    __syncthreads();  // every warp has read the length
    if (threadIdx.x == 0) p.seq_lens[b] = L + T;
  }
}

// ---- tiles of a block's rows ---------------------------------------------------------------

constexpr int kTilesThreads = 256;
constexpr int kTilesCtas = 450;  // CTAs a rotation's launch aims for: one and a half waves of two per SM
constexpr int kVecs = 8;  // 16-byte vectors a thread holds: 128 bytes in flight

// The rotation table of a tile in shared memory: cosines, then sines, of every (row, pair), the
// pairs of a row in the order that gives a warp's 16-byte reads consecutive addresses (for 8-pair
// vectors: the first four pairs of every vector, then the last four).
template <typename E, int D>
__device__ __forceinline__ int table_at(int row, int i) {
  constexpr int VE = 16 / sizeof(E);
  if constexpr (VE == 8) return row * (D / 2) + ((i >> 2) & 1) * (D / 4) + (i >> 3) * 4 + (i & 3);
  return row * (D / 2) + i;
}

template <typename E, int D>
__device__ __forceinline__ void load_table(const float *tab, int sines, int row, int v, float (&c)[16 / sizeof(E)],
                                           float (&s)[16 / sizeof(E)]) {
  constexpr int VE = 16 / sizeof(E);
#pragma unroll
  for (int e = 0; e < VE; e += 4) {
    const int at = table_at<E, D>(row, v * VE + e);
    const float4 cv = *reinterpret_cast<const float4 *>(tab + at);
    const float4 sv = *reinterpret_cast<const float4 *>(tab + sines + at);
    c[e] = cv.x, c[e + 1] = cv.y, c[e + 2] = cv.z, c[e + 3] = cv.w;
    s[e] = sv.x, s[e + 1] = sv.y, s[e + 2] = sv.z, s[e + 3] = sv.w;
  }
}

__device__ __forceinline__ void copy_pairs(uint4 (&lo)[kVecs / 2], uint4 (&hi)[kVecs / 2],
                                           const uint4 (&next_lo)[kVecs / 2], const uint4 (&next_hi)[kVecs / 2]) {
#pragma unroll
  for (int k = 0; k < kVecs / 2; ++k) lo[k] = next_lo[k], hi[k] = next_hi[k];
}

// blockIdx: x the touched block, y the group of heads (K heads, then V heads, then query heads),
// z the sequence. The CTA's warps form teams of `p.team` threads, enough to hold a block's rows of
// one head (team * kVecs vectors), and the teams take the group's heads in turn. A rotation's
// table rows are gathered once per CTA, into shared memory.
// At most 256 threads for bf16 rows, 512 for fp32 ones (blocks of 128 rows of 512 bytes).
template <typename E, int D, bool ROPE>
__global__ void __launch_bounds__(sizeof(E) == 2 ? 256 : 512, (ROPE ? 2 : 4) * (int)sizeof(__nv_bfloat16) / (int)sizeof(E))
    append_f8_tiles_kernel(const AppendF8 p) {
  constexpr int VE = 16 / sizeof(E), NV = D / VE, NH = NV / 2, H = D / 2;
  extern __shared__ __align__(16) float tab[];
  __shared__ uint32_t s_max[2][16];
  const int b = blockIdx.z, tid = threadIdx.x, threads = p.team;
  const int team = tid / threads, teams = blockDim.x / threads, tt = tid % threads;
  griddep_wait();
  griddep_launch_dependents();
  const long long L64 = p.seq_lens[b];
  const int T = p.T;
  if (L64 < 0 || L64 + T > p.Smax) {
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) report(p.status, TD_DEV_APPEND_OVERFLOW);
    return;
  }
  const int L = (int)L64;
  const int j = (L >> p.block_log2) + blockIdx.x;
  const int base = j << p.block_log2;
  const int r0 = max(L, base), r1 = min(L + T, base + (1 << p.block_log2));
  if (r0 >= r1) return;
  const int n = r1 - r0, t0 = r0 - L;
  const int units = 2 * p.Hkv + (ROPE && p.q != nullptr ? p.Hq : 0);
  const int u0 = blockIdx.y * p.per_cta, u1 = min(u0 + p.per_cta, units);
  const bool held = r0 > base;
  // a head's tile as pairs of vectors (v, v + D/2) of a row, kVecs / 2 pairs a thread; a rotation's
  // CTA fetches each head's one round ahead, the first while it gathers its table
  uint4 lo[kVecs / 2], hi[kVecs / 2];
  auto fetch = [&](int u, uint4(&x0)[kVecs / 2], uint4(&x1)[kVecs / 2]) {
    const bool isq = u >= 2 * p.Hkv, isv = !isq && u >= p.Hkv;
    const long long head = isq ? (long long)b * p.Hq + u - 2 * p.Hkv : (long long)b * p.Hkv + (isv ? u - p.Hkv : u);
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const E *>(isq ? p.q : isv ? p.v_new : p.k_new) +
                                                     (head * T + t0) * D);
#pragma unroll
    for (int k = 0; k < kVecs / 2; ++k) {
      const int i = tt + k * threads;
      if (u < u1 && i < n * NH) {
        const uint4 *row = x + (i / NH) * NV + i % NH;
        x0[k] = __ldcs(row);
        x1[k] = __ldcs(row + NH);
      }
    }
  };
  if constexpr (ROPE) fetch(u0 + team, lo, hi);
  const int sines = H << p.block_log2;
  if constexpr (ROPE) {
    for (int i = tid; i < n * (H / 4); i += blockDim.x) {
      const int r = i / (H / 4), pair = i % (H / 4) * 4;
      float c[4], s[4];
      load_turn<D, 4>(p, b, t0 + r, L, pair, c, s);
      *reinterpret_cast<float4 *>(tab + table_at<E, D>(r, pair)) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4 *>(tab + sines + table_at<E, D>(r, pair)) = make_float4(s[0], s[1], s[2], s[3]);
    }
    __syncthreads();
  }
  int flip = 0;
  // rounds of one head per team; the barrier of a round with K or V heads is the whole CTA's
#pragma unroll 1
  for (int first = u0; first < u1; first += teams) {
    const int u = first + team;
    const bool mine = u < u1;
    const bool isq = u >= 2 * p.Hkv, isv = !isq && u >= p.Hkv;
    const int h = isq ? u - 2 * p.Hkv : isv ? u - p.Hkv : u;
    const long long head = (long long)b * (isq ? p.Hq : p.Hkv) + h;
    uint8_t *codes = (isv ? p.v_codes : p.k_codes) + (head * p.Smax + base) * D;
    float *scale = (isv ? p.v_scales : p.k_scales) + head * p.NB + j;
    const float s_old = held && mine && !isq ? *scale : 0.f;
    const int items = mine ? n * NH : 0;
    uint4 next_lo[kVecs / 2], next_hi[kVecs / 2];
    if constexpr (!ROPE)
      fetch(u, lo, hi);
    else if (first + teams < u1)
      fetch(u + teams, next_lo, next_hi);
    if (ROPE && isq) {
      uint4 *y = reinterpret_cast<uint4 *>(static_cast<E *>(p.q_out) + (head * T + t0) * D);
#pragma unroll
      for (int k = 0; k < kVecs / 2; ++k) {
        const int i = tt + k * threads;
        if (i < items) {
          float a[VE], z[VE], c[VE], s[VE];
          load_widen<E, VE>(&lo[k], a);
          load_widen<E, VE>(&hi[k], z);
          load_table<E, D>(tab, sines, i / NH, i % NH, c, s);
          rotate<VE>(a, z, c, s);
          E *row = reinterpret_cast<E *>(y + (i / NH) * NV + i % NH);
          store_n<E, VE>(row, a);
          store_n<E, VE>(row + H, z);
        }
      }
    }
    if (ROPE && first >= 2 * p.Hkv) {  // query heads alone in this round: no barrier
      copy_pairs(lo, hi, next_lo, next_hi);
      continue;
    }
    // fp32 rows are rotated in place; bf16 rows stay as read (their rotation has more bits than
    // the register holds) and are rotated again for the conversion
    const int stored = isq ? 0 : items;
    float big = 0.f;
#pragma unroll
    for (int k = 0; k < kVecs / 2; ++k) {
      const int i = tt + k * threads;
      if (i < stored) {
        float a[VE], z[VE];
        load_widen<E, VE>(&lo[k], a);
        load_widen<E, VE>(&hi[k], z);
        if (ROPE && !isv) {
          float c[VE], s[VE];
          load_table<E, D>(tab, sines, i / NH, i % NH, c, s);
          rotate_keys<VE>(a, z, c, s);
          if constexpr (sizeof(E) == 4) {
            store_n<E, VE>(reinterpret_cast<E *>(&lo[k]), a);
            store_n<E, VE>(reinterpret_cast<E *>(&hi[k]), z);
          }
        }
        big = finite_max<VE>(finite_max<VE>(big, a), z);
      }
    }
    uint32_t amax = warp_amax(big);
    if (threads > 32) {
      // two areas in turn: a warp may still read one unit's while another writes the next's
      if ((tid & 31) == 0) s_max[flip][tid >> 5] = amax;
      __syncthreads();
#pragma unroll 1
      for (int w = 0; w < (threads >> 5); ++w) amax = max(amax, s_max[flip][team * (threads >> 5) + w]);
      flip ^= 1;
    } else {
      __syncwarp();  // every thread of the team holds the old scale before one writes the new
    }
    const float sn = block_scale(amax, held, s_old);
    const float inv = __fdiv_rn(1.f, sn);
#pragma unroll
    for (int k = 0; k < kVecs / 2; ++k) {
      const int i = tt + k * threads;
      if (i < stored) {
        float a[VE], z[VE];
        load_widen<E, VE>(&lo[k], a);
        load_widen<E, VE>(&hi[k], z);
        if (ROPE && !isv && sizeof(E) == 2) {
          float c[VE], s[VE];
          load_table<E, D>(tab, sines, i / NH, i % NH, c, s);
          rotate_keys<VE>(a, z, c, s);
        }
        uint8_t *dst = codes + (r0 - base + i / NH) * D + (i % NH) * VE;
        store_codes<VE>(dst, a, inv);
        store_codes<VE>(dst + H, z, inv);
      }
    }
    if (stored > 0 && held && sn > s_old) {
      const float ratio = __fdiv_rn(s_old, sn);
      uint32_t *w = reinterpret_cast<uint32_t *>(codes);
#pragma unroll 1
      for (int i = tt; i < (r0 - base) * (D / 4); i += threads) w[i] = rescale4_e4m3(w[i], ratio);
    }
    if (stored > 0 && tt == 0) *scale = sn;
    if constexpr (ROPE) copy_pairs(lo, hi, next_lo, next_hi);
  }
}

// seq_lens[b] += T for the sequences whose rows fitted, after the tiles' launch.
__global__ void advance_f8_kernel(int32_t *seq_lens, int B, int T, int Smax) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  const long long L = seq_lens[b];
  if (L >= 0 && L + T <= Smax) seq_lens[b] = (int32_t)(L + T);
}

// Whether T rows of each of `heads` heads (of all sequences) go to the rows kernel. A warp there
// takes its rows one after another, whatever the number of sequences; the tiles kernel takes a
// block's rows at once, in more rounds the more heads there are. Measured in us, rows / tiles, 48
// heads a sequence rotated: 1 sequence T = 1 3.2 / 3.4, T = 4 5.2 / 3.8; 24 sequences T = 4 5.3 / 7.0,
// T = 8 8.1 / 7.3; 64 sequences T = 12 11.2 / 12, T = 16 16.5 / 12.8. 16 heads, plain: 1 sequence T = 4
// 3.1 / 3.5, T = 8 3.6 / 3.3; 64 sequences T = 8 3.9 / 5.3, T = 16 4.8 / 5.6. The rows kernel's launch counts on
// one block a chunk; where a plain one crosses into another, some warps take a second unit (16 heads of 24
// sequences, T = 4 2.0 against 3.0, T = 8 2.5 against 3.8; rotated ones, whose units get shorter, lose 3 % at
// most and gain up to a fifth).
bool takes_rows(bool rope, int T, long long heads) {
  return T <= kF8RowsT && T <= (rope ? 1 + heads / 240 : 4 + heads / 50);
}

cudaError_t launch_advance(const AppendF8 &p, cudaStream_t stream) {
  return launch_pdl(advance_f8_kernel, dim3((p.B + 255) / 256), dim3(256), 0, stream, p.seq_lens, p.B, p.T, p.Smax);
}

template <typename E, int D, bool ROPE>
cudaError_t launch(const AppendF8 &args, cudaStream_t stream) {
  AppendF8 p = args;
  const int units = 2 * p.Hkv + (p.q != nullptr ? p.Hq : 0);
  if (takes_rows(ROPE, p.T, (long long)p.B * units)) {
    // warps with work (one block touched). A CTA that holds them all in one round can advance the
    // length; else they spread over CTAs of 8 and a second launch advances (32 sequences, one token,
    // 16 K/V and 32 query heads: 4.1 us in one CTA a sequence, 3.2 in six, 4.0 with the second launch)
    const long long work = 2 * p.Hkv + (p.q != nullptr ? (long long)p.Hq * p.T : 0);
    const bool apart = p.advance && work > kF8RowsThreads / 32;
    const int warps = (int)(p.advance && !apart ? work : work > 8 ? 8 : work);
    const long long spread = p.advance && !apart ? 1 : (work + warps - 1) / warps;
    if (apart) p.advance = 0;
    cudaError_t e = launch_pdl(append_f8_rows_kernel<E, D, ROPE>, dim3(p.B, (unsigned)(spread > 1024 ? 1024 : spread)),
                               dim3(32 * warps), 0, stream, p);
    if (e == cudaSuccess && apart) e = launch_advance(p, stream);
    return e;
  }
  const int block = 1 << p.block_log2;
  const int vecs = block * D * (int)sizeof(E) / 16;
  p.team = vecs / kVecs < 32 ? 32 : vecs / kVecs;
  // a rotation's CTAs share their table among several teams and heads; plain appends share nothing
  const int threads = !ROPE || p.team > kTilesThreads ? p.team : kTilesThreads;
  const int teams = threads / p.team;
  const int nblk = (p.T + block - 2) / block + 1;
  // heads of a CTA: a round of its teams or more, as long as the grid still fills the GPU
  const long long tiles = (long long)nblk * p.B;
  long long per = ROPE ? tiles * units / kTilesCtas / teams * teams : 1;
  if (per < teams) per = teams;
  int groups = per >= units ? 1 : (int)((units + per - 1) / per);
  p.per_cta = ((units + groups - 1) / groups + teams - 1) / teams * teams;  // the groups alike
  groups = (units + p.per_cta - 1) / p.per_cta;
  const int smem = ROPE ? block * D * (int)sizeof(float) : 0;
  const void *fn = reinterpret_cast<const void *>(&append_f8_tiles_kernel<E, D, ROPE>);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = launch_pdl(append_f8_tiles_kernel<E, D, ROPE>, dim3(nblk, groups, p.B), dim3(threads), smem, stream, p);
  if (e == cudaSuccess && p.advance) e = launch_advance(p, stream);
  return e;
}

template <typename E, int D>
cudaError_t launch_d(const AppendF8 &p, cudaStream_t stream) {
  return p.cos_t != nullptr ? launch<E, D, true>(p, stream) : launch<E, D, false>(p, stream);
}

}  // namespace

cudaError_t launch_append_f8(size_t elem_bytes, int D, const AppendF8 &p, cudaStream_t stream) {
  cudaError_t e;
  if (elem_bytes == 2)
    e = D == 64 ? launch_d<__nv_bfloat16, 64>(p, stream) : launch_d<__nv_bfloat16, 128>(p, stream);
  else
    e = D == 64 ? launch_d<float, 64>(p, stream) : launch_d<float, 128>(p, stream);
  return e;
}

}  // namespace td
