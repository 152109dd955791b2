// Cache append into the block-scaled 8-bit cache, and the same with a rotation first.
//
// For every (sequence b, kv head h, cache block j) that new rows L .. L+T-1 touch, K and V apart:
//   amax = the largest finite |x| of the block's new rows, c = 2^k, k the least with amax <= 448 c
//   s    = max(s_old, c) if the block already holds rows below L, else c
//   older codes of the block: code * (s_old / s), rounded, if s > s_old
//   new codes: x * (1 / s), rounded to nearest even (NaN and infinities: NaN)
// The rotation (td_rope.cuh's pairs, in fp32) is quantised directly from fp32: one rounding.
// Pair i of token t turns by the table row L + t, or by positions[b, t, axes[i]].
//
// Two kernels share the arithmetic. Both are bound by memory: a long chunk by its bytes, a
// token's rows by the chain of dependent loads (length, then scale and table row).
//  * rows (T <= kRowsT): one CTA per sequence, a warp per (head, block) or query row, which
//    advances the length itself once its warps have read it;
//  * tiles: one CTA per (block, group of heads), the block's rows held in registers between the
//    maximum and the conversion (128 bytes a thread in flight), so the rows cross once; the
//    lengths are advanced by a second launch, after every read of them.
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
  if constexpr (N * sizeof(E) == 16) {
    uint4 w;
    E *e = reinterpret_cast<E *>(&w);
#pragma unroll
    for (int i = 0; i < N; ++i) store_elem<E>(e + i, f[i]);
    *reinterpret_cast<uint4 *>(y) = w;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) store_elem<E>(y + i, f[i]);
  }
}
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *c, const float (&f)[N], float inv) {
  if constexpr (N == 1) {
    c[0] = (uint8_t)quant2_e4m3(f[0], 0.f, inv);
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint16_t *>(c) = quant2_e4m3(f[0], f[1], inv);
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4)
      *reinterpret_cast<uint32_t *>(c + e) =
          (uint32_t)quant2_e4m3(f[e], f[e + 1], inv) | ((uint32_t)quant2_e4m3(f[e + 2], f[e + 3], inv) << 16);
  }
}
template <int N>
__device__ __forceinline__ void rotate(float (&lo)[N], float (&hi)[N], const float (&c)[N], const float (&s)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float a = lo[e], b = hi[e];
    rope_pair(a, b, c[e], s[e], lo[e], hi[e]);
  }
}

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
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const long long L64 = p.seq_lens[b];
  const bool fits = L64 >= 0 && L64 + p.T <= p.Smax;
  const int L = (int)L64, T = p.T;
  if (!fits) {
    if (threadIdx.x == 0) report(p.status, TD_DEV_APPEND_OVERFLOW);
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
    uint32_t amax = 0;
    for (int r = r0; r < r1; ++r) {
      load_n<E, N>(x + (long long)(r - r0) * D, lo);
      load_n<E, N>(x + (long long)(r - r0) * D + H, hi);
      if (ROPE && !isv) {
        float c[N], s[N];
        load_turn<D, N>(p, b, r - L, L, lane * N, c, s);
        rotate<N>(lo, hi, c, s);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) amax = max(amax, max(finite_abs_bits(lo[e]), finite_abs_bits(hi[e])));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    const float sn = block_scale(amax, held, s_old);
    const float inv = __fdiv_rn(1.f, sn);
    if (held && sn > s_old) {
      const float ratio = __fdiv_rn(s_old, sn);
      uint32_t *w = reinterpret_cast<uint32_t *>(codes);
      for (int i = lane; i < (r0 - base) * (D / 4); i += 32) w[i] = rescale4_e4m3(w[i], ratio);
    }
    for (int r = r0; r < r1; ++r) {
      if (r1 - r0 > 1) {  // one row is still in registers
        load_n<E, N>(x + (long long)(r - r0) * D, lo);
        load_n<E, N>(x + (long long)(r - r0) * D + H, hi);
        if (ROPE && !isv) {
          float c[N], s[N];
          load_turn<D, N>(p, b, r - L, L, lane * N, c, s);
          rotate<N>(lo, hi, c, s);
        }
      }
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

constexpr int kVecs = 8;  // 16-byte vectors a thread holds

// blockIdx: x the touched block, y the group of heads (K heads, then V heads, then query heads),
// z the sequence. blockDim.x * kVecs >= rows of a block * vectors of a row.
template <typename E, int D, bool ROPE>
__global__ void __launch_bounds__(512) append_f8_tiles_kernel(const AppendF8 p) {
  constexpr int VE = 16 / sizeof(E), NV = D / VE, NH = NV / 2, H = D / 2;
  __shared__ uint32_t s_max[2][16];
  const int b = blockIdx.z, tid = threadIdx.x, threads = blockDim.x;
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
  int flip = 0;
  for (int u = u0; u < u1; ++u) {
    const bool isq = u >= 2 * p.Hkv, isv = !isq && u >= p.Hkv;
    const int h = isq ? u - 2 * p.Hkv : isv ? u - p.Hkv : u;
    const long long head = (long long)b * (isq ? p.Hq : p.Hkv) + h;
    const E *x = static_cast<const E *>(isq ? p.q : isv ? p.v_new : p.k_new) + (head * T + t0) * D;
    if (ROPE && isq) {
      E *y = static_cast<E *>(p.q_out) + (head * T + t0) * D;
      for (int i = tid; i < n * NH; i += threads) {
        const int r = i / NH, v = i % NH;
        float lo[VE], hi[VE], c[VE], s[VE];
        load_n<E, VE>(x + (long long)r * D + v * VE, lo);
        load_n<E, VE>(x + (long long)r * D + v * VE + H, hi);
        load_turn<D, VE>(p, b, t0 + r, L, v * VE, c, s);
        rotate<VE>(lo, hi, c, s);
        store_n<E, VE>(y + (long long)r * D + v * VE, lo);
        store_n<E, VE>(y + (long long)r * D + v * VE + H, hi);
      }
      continue;
    }
    uint8_t *codes = (isv ? p.v_codes : p.k_codes) + (head * p.Smax + base) * D;
    float *scale = (isv ? p.v_scales : p.k_scales) + head * p.NB + j;
    const bool held = r0 > base;
    const float s_old = held ? *scale : 0.f;
    // the tile as pairs of vectors (v, v + D/2) of a row: kVecs / 2 pairs a thread
    uint4 lo[kVecs / 2], hi[kVecs / 2];
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < kVecs / 2; ++k) {
      const int i = tid + k * threads;
      if (i < n * NH) {
        const uint4 *row = reinterpret_cast<const uint4 *>(x + (long long)(i / NH) * D) + i % NH;
        lo[k] = row[0];
        hi[k] = row[NH];
      }
    }
    // fp32 rows are rotated in place; bf16 rows stay as read (their rotation has more bits than
    // the register holds) and are rotated again for the conversion
#pragma unroll
    for (int k = 0; k < kVecs / 2; ++k) {
      const int i = tid + k * threads;
      if (i < n * NH) {
        float a[VE], z[VE];
        load_widen<E, VE>(&lo[k], a);
        load_widen<E, VE>(&hi[k], z);
        if (ROPE && !isv) {
          float c[VE], s[VE];
          load_turn<D, VE>(p, b, t0 + i / NH, L, (i % NH) * VE, c, s);
          rotate<VE>(a, z, c, s);
          if constexpr (sizeof(E) == 4) {
            store_n<E, VE>(reinterpret_cast<E *>(&lo[k]), a);
            store_n<E, VE>(reinterpret_cast<E *>(&hi[k]), z);
          }
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) amax = max(amax, max(finite_abs_bits(a[e]), finite_abs_bits(z[e])));
      }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    // every thread holds the old scale before one of them writes the new
    if (threads == 32) {
      __syncwarp();
    } else {
      // two areas in turn: a warp may still read one unit's while another writes the next's
      if ((tid & 31) == 0) s_max[flip][tid >> 5] = amax;
      __syncthreads();
      for (int w = 0; w < (threads >> 5); ++w) amax = max(amax, s_max[flip][w]);
      flip ^= 1;
    }
    const float sn = block_scale(amax, held, s_old);
    const float inv = __fdiv_rn(1.f, sn);
#pragma unroll
    for (int k = 0; k < kVecs / 2; ++k) {
      const int i = tid + k * threads;
      if (i < n * NH) {
        float a[VE], z[VE];
        load_widen<E, VE>(&lo[k], a);
        load_widen<E, VE>(&hi[k], z);
        if (ROPE && !isv && sizeof(E) == 2) {
          float c[VE], s[VE];
          load_turn<D, VE>(p, b, t0 + i / NH, L, (i % NH) * VE, c, s);
          rotate<VE>(a, z, c, s);
        }
        uint8_t *dst = codes + (long long)(r0 - base + i / NH) * D + (i % NH) * VE;
        store_codes<VE>(dst, a, inv);
        store_codes<VE>(dst + H, z, inv);
      }
    }
    if (held && sn > s_old) {
      const float ratio = __fdiv_rn(s_old, sn);
      uint32_t *w = reinterpret_cast<uint32_t *>(codes);
      for (int i = tid; i < (r0 - base) * (D / 4); i += threads) w[i] = rescale4_e4m3(w[i], ratio);
    }
    if (tid == 0) *scale = sn;
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

template <typename E, int D, bool ROPE>
cudaError_t launch(const AppendF8 &args, cudaStream_t stream) {
  AppendF8 p = args;
  const int units = 2 * p.Hkv + (p.q != nullptr ? p.Hq : 0);
  if (p.T <= kF8RowsT) {
    const int most = 2 * p.Hkv + (p.q != nullptr ? p.Hq * p.T : 0);  // warps with work, one block touched
    const int threads = 32 * (most > kF8RowsThreads / 32 ? kF8RowsThreads / 32 : most);
    return launch_pdl(append_f8_rows_kernel<E, D, ROPE>, dim3(p.B), dim3(threads), 0, stream, p);
  }
  const int block = 1 << p.block_log2;
  const int vecs = block * D * (int)sizeof(E) / 16;
  const int threads = vecs / kVecs < 32 ? 32 : vecs / kVecs;
  const int nblk = (p.T + block - 2) / block + 1;
  // heads of a CTA: enough that the grid is a few waves, so a tile's table rows stay in L1 for
  // the next head
  const long long tiles = (long long)nblk * units * p.B;
  long long per = tiles / 4096;
  p.per_cta = (int)(per < 1 ? 1 : per > 8 ? 8 : per);
  const int groups = (units + p.per_cta - 1) / p.per_cta;
  cudaError_t e = launch_pdl(append_f8_tiles_kernel<E, D, ROPE>, dim3(nblk, groups, p.B), dim3(threads), 0, stream, p);
  if (e == cudaSuccess && p.advance)
    e = launch_pdl(advance_f8_kernel, dim3((p.B + 255) / 256), dim3(256), 0, stream, p.seq_lens, p.B, p.T, p.Smax);
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
