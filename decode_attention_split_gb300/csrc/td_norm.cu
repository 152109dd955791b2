// Query and key norms with the rotation and the cache write, one pass over the new rows.
//
//   y = x * w / sqrt(mean_i x_i^2 + eps)   (a query or key row x of one head, D elements, weights w)
//   then the pairs (y[i], y[i + D/2]) turn by the row's angles; keys and values go to cache rows
//   seq_lens[b] + t, queries to q_out.
//
// All of it in fp32 (the sum of squares too), one rounding at the end: the norm's result is not rounded
// to the rows' type before the rotation, which would cost a second half step of it.
//
// Bound by memory: every new row is read once and written once (2 * (Hq + 2 Hkv) * D elements a token),
// about seven operations an element. NH = D / 2 * sizeof(E) / 16 lanes hold a row, each one 16-byte vector of
// its lower and one of its upper half, so a pair is in one thread and the sum of squares is a few
// shuffles. Two kernels: a chunk's row groups of lanes stay with one token and walk over heads, so the token's cosines and
// sines (4 D bytes, twice a bf16 row) are fetched once for all of them; a few tokens' take a row each.
// Measured (GPU time in a graph): a 4096-token chunk of 24 + 16 heads of 128, bf16, 16.8 us (86 MB, 5.1 TB/s); one token
// of 8 sequences (15 + 5 heads of 64) 1.7 us.
#include "td_device.cuh"
#include "td_internal.h"
#include "td_rope.cuh"

namespace td {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormCtas = 6 * 152;  // CTAs a chunk's launch aims for

// Cosines and sines of this lane's pairs.
template <int VE>
struct Turn {
  float c[VE], s[VE];
};

// Those of token t, whose cache row is `row`: pairs i0 .. i0 + VE - 1. A pair whose position or axis is out of range
// turns by no angle.
template <int D, int VE>
__device__ __forceinline__ Turn<VE> load_turn(const NormAppend &p, int b, int t, int row, int i0, uint32_t &bits) {
  Turn<VE> a;
  if (p.positions == nullptr) {
    const long long at = (long long)row * (D / 2) + i0;
#pragma unroll
    for (int j = 0; j < VE; j += 4) {
      *reinterpret_cast<float4 *>(a.c + j) = *reinterpret_cast<const float4 *>(p.cos_t + at + j);
      *reinterpret_cast<float4 *>(a.s + j) = *reinterpret_cast<const float4 *>(p.sin_t + at + j);
    }
    return a;
  }
#pragma unroll
  for (int j = 0; j < VE; ++j) {
    const int axis = p.axes == nullptr ? 0 : p.axes[i0 + j];
    const bool known = axis >= 0 && axis < p.A;
    const int pos = known ? p.positions[((long long)b * p.T + t) * p.A + axis] : -1;
    const bool in = pos >= 0 && pos < p.table_rows;
    const long long at = (long long)(in ? pos : 0) * (D / 2) + i0 + j;
    a.c[j] = in ? p.cos_t[at] : 1.f;
    a.s[j] = in ? p.sin_t[at] : 0.f;
    if (!in) bits |= TD_DEV_BAD_POSITION;
  }
  return a;
}

template <typename E, int VE>
__device__ __forceinline__ uint4 pack_row(const float (&x)[VE]) {
  uint4 v;
  if constexpr (sizeof(E) == 2) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 r = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t *>(&r);
    }
  } else {
    v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  return v;
}

// The weights of this lane's elements, of the row's lower and upper half.
template <int D, int VE>
__device__ __forceinline__ void load_weights(const float *w, float (&wa)[VE], float (&wz)[VE]) {
#pragma unroll
  for (int j = 0; j < VE; j += 4) {
    *reinterpret_cast<float4 *>(wa + j) = *reinterpret_cast<const float4 *>(w + j);
    *reinterpret_cast<float4 *>(wz + j) = *reinterpret_cast<const float4 *>(w + D / 2 + j);
  }
}

// A row's halves x and z (this lane's elements): divided by the row's root mean square, weighted, turned.
// Warp-wide: the row's lanes exchange their sums of squares.
template <int D, int VE>
__device__ __forceinline__ void norm_turn(float eps, const Turn<VE> &turn, const float (&wa)[VE], const float (&wz)[VE],
                                          float (&x)[VE], float (&z)[VE]) {
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < VE; ++j) ss = fmaf(x[j], x[j], fmaf(z[j], z[j], ss));
#pragma unroll
  for (int o = D / 4 / VE; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float r = rsqrtf(ss * (1.f / D) + eps);
#pragma unroll
  for (int j = 0; j < VE; ++j) {
    const float n0 = x[j] * r * wa[j], n1 = z[j] * r * wz[j];
    rope_pair(n0, n1, turn.c[j], turn.s[j], x[j], z[j]);
  }
}

// What becomes of a row: normed and turned, or copied.
enum : int { kQuery = 0, kKey = 1, kValue = 2 };

// Heads [first, h1) of one kind; of a kind that this CTA has no heads of nothing is read (without queries there are no
// weights of theirs). Every lane of a warp makes every round (the exchanges are warp-wide); a row that is not there is not
// loaded or stored.
template <typename E, int D, int KIND, int VE>
__device__ __forceinline__ void norm_heads(const NormAppend &p, const Turn<VE> &turn, int b, int t, int L, bool there,
                                           bool fits, int v, int first, int h1) {
  constexpr int NH = D / 2 / VE, NV = 2 * NH;
  if (first >= h1) return;  // the same in every thread of the CTA
  const int H = KIND == kQuery ? p.Hq : p.Hkv;
  const uint4 *src = static_cast<const uint4 *>(KIND == kQuery ? p.q : KIND == kKey ? p.k_new : p.v_new) +
                     ((long long)b * H * p.T + t) * NV + v;
  uint4 *dst = static_cast<uint4 *>(KIND == kQuery ? p.q_out : KIND == kKey ? p.k_cache : p.v_cache) + v;
  dst += KIND == kQuery ? ((long long)b * H * p.T + t) * NV : ((long long)b * H * p.Smax + L + t) * NV;
  const long long sstride = (long long)p.T * NV, dstride = KIND == kQuery ? sstride : (long long)p.Smax * NV;
  float wa[VE], wz[VE];
  if constexpr (KIND != kValue) load_weights<D, VE>((KIND == kQuery ? p.q_weight : p.k_weight) + v * VE, wa, wz);
  for (int h = first; h < h1; ++h) {
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (there) {
      lo = src[h * sstride];
      hi = src[h * sstride + NH];
    }
    if constexpr (KIND != kValue) {
      float x[VE], z[VE];
      load_widen<E, VE>(&lo, x);
      load_widen<E, VE>(&hi, z);
      norm_turn<D, VE>(p.eps, turn, wa, wz, x, z);
      lo = pack_row<E, VE>(x);
      hi = pack_row<E, VE>(z);
    }
    if (there && fits) {
      dst[h * dstride] = lo;
      dst[h * dstride + NH] = hi;
    }
  }
}

// A chunk. Grid: (token tiles x head groups, B); a row group for every token of the tile, walking over the CTA's heads.
template <typename E, int D>
__global__ void __launch_bounds__(kNormThreads, 4) norm_append_kernel(const NormAppend p) {
  constexpr int VE = 16 / sizeof(E);
  constexpr int NH = D / 2 / VE;  // lanes of a row
  const int b = blockIdx.y;
  const int tile = blockIdx.x / p.head_groups, hg = blockIdx.x % p.head_groups;
  const int v = threadIdx.x % NH;
  const int tok = tile * (kNormThreads / NH) + threadIdx.x / NH;
  const bool there = tok < p.T;
  const int t = there ? tok : 0;

  griddep_wait();  // rows, lengths and cache may come from the previous kernel in the stream
  griddep_launch_dependents();
  const long long raw = p.seq_lens[b];
  const bool fits = raw >= 0 && raw + p.T <= p.Smax;
  const int L = fits ? (int)raw : 0;
  uint32_t bits = fits ? 0u : TD_DEV_APPEND_OVERFLOW;
  const Turn<VE> turn = load_turn<D, VE>(p, b, t, fits ? L + t : 0, v * VE, bits);
  if (bits != 0 && hg == 0 && there) report(p.status, fits ? bits : TD_DEV_APPEND_OVERFLOW);

  // the heads of this CTA, queries before keys before values
  const int c0 = hg * p.per_cta, c1 = c0 + p.per_cta, k0 = p.Hq, v0 = p.Hq + p.Hkv;
  norm_heads<E, D, kQuery, VE>(p, turn, b, t, L, there, fits, v, c0, min(c1, p.Hq));
  norm_heads<E, D, kKey, VE>(p, turn, b, t, L, there, fits, v, max(c0 - k0, 0), min(c1 - k0, p.Hkv));
  norm_heads<E, D, kValue, VE>(p, turn, b, t, L, there, fits, v, max(c0 - v0, 0), min(c1 - v0, p.Hkv));
}

// Few rows: a row group for every row (with `advance`, one CTA for a sequence, its groups taking several). What
// bounds a token's call is its chain of loads, so the row and its weights are asked for before the length.
template <typename E, int D>
__global__ void __launch_bounds__(kNormThreads) norm_append_rows_kernel(const NormAppend p) {
  constexpr int VE = 16 / sizeof(E);
  constexpr int NH = D / 2 / VE, NV = 2 * NH;
  const int b = blockIdx.y, v = threadIdx.x % NH;
  const int rows = (p.Hq + 2 * p.Hkv) * p.T, step = gridDim.x * (kNormThreads / NH);
  griddep_wait();
  griddep_launch_dependents();
  for (int base = blockIdx.x * (kNormThreads / NH); base < rows; base += step) {
    const int row = base + threadIdx.x / NH;
    const bool there = row < rows;
    const int h = there ? row / p.T : 0, t = there ? row % p.T : 0;
    const bool isq = h < p.Hq, isv = h >= p.Hq + p.Hkv;
    const int kvh = isv ? h - p.Hq - p.Hkv : h - p.Hq;
    const uint4 *src = static_cast<const uint4 *>(isq ? p.q : isv ? p.v_new : p.k_new) +
                       ((isq ? (long long)b * p.Hq + h : (long long)b * p.Hkv + kvh) * p.T + t) * NV + v;
    uint4 lo = src[0], hi = src[NH];
    float wa[VE], wz[VE];
    load_weights<D, VE>((isq ? p.q_weight : p.k_weight) + v * VE, wa, wz);
    const long long raw = p.seq_lens[b];
    const bool fits = raw >= 0 && raw + p.T <= p.Smax;
    const int L = fits ? (int)raw : 0;
    uint32_t bits = fits ? 0u : TD_DEV_APPEND_OVERFLOW;
    const Turn<VE> turn = load_turn<D, VE>(p, b, t, fits ? L + t : 0, v * VE, bits);
    if (bits != 0) report(p.status, fits ? bits : TD_DEV_APPEND_OVERFLOW);
    float x[VE], z[VE];
    load_widen<E, VE>(&lo, x);
    load_widen<E, VE>(&hi, z);
    norm_turn<D, VE>(p.eps, turn, wa, wz, x, z);
    if (!there || !fits) continue;
    if (!isv) {
      lo = pack_row<E, VE>(x);
      hi = pack_row<E, VE>(z);
    }
    uint4 *dst = isq ? static_cast<uint4 *>(p.q_out) + (((long long)b * p.Hq + h) * p.T + t) * NV
                     : static_cast<uint4 *>(isv ? p.v_cache : p.k_cache) +
                           (((long long)b * p.Hkv + kvh) * p.Smax + L + t) * NV;
    dst[v] = lo;
    dst[v + NH] = hi;
  }
  if (p.advance) {
    __syncthreads();  // every thread has read the length
    if (threadIdx.x == 0) {
      const long long raw = p.seq_lens[b];
      if (raw >= 0 && raw + p.T <= p.Smax) p.seq_lens[b] = (int32_t)(raw + p.T);
    }
  }
}

// Chunks of fewer tokens than a CTA has row groups go to the rows kernel. Measured in us (24 + 16 heads of 128, bf16),
// rows / heads: one token of 1 sequence 1.9 / 2.8, of 64 2.0 / 2.9, of 256 3.8 / 5.0; 16 tokens of 1 2.0 / 2.3, of 32
// 4.5 / 5.4. The heads kernel's CTAs: with 6, 8, 12 and 24 of them an SM in all a 4096-token chunk takes 17.3, 18.3,
// 18.4 and 21.0; two heads in flight a row group instead of one change that by 0.1 and cost a 1000-token chunk 6.6 -> 8.2.
template <typename E, int D>
cudaError_t launch_d(const NormAppend &args, cudaStream_t stream) {
  constexpr int groups = kNormThreads / (D / 2 * (int)sizeof(E) / 16);
  NormAppend p = args;
  const int Hall = p.Hq + 2 * p.Hkv;
  const long long rows = (long long)Hall * p.T;
  bool apart = p.advance;  // a second launch moves the lengths
  p.advance = 0;
  cudaError_t e;
  if (p.T < groups) {
    const long long ctas = (rows + groups - 1) / groups;
    p.advance = apart && ctas <= 4;  // one CTA takes the sequence's rows in up to four rounds
    apart = apart && !p.advance;
    e = launch_pdl(norm_append_rows_kernel<E, D>, dim3(p.advance ? 1 : (unsigned)ctas, p.B), dim3(kNormThreads), 0, stream,
                   p);
  } else {
    const long long tiles = (p.T + groups - 1) / groups;
    long long per = Hall * tiles * p.B / kNormCtas;
    if (per < 1) per = 1;
    if (per > Hall) per = Hall;
    p.per_cta = (int)per;
    p.head_groups = (int)((Hall + per - 1) / per);
    e = launch_pdl(norm_append_kernel<E, D>, dim3((unsigned)(tiles * p.head_groups), p.B), dim3(kNormThreads), 0, stream, p);
  }
  if (e == cudaSuccess && apart) e = launch_advance(p.seq_lens, p.B, p.T, p.Smax, stream);
  return e;
}

}  // namespace

cudaError_t launch_norm_append(size_t elem_bytes, int D, const NormAppend &p, cudaStream_t stream) {
  if (elem_bytes == 2) return D == 64 ? launch_d<__nv_bfloat16, 64>(p, stream) : launch_d<__nv_bfloat16, 128>(p, stream);
  return D == 64 ? launch_d<float, 64>(p, stream) : launch_d<float, 128>(p, stream);
}

}  // namespace td
