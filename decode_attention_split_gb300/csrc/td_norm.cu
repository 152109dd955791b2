// Query and key norms with the rotation and the cache write, one pass over the new rows.
//
//   y = x * w / sqrt(mean_i x_i^2 + eps)   (a query or key row x of one head, D elements, weights w)
//   then the pairs (y[i], y[i + D/2]) turn by the row's angles; keys and values go to cache rows
//   seq_lens[b] + t, queries to q_out.
//
// fp32 throughout (the sum of squares too), one rounding at the end: the norm's result is not rounded
// to the rows' type before the rotation, which would cost a second half step of it.
//
// Bound by memory: every new row is read once and written once (2 * (Hq + 2 Hkv) * D elements a token),
// about seven operations an element. NH = D / 2 * sizeof(E) / 16 lanes hold a row, each one 16-byte vector of
// its lower and one of its upper half, so a pair is in one thread and the sum of squares is a few
// shuffles. A row group of lanes stays with one token and walks over heads: the token's cosines and sines
// (4 D bytes, twice a bf16 row) are fetched once for all of them.
#include "td_device.cuh"
#include "td_internal.h"
#include "td_rope.cuh"

namespace td {

namespace {

constexpr int kNormThreads = 256;

// Cosines and sines of this lane's pairs, and a bit per pair that has none (its position or axis is out of
// range: the pair stays as it is).
template <int VE>
struct Turn {
  float c[VE], s[VE];
  uint32_t off;
};

template <typename E, int D, int VE>
__device__ __forceinline__ Turn<VE> load_turn(const NormAppend &p, int b, int t, int L, int i0, uint32_t &bits) {
  Turn<VE> a;
  a.off = 0;
  if (p.positions == nullptr) {
    const long long at = (long long)(L + t) * (D / 2) + i0;
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
    if (!in) a.off |= 1u << j;
  }
  if (a.off != 0) bits |= TD_DEV_BAD_POSITION;
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

// Grid: (token tiles x head groups, B). A CTA's row groups are tokens x heads: group g has token
// tile * tok + g % tok and heads first + g / tok, stepping by the groups' count over tok.
template <typename E, int D>
__global__ void __launch_bounds__(kNormThreads) norm_append_kernel(const NormAppend p) {
  constexpr int VE = 16 / sizeof(E);
  constexpr int NH = D / 2 / VE;               // lanes of a row
  constexpr int NV = 2 * NH;                   // 16-byte vectors of a row
  const int b = blockIdx.y;
  const int tile = blockIdx.x / p.head_groups, hg = blockIdx.x % p.head_groups;
  const int g = threadIdx.x / NH, v = threadIdx.x % NH;
  const int t = tile * p.tok + g % p.tok;
  const int step = blockDim.x / NH / p.tok;
  const int Hall = p.Hq + 2 * p.Hkv;
  const int h1 = min(Hall, (hg + 1) * p.per_cta);

  griddep_wait();  // rows, lengths and cache may come from the previous kernel in the stream
  griddep_launch_dependents();
  const long long raw = p.seq_lens[b];
  const bool fits = raw >= 0 && raw + p.T <= p.Smax;
  const int L = fits ? (int)raw : 0;
  uint32_t bits = fits ? 0u : TD_DEV_APPEND_OVERFLOW;
  const bool here = fits && t < p.T;
  Turn<VE> turn = {};
  if (here) turn = load_turn<E, D, VE>(p, b, t, L, v * VE, bits);
  if (bits != 0 && hg == 0) report(p.status, bits);

  const int tt = here ? t : 0;
  // every lane makes every round (the shuffles are warp-wide): values are normed in vain, and a head past
  // the last is skipped at its loads and stores
  for (int base = hg * p.per_cta; base < h1; base += step) {
    const int h = base + g / p.tok;
    const bool mine = here && h < h1;
    const bool isq = h < p.Hq, isv = h >= p.Hq + p.Hkv;
    const int kvh = isv ? h - p.Hq - p.Hkv : h - p.Hq;
    const uint4 *src = static_cast<const uint4 *>(isq ? p.q : isv ? p.v_new : p.k_new) +
                       (isq ? ((long long)b * p.Hq + h) * p.T + tt : ((long long)b * p.Hkv + kvh) * p.T + tt) * NV;
    uint4 *dst = isq ? static_cast<uint4 *>(p.q_out) + (((long long)b * p.Hq + h) * p.T + tt) * NV
                     : static_cast<uint4 *>(isv ? p.v_cache : p.k_cache) +
                           (((long long)b * p.Hkv + kvh) * p.Smax + L + tt) * NV;
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (mine) {
      lo = src[v];
      hi = src[v + NH];
    }
    float x[VE], z[VE];
    load_widen<E, VE>(&lo, x);
    load_widen<E, VE>(&hi, z);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VE; ++j) ss = fmaf(x[j], x[j], fmaf(z[j], z[j], ss));
#pragma unroll
    for (int o = NH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!mine) continue;
    if (!isv) {
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      const float *w = isq ? p.q_weight : p.k_weight;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float a = x[j] * r * w[v * VE + j], c = z[j] * r * w[D / 2 + v * VE + j];
        if ((turn.off >> j) & 1u) {
          x[j] = a;
          z[j] = c;
        } else {
          rope_pair(a, c, turn.c[j], turn.s[j], x[j], z[j]);
        }
      }
      lo = pack_row<E, VE>(x);
      hi = pack_row<E, VE>(z);
    }
    dst[v] = lo;
    dst[v + NH] = hi;
  }
  if (p.advance) {  // one CTA has the whole sequence
    __syncthreads();  // every thread has read the length
    if (threadIdx.x == 0 && fits) p.seq_lens[b] = L + p.T;
  }
}

template <typename E, int D>
cudaError_t launch_d(const NormAppend &args, cudaStream_t stream) {
  constexpr int groups = kNormThreads / (D / 2 * (int)sizeof(E) / 16);
  NormAppend p = args;
  const int Hall = p.Hq + 2 * p.Hkv;
  p.tok = 1;
  while (p.tok < p.T && p.tok < groups) p.tok *= 2;
  const int step = groups / p.tok;
  const long long tiles = (p.T + p.tok - 1) / p.tok;
  // heads of a CTA: as many as leave four CTAs to an SM
  const long long want = 4LL * 152;
  long long per = Hall * tiles * p.B / want / step * step;
  if (per < step) per = step;
  if (per > Hall) per = Hall;
  const bool whole = p.advance && tiles == 1 && Hall <= 4 * step;
  if (whole) per = Hall;
  p.per_cta = (int)per;
  p.head_groups = (int)((Hall + per - 1) / per);
  const bool apart = p.advance && !whole;
  if (apart) p.advance = 0;
  cudaError_t e = launch_pdl(norm_append_kernel<E, D>, dim3((unsigned)(tiles * p.head_groups), p.B), dim3(kNormThreads), 0,
                             stream, p);
  if (e == cudaSuccess && apart) e = launch_advance(p.seq_lens, p.B, p.T, p.Smax, stream);
  return e;
}

}  // namespace

cudaError_t launch_norm_append(size_t elem_bytes, int D, const NormAppend &p, cudaStream_t stream) {
  if (elem_bytes == 2) return D == 64 ? launch_d<__nv_bfloat16, 64>(p, stream) : launch_d<__nv_bfloat16, 128>(p, stream);
  return D == 64 ? launch_d<float, 64>(p, stream) : launch_d<float, 128>(p, stream);
}

}  // namespace td
