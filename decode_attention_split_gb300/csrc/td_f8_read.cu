// Read-back of the block-scaled 8-bit cache: rows start[b] .. start[b]+N-1 of every head as
// code * scale in bf16 or fp32, K and V in one launch; rows at or past the sequence's length (and
// before row 0) leave the output as it was. Bound by memory: one byte read and 2 or 4 written per
// element. A thread converts 16 bytes of output at a time, with kReadVecs such loads in flight.
#include "td_f8.cuh"
#include "td_internal.h"

namespace td {

namespace {

constexpr int kReadThreads = 256;
constexpr int kReadVecs = 4;  // vectors of a thread, loads first

// blockIdx: x the tile of rows, y the head (K heads, then V heads), z the sequence
template <typename E, int D>
__global__ void __launch_bounds__(kReadThreads) read_f8_kernel(const ReadF8 p) {
  constexpr int VE = 16 / sizeof(E), NV = D / VE, ROWS = kReadThreads * kReadVecs / NV;
  const int b = blockIdx.z, tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int raw = p.seq_lens[b];
  const int first = p.start != nullptr ? p.start[b] : 0;
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
    if (raw < 0) report(p.status, TD_DEV_NEGATIVE_SEQLEN);
    if (raw > p.Smax) report(p.status, TD_DEV_SEQLEN_CLAMPED);
  }
  const int L = min(max(raw, 0), p.Smax);
  const bool isv = (int)blockIdx.y >= p.Hkv;
  const long long head = (long long)b * p.Hkv + (isv ? blockIdx.y - p.Hkv : blockIdx.y);
  const uint8_t *codes = (isv ? p.v_codes : p.k_codes) + head * p.Smax * D;
  const float *scales = (isv ? p.v_scales : p.k_scales) + head * p.NB;
  E *out = static_cast<E *>(isv ? p.v_out : p.k_out) + head * p.N * D;
  const int t0 = blockIdx.x * ROWS;
  uint2 w[kReadVecs];
  float s[kReadVecs];
  bool in[kReadVecs];
#pragma unroll
  for (int k = 0; k < kReadVecs; ++k) {
    const int i = tid + k * kReadThreads;
    const int t = t0 + i / NV;
    const long long j = (long long)first + t;
    in[k] = t < p.N && j >= 0 && j < L;
    if (in[k]) {
      const uint8_t *src = codes + j * D + (i % NV) * VE;
      if constexpr (VE == 8)
        w[k] = *reinterpret_cast<const uint2 *>(src);
      else
        w[k].x = *reinterpret_cast<const uint32_t *>(src);
      s[k] = scales[j >> p.block_log2];
    }
  }
#pragma unroll
  for (int k = 0; k < kReadVecs; ++k) {
    if (!in[k]) continue;
    const int i = tid + k * kReadThreads;
    float f[VE];
#pragma unroll
    for (int e = 0; e < VE; e += 2) {
      const uint32_t word = e < 4 ? w[k].x : w[k].y;
      const float2 v = e4m3x2_float2((uint16_t)(word >> (8 * (e & 3))));
      f[e] = v.x * s[k];
      f[e + 1] = v.y * s[k];
    }
    uint4 o;
    E *oe = reinterpret_cast<E *>(&o);
#pragma unroll
    for (int e = 0; e < VE; ++e) store_elem<E>(oe + e, f[e]);
    *reinterpret_cast<uint4 *>(out + (long long)(t0 + i / NV) * D + (i % NV) * VE) = o;
  }
}

template <typename E, int D>
cudaError_t launch(const ReadF8 &p, cudaStream_t stream) {
  constexpr int ROWS = kReadThreads * kReadVecs / (D * (int)sizeof(E) / 16);
  return launch_pdl(read_f8_kernel<E, D>, dim3((p.N + ROWS - 1) / ROWS, 2 * p.Hkv, p.B), dim3(kReadThreads), 0, stream,
                    p);
}

}  // namespace

cudaError_t launch_read_f8(size_t elem_bytes, int D, const ReadF8 &p, cudaStream_t stream) {
  if (elem_bytes == 2) return D == 64 ? launch<__nv_bfloat16, 64>(p, stream) : launch<__nv_bfloat16, 128>(p, stream);
  return D == 64 ? launch<float, 64>(p, stream) : launch<float, 128>(p, stream);
}

}  // namespace td
