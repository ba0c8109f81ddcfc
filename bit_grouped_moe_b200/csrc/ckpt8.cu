// ckpt8.cu -- the expert MLP's gated activation for training, with gate_up
// kept in 8 bits between the forward and the backward pass.
//
// Forward, per row:  h = silu(g) * u,  and the checkpoint of the row's 2I
// gate_up values as MXFP8: per 32 consecutive values X = max(floor(log2(max
// |v|)) - 7, -127), code = e4m3(v * 2^-X), ties to even.  The exponent leaves
// one binade of headroom (as the two-term split's hi term does), so nothing
// saturates and every element keeps 4 significant bits down to 2^-13 of the
// block's largest; the OCP exponent (- 8) would clip values above 448/512 of
// their binade by up to 1/8.  A non-finite value is stored as the e4m3 NaN
// and does not enter its block's scale.
//
// Backward, per row with router weight w (1 without routing), from the
// decoded g^, u^ and s = 1 / (1 + exp(-g^)):
//     du = w dh g^ s,   dg = w dh u^ s (1 + g^ (1 - s)),
//     d_weight = sum_i dh[i] g^ s u^,
// where dh is the gradient of the expert output through the down projection
// without w.  The weight's gradient is <dout, y> = <dout, D h> = <D^T dout, h>,
// so it needs neither the expert outputs y nor a second pass.
//
// All arithmetic is fp32 on decoded values; h and the gradients are rounded
// once to bf16, sums stay fp32 and are added in a fixed order.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace gnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float sigmoid_f32(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    o[i] = *reinterpret_cast<uint32_t*>(&b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void decode8(uint2 c, float sc, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = e4m3x2_to_f32(((i & 2 ? c.y : c.x) >> (16 * (i & 1))) & 0xFFFFu);
    f[2 * i] = p.x * sc;
    f[2 * i + 1] = p.y * sc;
  }
}

// Eight consecutive values of a 32-block shared by lanes 4i..4i+3: the codes,
// and the scale byte (the same in the four lanes).
__device__ __forceinline__ uint2 quant8(uint4 v, uint32_t* scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;  // |bf16| compares like its bits with the sign cleared
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFFu, b = (w[i] >> 16) & 0x7FFFu;
    m = max(m, max(a >= 0x7F80u ? 0u : a, b >= 0x7F80u ? 0u : b));
  }
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const int ef = (int)(m >> 7);  // exponent field; 0: zero or subnormal, below the smallest scale
  const int X = ef == 0 ? -127 : max(ef - 127 - 7, -127);
  const float inv = __uint_as_float((uint32_t)(127 - X) << 23);  // 2^-X: 127 - X is in [7, 254]
  float f[8];
  unpack8(v, f);
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    // an infinity times 0 is NaN: the finite-saturating conversion would store it as 448
    const float a = fabsf(f[i]) == INFINITY ? __uint_as_float(0x7fc00000u) : f[i] * inv;
    const float b = fabsf(f[i + 1]) == INFINITY ? __uint_as_float(0x7fc00000u) : f[i + 1] * inv;
    out[i >> 2] |= cvt_e4m3x2(b, a) << (8 * (i & 2));
  }
  *scale = (uint32_t)(X + 127);
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ int live_rows(const int* num_rows, int M) {
  return num_rows == nullptr ? M : min(max(__ldg(num_rows), 0), M);
}

// One thread: 8 gate values, the 8 matching up values, 8 outputs.
template <typename Idx>
__global__ void __launch_bounds__(kThreads) swiglu_ckpt8_kernel(const __nv_bfloat16* __restrict__ gate_up, int M,
                                                                int I8, const int* __restrict__ num_rows,
                                                                uint4* __restrict__ h, uint2* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int rows = live_rows(num_rows, M);
  const Idx o = (Idx)blockIdx.x * kThreads + threadIdx.x;
  const Idx total = (Idx)rows * (Idx)I8;  // a multiple of 4: lanes 4i..4i+3 are in or out together
  if (o - (threadIdx.x & 31) >= total) return;
  const bool ok = o < total;
  const Idx r = ok ? o / (Idx)I8 : 0;
  const int c = ok ? (int)(o - r * (Idx)I8) : 0;
  const size_t row = (size_t)r * 2 * I8;  // octets
  const uint4* src = reinterpret_cast<const uint4*>(gate_up) + row;
  const uint4 gv = ldg_nc_u128(src + c), uv = ldg_nc_u128(src + I8 + c);
  uint32_t gs, us;
  const uint2 gc = quant8(gv, &gs), uc = quant8(uv, &us);
  if (!ok) return;
  float g[8], u[8];
  unpack8(gv, g);
  unpack8(uv, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = silu_mul(g[i], u[i]);
  h[(size_t)r * I8 + c] = pack8(g);
  codes[row + c] = gc;
  codes[row + I8 + c] = uc;
  if ((c & 3) == 0) {
    scales[(row + c) >> 2] = (uint8_t)gs;
    scales[(row + I8 + c) >> 2] = (uint8_t)us;
  }
}

// WPR warps per row; the row's dot product is added lane by lane, then by
// shuffles, then warp by warp.
template <int WPR>
__global__ void __launch_bounds__(kThreads) swiglu_ckpt8_backward_kernel(
    const uint4* __restrict__ dh, const uint2* __restrict__ codes, const uint8_t* __restrict__ scales,
    const int* __restrict__ num_rows, const int* __restrict__ s2f, const int* __restrict__ f2s,
    const float* __restrict__ weights, int M, int I8, uint4* __restrict__ dgu, uint4* __restrict__ h,
    float* __restrict__ d_weights) {
  __shared__ float red[kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * (kWarps / WPR) + warp / WPR;
  const int rows = live_rows(num_rows, M);
  int f = -1;
  bool live = r < rows;
  float w = 1.0f;
  if (live && s2f != nullptr) {
    f = __ldg(s2f + r);
    live = f >= 0 && f < M;
    if (live && weights != nullptr) w = __ldg(weights + f);
  }
  float dot = 0.f;
  if (live) {
    const size_t row = (size_t)r * 2 * I8;
    const uint4* dhr = dh + (size_t)r * I8;
    for (int c = (warp % WPR) * 32 + lane; c < I8; c += 32 * WPR) {
      const uint2 gc = ldg_nc_u64(codes + row + c), uc = ldg_nc_u64(codes + row + I8 + c);
      const uint4 dv = ldg_nc_u128(dhr + c);
      const float gs = e8m0_to_f32(__ldg(scales + ((row + c) >> 2)));
      const float us = e8m0_to_f32(__ldg(scales + ((row + I8 + c) >> 2)));
      float g[8], u[8], d[8], hv[8];
      decode8(gc, gs, g);
      decode8(uc, us, u);
      unpack8(dv, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = sigmoid_f32(g[i]);
        const float gsig = g[i] * s;  // silu(g)
        const float slope = s * fmaf(g[i], 1.0f - s, 1.0f);
        hv[i] = gsig * u[i];
        dot = fmaf(d[i], hv[i], dot);
        const float wd = w * d[i];
        g[i] = slope * u[i] * wd;
        u[i] = gsig * wd;
      }
      dgu[row + c] = pack8(g);
      dgu[row + I8 + c] = pack8(u);
      if (h != nullptr) h[(size_t)r * I8 + c] = pack8(hv);
    }
  }
  if (d_weights == nullptr) return;  // uniform over the grid
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if (WPR > 1) {
    if (lane == 0) red[warp] = dot;
    __syncthreads();
  }
  if (lane == 0 && warp % WPR == 0 && r < M) {
    if (WPR > 1)
      for (int i = 1; i < WPR; ++i) dot += red[warp + i];
    if (live) d_weights[f] = dot;
    const int q = __ldg(f2s + r);  // pair r: a pair without a live row has no gradient
    if (q < 0 || q >= rows) d_weights[r] = 0.f;
  }
}

}  // namespace

cudaError_t launch_swiglu_ckpt8(const __nv_bfloat16* gate_up, int M, int I, const int32_t* num_rows,
                                __nv_bfloat16* h, uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  const long long octets = (long long)M * (I / 8);
  const long long grid = (octets + kThreads - 1) / kThreads;
  auto* kernel = octets < (1LL << 31) ? swiglu_ckpt8_kernel<uint32_t> : swiglu_ckpt8_kernel<unsigned long long>;
  return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), 0, stream, gate_up, M, I / 8, num_rows,
                    reinterpret_cast<uint4*>(h), reinterpret_cast<uint2*>(codes), scales);
}

cudaError_t launch_swiglu_ckpt8_backward(const __nv_bfloat16* dh, const uint8_t* codes, const uint8_t* scales,
                                         const int32_t* num_rows, const int32_t* s2f, const int32_t* f2s,
                                         const float* weights, int M, int I, __nv_bfloat16* d_gate_up,
                                         __nv_bfloat16* h, float* d_weights, cudaStream_t stream) {
  const int rpc = kWarps;  // rows per CTA
  return launch_pdl(swiglu_ckpt8_backward_kernel<1>, dim3((unsigned)((M + rpc - 1LL) / rpc)), dim3(kThreads), 0,
                    stream, reinterpret_cast<const uint4*>(dh), reinterpret_cast<const uint2*>(codes), scales, num_rows, s2f,
                    f2s, weights, M, I / 8, reinterpret_cast<uint4*>(d_gate_up), reinterpret_cast<uint4*>(h), d_weights);
}

}  // namespace gnf4
