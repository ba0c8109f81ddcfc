// ckpt8.cu -- the expert MLP's gated activation for training, with gate_up
// kept in 8 bits between the forward and the backward pass.
//
// Forward, per row:  h = silu(g) * u,  and the checkpoint of the row's 2I
// gate_up values as MXFP8: per 32 consecutive values X = max(floor(log2(max
// |v|)) - 7, -127), code = e4m3(v * 2^-X), ties to even.  The exponent leaves
// one binade of headroom (as the two-term split's hi term does), so nothing
// saturates (but 1.9375 2^127 and above, kept as 1.875 2^127: the next e4m3
// value is no fp32 number) and every element keeps 4 significant bits down to
// 2^-13 of the block's largest; the OCP exponent (- 8) would clip values above
// 448/512 of their binade by up to 1/8.  A non-finite value is stored as the e4m3 NaN
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
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace gnf4 {
namespace {

constexpr int kThreads = 256;                                                     // forward
constexpr int row_threads(int wpr) { return wpr == 8 ? 256 : 128; }               // backward (smaller CTAs: 4% faster)

__device__ __forceinline__ uint32_t cvt_e4m3x2(float hi, float lo) {
  uint16_t pr;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pr) : "f"(hi), "f"(lo));
  return pr;
}
// e4m3 pair (low byte = first element) -> two floats, exactly (through f16).
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t pr) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)pr));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two floats in a register pair, for the packed fp32 instructions: the forward
// kernel is bound by issue before it is by memory (78% of the issue slots with
// one value per instruction; 89 us for 32768 rows of 2048, 86 packed).  The
// backward kernel has three outputs to hold: its pairs cost registers, and the
// loads in flight with them (97 us instead of 92).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 both(float a) { return pair(a, a); }

// s = 1 / (1 + 2^(-g log2 e)), computed as 4 s = 1 / (1/4 + 2^(-g log2 e - 2)):
// the approximate reciprocal flushes results below 2^-126, which this moves to
// where 1 + e^-g overflows in fp32 anyway (g < -88.7: s = 0).  The approximate
// instructions are within a few units of 2^-23, the exponent's rounding adds
// (1 + |g|) 2^-23 at most: below a bf16 step even at g = -88.
__device__ __forceinline__ float exp2_approx(float x) {
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
__device__ __forceinline__ float rcp_approx(float x) {
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x));
  return x;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_f32(float g) {
  return 0.25f * rcp_approx(0.25f + exp2_approx(fmaf(-kLog2e, g, -2.0f)));
}
__device__ __forceinline__ F2 sigmoid2_times4(F2 g) {
  const float2 e = split(fma2(g, both(-kLog2e), both(-2.0f)));
  const float2 d = split(add2(pair(exp2_approx(e.x), exp2_approx(e.y)), both(0.25f)));
  return pair(rcp_approx(d.x), rcp_approx(d.y));
}

__device__ __forceinline__ void unpack8(uint4 v, F2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack2(F2 f) {
  const float2 p = split(f);
  __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
  return *reinterpret_cast<uint32_t*>(&b);
}
__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
  return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

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

// Eight consecutive values f (bf16 bits v) of a 32-block shared by lanes
// 4i..4i+3: the codes, and the scale byte (the same in the four lanes).
__device__ __forceinline__ uint2 quant8(uint4 v, const F2 (&f)[4], uint32_t* scale) {
  // |bf16| compares like its bits with the sign cleared
  uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  m = max(m & 0xFFFFu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const bool rare = m >= 0x7F00u;  // values from 2^127 on, or an infinity or a NaN, which stay out of the maximum
  const bool any_rare = __any_sync(0xffffffffu, rare);
  if (any_rare) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = w[i] & 0x7FFFu, b = (w[i] >> 16) & 0x7FFFu;
      n = max(n, max(a >= 0x7F80u ? 0u : a, b >= 0x7F80u ? 0u : b));
    }
    n = max(n, __shfl_xor_sync(0xffffffffu, n, 1));
    m = max(n, __shfl_xor_sync(0xffffffffu, n, 2));
  }
  // exponent field of the maximum - 7 (one binade of headroom), at least that of the smallest scale: 2^-127
  const int X = max((int)(m >> 7) - 127 - 7, -127);
  const float inv = __uint_as_float((uint32_t)(127 - X) << 23);  // 2^-X: 127 - X is in [7, 254]
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = split(mul2(f[i], both(inv)));
    out[i >> 1] |= cvt_e4m3x2(a.y, a.x) << (16 * (i & 1));
  }
  if (any_rare) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 p = split(f[i >> 1]);
      const uint32_t at = 8 * (i & 3), c = (out[i >> 2] >> at) & 0x7Fu;
      if (!isfinite(i & 1 ? p.y : p.x))  // the conversion stores an infinity as 448
        out[i >> 2] = (out[i >> 2] & ~(0xFFu << at)) | (0x7Fu << at);
      else if (X == 120 && c == 0x78u)  // 256 2^120 is no fp32 number: the value below, 240
        out[i >> 2] -= 1u << at;
    }
  }
  *scale = (uint32_t)(X + 127);
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ int live_rows(const int* num_rows, int M) {
  return num_rows == nullptr ? M : min(max(__ldg(num_rows), 0), M);
}

// One thread, PER times: 8 gate values, the 8 matching up values, 8 outputs.
// All loads of a thread are issued before the first is used.  32768 rows of
// 2048: 86 us (6.3 TB/s) with PER = 4, 9 us more with 1; 72 rows of 1024: 2.0
// us with 1, 3.6 with 4, so few values take 1.  64 registers (4 CTAs per SM): 8 us
// less than the 76 the compiler takes by itself.
template <typename Idx, int PER>
__global__ void __launch_bounds__(kThreads, PER == 4 && sizeof(Idx) == 4 ? 4 : 1)
    swiglu_ckpt8_kernel(const __nv_bfloat16* __restrict__ gate_up, int M, int I8, const int* __restrict__ num_rows,
                        uint4* __restrict__ h, uint2* __restrict__ codes, uint8_t* __restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int rows = live_rows(num_rows, M);
  const Idx total = (Idx)rows * (Idx)I8;  // a multiple of 4: lanes 4i..4i+3 are in or out together
  const Idx o0 = (Idx)blockIdx.x * (kThreads * PER) + threadIdx.x;
  uint4 gv[PER], uv[PER];
  size_t at[PER];  // octet of the gate values
  int c[PER];
#pragma unroll
  for (int n = 0; n < PER; ++n) {
    const Idx o = o0 + n * kThreads;
    const bool ok = o < total;
    const Idx r = ok ? o / (Idx)I8 : 0;
    c[n] = ok ? (int)(o - r * (Idx)I8) : -1;
    at[n] = (size_t)r * 2 * I8 + (ok ? c[n] : 0);
    if (!ok) at[n] = 0;
    const uint4* src = reinterpret_cast<const uint4*>(gate_up) + at[n];
    gv[n] = uv[n] = make_uint4(0u, 0u, 0u, 0u);
    if (ok) gv[n] = ldg_nc_u128(src), uv[n] = ldg_nc_u128(src + I8);
  }
#pragma unroll
  for (int n = 0; n < PER; ++n) {
    F2 g[4], u[4];
    unpack8(gv[n], g);
    unpack8(uv[n], u);
    uint32_t gs, us;
    const uint2 gc = quant8(gv[n], g, &gs), uc = quant8(uv[n], u, &us);
    if (c[n] < 0) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = mul2(mul2(mul2(g[i], both(0.25f)), sigmoid2_times4(g[i])), u[i]);
    h[(at[n] + c[n]) >> 1] = pack8(g);  // at = 2 I8 row + c, h lies at I8 row + c
    codes[at[n]] = gc;
    codes[at[n] + I8] = uc;
    if ((c[n] & 3) == 0) {
      scales[at[n] >> 2] = (uint8_t)gs;
      scales[(at[n] + I8) >> 2] = (uint8_t)us;
    }
  }
}

// WPR warps per row, a lane's next 16 values fetched while it works on the
// present ones; the row's dot product is added lane by lane, then by shuffles,
// then warp by warp.  32768 rows of 2048 in 92 us (5.9 TB/s; without the early
// fetch and with 59 registers per thread 106 us).
template <int WPR>
__global__ void __launch_bounds__(row_threads(WPR), 1280 / row_threads(WPR)) swiglu_ckpt8_backward_kernel(
    const uint4* __restrict__ dh, const uint2* __restrict__ codes, const uint8_t* __restrict__ scales,
    const int* __restrict__ num_rows, const int* __restrict__ s2f, const int* __restrict__ f2s,
    const float* __restrict__ weights, int M, int I8, uint4* __restrict__ dgu, uint4* __restrict__ h,
    float* __restrict__ d_weights) {
  constexpr int kWarps = row_threads(WPR) / 32;
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
    struct {
      uint2 g, u;
      uint4 d;
      uint32_t gs, us;
    } now, next = {};
    auto fetch = [&](int c) {
      if (c >= I8) return;
      next.g = ldg_nc_u64(codes + row + c);
      next.u = ldg_nc_u64(codes + row + I8 + c);
      next.d = ldg_nc_u128(dhr + c);
      next.gs = __ldg(scales + ((row + c) >> 2));
      next.us = __ldg(scales + ((row + I8 + c) >> 2));
    };
    int c = (warp % WPR) * 32 + lane;
    fetch(c);
    for (; c < I8; c += 32 * WPR) {
      now = next;
      fetch(c + 32 * WPR);
      float g[8], u[8], d[8], hv[8];
      decode8(now.g, e8m0_to_f32(now.gs), g);
      decode8(now.u, e8m0_to_f32(now.us), u);
      unpack8(now.d, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = sigmoid_f32(g[i]);
        const float gsig = g[i] * s;  // silu(g)
        const float slope = s * fmaf(g[i], 1.0f - s, 1.0f);
        hv[i] = gsig * u[i];
        dot = fmaf(d[i], hv[i], dot);
        const float wd = w * d[i];
        g[i] = slope * (u[i] * wd);  // slope (at most 1.1) times the largest u may pass fp32
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
  auto launch = [&](auto* kernel, int per) {
    const long long chunk = (long long)kThreads * per;
    return launch_pdl(kernel, dim3((unsigned)((octets + chunk - 1) / chunk)), dim3(kThreads), 0, stream, gate_up, M,
                      I / 8, num_rows, reinterpret_cast<uint4*>(h), reinterpret_cast<uint2*>(codes), scales);
  };
  if (octets < (1LL << 18)) return launch(swiglu_ckpt8_kernel<uint32_t, 1>, 1);  // under one wave of CTAs
  if (octets < (1LL << 31)) return launch(swiglu_ckpt8_kernel<uint32_t, 4>, 4);
  return launch(swiglu_ckpt8_kernel<unsigned long long, 4>, 4);
}

cudaError_t launch_swiglu_ckpt8_backward(const __nv_bfloat16* dh, const uint8_t* codes, const uint8_t* scales,
                                         const int32_t* num_rows, const int32_t* s2f, const int32_t* f2s,
                                         const float* weights, int M, int I, __nv_bfloat16* d_gate_up,
                                         __nv_bfloat16* h, float* d_weights, cudaStream_t stream) {
  auto launch = [&](auto* kernel, int warps) {
    const int threads = row_threads(warps), rpc = threads / 32 / warps;  // rows per CTA
    return launch_pdl(kernel, dim3((unsigned)((M + rpc - 1LL) / rpc)), dim3((unsigned)threads), 0, stream,
                      reinterpret_cast<const uint4*>(dh), reinterpret_cast<const uint2*>(codes), scales, num_rows, s2f,
                      f2s, weights, M, I / 8, reinterpret_cast<uint4*>(d_gate_up), reinterpret_cast<uint4*>(h),
                      d_weights);
  };
  switch (warps_per_row(M, I / 8)) {
    case 8: return launch(swiglu_ckpt8_backward_kernel<8>, 8);
    case 4: return launch(swiglu_ckpt8_backward_kernel<4>, 4);
    case 2: return launch(swiglu_ckpt8_backward_kernel<2>, 2);
    default: return launch(swiglu_ckpt8_backward_kernel<1>, 1);
  }
}

}  // namespace gnf4
