// backward.cu -- backward passes of the two ends of a routed layer: the top-k
// weighted sum (combine) and the router's top-k softmax.
//
// combine:  out[t] = sum_j w[t,j] y[f2s[t*k+j]], so with f = s2f[r], t = f / k
//     dy[r] = w[f] dout[t],   d_w[f] = <dout[t], y[r]>.
// Rows without a pair (s2f[r] < 0) are written as zeros: the data gradient
// GEMM may read them.  dout rows are read once per slot through L2 (a token's
// rows are scattered over the experts), y and dy stream once.
//
// router:  p = softmax of the k selected logits, the others do not enter, so
//     d_logit[t, id_j] = p_j (d_j - sum_i p_i d_i),   0 elsewhere.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace gnf4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// WPR warps per row; one lane moves 8 values with 16-byte loads and stores.
// Rows in their own order: y and dy stream, and a token's dout is read k times
// from the L2.  2048 tokens, top-8, 2048 wide: 28.6 us (a plain copy of the
// same bytes 25), as a gather 14.9 (floor 11.7; 4096 tokens 27.0, floor 23.4);
// in the order of the pairs, whose warps share dout in the L1
// but scatter the rows, 30.0; with four pieces of a row unrolled 33.3.
template <int WPR>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(
    const uint4* __restrict__ dout, const uint4* __restrict__ y, const int* __restrict__ s2f,
    const int* __restrict__ f2s, const float* __restrict__ weights, int M, int k, int N8, uint4* __restrict__ dy,
    float* __restrict__ d_weights) {
  __shared__ float red[kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * (kWarps / WPR) + warp / WPR;
  const int f = r < M ? __ldg(s2f + r) : -1;
  const bool live = f >= 0 && f < M;
  float dot = 0.f;
  if (r < M) {
    uint4* dst = dy + (size_t)r * N8;
    const int c0 = (warp % WPR) * 32 + lane;
    if (!live) {
      for (int c = c0; c < N8; c += 32 * WPR) dst[c] = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4* src = dout + (size_t)(f / k) * N8;
      const float w = weights != nullptr ? __ldg(weights + f) : 1.0f;
      for (int c = c0; c < N8; c += 32 * WPR) {
        const uint4 v = ldg_u128(src + c);
        const uint32_t a[4] = {v.x, v.y, v.z, v.w};
        if (y != nullptr) {
          const uint4 q = ldg_nc_u128(y + (size_t)r * N8 + c);
          const uint32_t b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dot = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), dot);
            dot = fmaf(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u), dot);
          }
        }
        uint4 o = v;
        if (weights != nullptr) {
          uint32_t s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 p =
                __floats2bfloat162_rn(w * __uint_as_float(a[i] << 16), w * __uint_as_float(a[i] & 0xFFFF0000u));
            s[i] = *reinterpret_cast<uint32_t*>(&p);
          }
          o = make_uint4(s[0], s[1], s[2], s[3]);
        }
        dst[c] = o;
      }
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
    const int q = __ldg(f2s + r);  // pair r: a dropped pair has no gradient
    if (q < 0 || q >= M) d_weights[r] = 0.f;
  }
}

// One warp per token (k <= 32): lane j holds slot j.  The row is zeroed, then
// the slots' values are stored over it; a slot whose expert appeared in an
// earlier slot adds to that one, so a repeated id neither races nor is lost.
__global__ void __launch_bounds__(kThreads) route_topk_backward_kernel(const int* __restrict__ ids,
                                                                       const float* __restrict__ probs,
                                                                       const float* __restrict__ dw, int T, int k,
                                                                       int E, float* __restrict__ d_logits) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= T) return;
  const size_t f = (size_t)t * k + lane;
  int id = -1;
  float p = 0.f, d = 0.f;
  if (lane < k) {
    id = __ldg(ids + f);
    p = __ldg(probs + f);
    d = __ldg(dw + f);
  }
  if (id < 0 || id >= E) id = -1;
  float s = lane < k ? p * d : 0.f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float v = p * (d - s);
  float* row = d_logits + (size_t)t * E;
  if ((E & 3) == 0 && (reinterpret_cast<uintptr_t>(d_logits) & 15u) == 0) {
    for (int e = 4 * lane; e < E; e += 128) *reinterpret_cast<float4*>(row + e) = make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    for (int e = lane; e < E; e += 32) row[e] = 0.f;
  }
  float sum = v;
  bool first = true;
  for (int j = 0; j < k; ++j) {
    const int oi = __shfl_sync(0xffffffffu, id, j);
    const float ov = __shfl_sync(0xffffffffu, v, j);
    if (oi == id && j < lane) first = false;
    if (oi == id && j > lane) sum += ov;
  }
  __syncwarp();  // the zeros before the values
  if (id >= 0 && first) row[id] = sum;
}

}  // namespace

cudaError_t launch_combine_backward(const __nv_bfloat16* dout, const __nv_bfloat16* y, const int32_t* s2f,
                                    const int32_t* f2s, const float* weights, int M, int k, int N,
                                    __nv_bfloat16* dy, float* d_weights, cudaStream_t stream) {
  auto launch = [&](auto* kernel, int warps) {
    const int rpc = kWarps / warps;  // rows per CTA
    return launch_pdl(kernel, dim3((unsigned)((M + rpc - 1LL) / rpc)), dim3(kThreads), 0, stream,
                      reinterpret_cast<const uint4*>(dout), reinterpret_cast<const uint4*>(y), s2f, f2s, weights, M, k,
                      N / 8, reinterpret_cast<uint4*>(dy), d_weights);
  };
  switch (warps_per_row(M, N / 8)) {
    case 8: return launch(combine_backward_kernel<8>, 8);
    case 4: return launch(combine_backward_kernel<4>, 4);
    case 2: return launch(combine_backward_kernel<2>, 2);
    default: return launch(combine_backward_kernel<1>, 1);
  }
}

cudaError_t launch_route_topk_backward(const int32_t* ids, const float* probs, const float* d_weights, int T, int k,
                                       int E, float* d_logits, cudaStream_t stream) {
  return launch_pdl(route_topk_backward_kernel, dim3((unsigned)((T + kWarps - 1LL) / kWarps)), dim3(kThreads), 0,
                    stream, ids, probs, d_weights, T, k, E, d_logits);
}

}  // namespace gnf4
