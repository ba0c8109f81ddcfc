// moe_decode.cu -- a whole routed MoE layer for a few tokens (T <= 8) in one
// launch, on the packed 4-bit expert stacks:
//   logits = x Wr^T (or given), ids / p = top-k softmax,
//   h[t, e] = silu(G_e x_t) * (U_e x_t),   out[t] = sum_j p[t,j] D_{e_j} h[t, e_j].
//
// The bytes are the hit experts' weights, each read once; everything between
// them is latency.  So one cooperative kernel, one CTA of 16 warps per SM,
// runs the phases with a grid barrier between them:
//   0 router: a CTA computes the logits of its experts (skipped when given);
//   1 every CTA selects the top-k of every token itself (a warp per token) and
//     lists the hit experts: cheaper than a barrier around one CTA doing it;
//   2 gate_up + SwiGLU: work unit = 8 gate rows and the 8 matching up rows of
//     a hit expert, one m16 tile, so a lane ends with both halves of a value;
//   3 down + combine: work unit = 16 output rows over ALL hit experts: the
//     router weight is folded into h, so the weighted sum over the experts is
//     the same fp32 accumulator and no per-expert output exists.
// A unit's K (phase 3: hit experts x K) is cut in items of 128 k; the item
// sequence of a CTA is divided evenly over its 16 warps and each warp streams
// a contiguous range, so every warp has the same number of 1 KB loads
// whatever the shapes are.  A warp that covers a whole unit finishes it in
// registers; split units are added through shared memory in warp order.  In
// phase 3 the item sequence is also divided evenly over the CTAs (16-row
// units would leave up to 39% of the SMs idle); a unit split between CTAs is
// added by the last CTA to finish it, in CTA order, from partial sums in the
// workspace.  Every sum has a fixed order: outputs do not depend on timing.
//
// MMA mapping (m16n8k16): A = decoded weights, B = activations, the MMA's 8
// columns are the T tokens.  In phase 2 all tokens share B, whichever expert
// they chose: products of tokens that did not choose it are computed (the
// MMA has the columns anyway) and dropped.  x lies in shared memory in
// fragment order.  In phase 3 lanes of tokens that did not choose the expert
// hold zeros.
//
// Decode: the per-lane pair table of the grouped GEMV (a byte = one PRMT and
// one shared load).
//   MXFP4: e2m1 x 2^(e-127) is exact in bf16 (a power-of-two multiply per pair).
//   NF4: a lane's 16 codes of a 64-block feed four MMAs whose fp32 result is
//     multiplied by absmax, so absmax is not rounded.  The codes are rounded
//     to bf16 after a multiplication by kNf4Gain, undone in fp32: the gain is
//     the one in [1, 2) that minimises the rounding error of the 16 codes
//     (rms 0.063% instead of 0.106%).
// Rounded to bf16: h times its router weight (once, from fp32), and out.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace gnf4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxT = kMoeDecodeMaxTokens;
constexpr int kMaxPairs = kMaxT * kMaxRouterTopK;  // hit experts never exceed this
constexpr int kMaxGrid = 160;                      // CTAs (one per SM; B200 has 148)
constexpr int kDK = 128;                           // k per item
constexpr int kStages = 4;                         // items in flight per warp
constexpr float kNf4Gain = 1.43701171875f;

// Shared memory: the pair table needs a 64 KB boundary of the shared window.
// x in fragment order goes below it: it starts at the first boundary that
// leaves room (0x10000 or 0x20000).  Everything else lies above the table.
struct Tables {
  float part[kWarps][2][32][4];       // partial sums: [0] of a unit begun by an earlier warp, [1] of one begun here
  float wt[kMaxPairs][kMaxT];         // router weight of (hit expert, token), 0 if not routed
  short row[kMaxPairs][kMaxT];        // row of hbuf of (hit expert, token), -1 if not routed
  short expert[kMaxPairs];            // hit expert ids, ascending
  uint32_t hit[kMaxExperts / 32];     // bit per expert
  float red[kWarps][kMaxT];           // router products per warp
  int sel_id[kMaxT][kMaxRouterTopK];
  float sel_p[kMaxT][kMaxRouterTopK];
  int nhit;
  int ok;
};

constexpr uint32_t kWindow = 0x400;  // start of the dynamic shared window that the host's layout assumes
constexpr int kSyncBytes = 256;      // workspace: words 0, 1 = grid barriers, 2 = CTAs that have left

template <int FMT>
__device__ __forceinline__ void build_table(uint32_t* lut, int tid) {
  for (int i = tid; i < 256 * 32; i += kThreads) {
    const uint32_t b = (uint32_t)i >> 5, l = (uint32_t)i & 31u;
    float lo, hi;
    if (FMT == 0) {
      lo = kNf4Code[b >> 4] * kNf4Gain;
      hi = kNf4Code[b & 15u] * kNf4Gain;
    } else {
      lo = e2m1_value(b & 15u);
      hi = e2m1_value(b >> 4);
    }
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    lut[b * 64u + l] = *reinterpret_cast<uint32_t*>(&v);
  }
}

// Byte j of `word` selects the entry; `lanesel` holds 4*lane in byte 0 and the table's 64 KB base in byte 2.
__device__ __forceinline__ uint32_t lookup(uint32_t word, uint32_t lanesel, uint32_t j) {
  uint32_t v;
  asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(prmt_b32(word, lanesel, 0x7604u | (j << 4))));
  return v;
}

// Offset inside a 128-k item of the 8 consecutive k that chunk c (0..3) of lane column t holds.
template <int FMT>
__device__ __forceinline__ int chunk_k(int t, int c) {
  return FMT == 0 ? 64 * (c >> 1) + 16 * t + 8 * (c & 1) : 32 * t + 8 * c;
}

// All CTAs of the grid meet (cooperative launch: they are all resident).
// Bounded: false after the wait limit, with the timeout flagged.
__device__ __forceinline__ bool grid_barrier(unsigned* ctr, unsigned* err, int* ok) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(ctr, 1u);
    const long long t0 = clock64();
    int good = 1;
    while (true) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
      if (v >= gridDim.x) break;
      if (clock64() - t0 > kSpinLimitCycles) {
        atomicOr(err, GNF4_DEVERR_TIMEOUT);
        good = 0;
        break;
      }
    }
    __threadfence();
    *ok = good;
  }
  __syncthreads();
  return *ok != 0;
}

// ---------------------------------------------------------------- router

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float acc) {
  const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(__uint_as_float(p[i] << 16), __uint_as_float(q[i] << 16), acc);
    acc = fmaf(__uint_as_float(p[i] & 0xFFFF0000u), __uint_as_float(q[i] & 0xFFFF0000u), acc);
  }
  return acc;
}

__device__ __forceinline__ void router_product(const MoeDecodeArgs& p, Tables& s, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  const int H8 = p.H / 8;
  const uint4* x = reinterpret_cast<const uint4*>(p.x);
  for (int e = blockIdx.x; e < p.E; e += gridDim.x) {
    const uint4* w = reinterpret_cast<const uint4*>(p.router_w) + (size_t)e * H8;
    float acc[kMaxT];
#pragma unroll
    for (int t = 0; t < kMaxT; ++t) acc[t] = 0.f;
    for (int i = tid; i < H8; i += kThreads) {
      const uint4 wv = ldg_nc_u128(w + i);
#pragma unroll
      for (int t = 0; t < kMaxT; ++t)
        if (t < p.T) acc[t] = dot8(wv, ldg_u128(x + (size_t)t * H8 + i), acc[t]);
    }
#pragma unroll
    for (int t = 0; t < kMaxT; ++t) {
      if (t >= p.T) break;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], d);
      if (lane == 0) s.red[warp][t] = acc[t];
    }
    __syncthreads();
    if (tid < p.T) {
      float v = 0.f;
      for (int i = 0; i < kWarps; ++i) v += s.red[i][tid];
      p.logits[(size_t)tid * p.E + e] = v;
    }
    __syncthreads();
  }
}

// Order-preserving key of a score: larger is better, equal floats (-0 and 0)
// equal, NaN below every number (1), 0 = taken.
__device__ __forceinline__ uint32_t score_key(float f) {
  if (f != f) return 1u;
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// One warp, one token: the k best of logit + bias (descending, ties to the
// lower expert, NaN last) and the softmax of their raw logits, as the
// router epilogue of the routing call.
__device__ __forceinline__ void select_topk(const MoeDecodeArgs& p, Tables& s, int t, int lane) {
  const float* row = p.logits + (size_t)t * p.E;
  uint32_t key[kMaxExperts / 32];
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) {
    key[i] = 0u;
    if (i * 32 >= p.E) continue;
    const int e = i * 32 + lane;
    if (e < p.E) {
      float v = __ldcg(row + e);
      if (p.bias != nullptr) v += __ldg(p.bias + e);
      key[i] = score_key(v);
    }
  }
  int mine = 0;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) {
      if (i * 32 >= p.E) break;
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const unsigned id = __reduce_min_sync(0xffffffffu, best == top ? (unsigned)(at * 32 + lane) : 0xFFFFFFFFu);
    if ((int)(id & 31u) == lane) {
#pragma unroll
      for (int i = 0; i < kMaxExperts / 32; ++i)
        if (i == (int)(id >> 5)) key[i] = 0u;
    }
    if (lane == j) mine = (int)id;
  }
  const float l = lane < p.k ? __ldcg(row + mine) : -INFINITY;
  float m = l;  // a NaN logit makes every weight NaN
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, m, d);
    if (m == m && (o != o || o > m)) m = o;
  }
  const float ex = lane < p.k ? expf(l - m) : 0.f;
  float sum = ex;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane < p.k) {
    const float w = ex / sum;
    s.sel_id[t][lane] = mine;
    s.sel_p[t][lane] = w;
    atomicOr(&s.hit[mine >> 5], 1u << (mine & 31));
    if (blockIdx.x == 0) {
      p.topk_ids[t * p.k + lane] = mine;
      p.topk_weights[t * p.k + lane] = w;
    }
  }
}

__device__ __forceinline__ void list_hits(const MoeDecodeArgs& p, Tables& s, int tid) {
  // rank of expert e = set bits below it
  auto rank = [&](int e) {
    int r = __popc(s.hit[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int i = 0; i < (e >> 5); ++i) r += __popc(s.hit[i]);
    return r;
  };
  const int words = (p.E + 31) / 32;
  if (tid == 0) {
    int n = 0;
    for (int i = 0; i < words; ++i) n += __popc(s.hit[i]);
    s.nhit = n;
  }
  for (int e = tid; e < p.E; e += kThreads)
    if ((s.hit[e >> 5] >> (e & 31)) & 1u) s.expert[rank(e)] = (short)e;
  for (int i = tid; i < kMaxPairs * kMaxT; i += kThreads) {
    s.wt[i / kMaxT][i % kMaxT] = 0.f;
    s.row[i / kMaxT][i % kMaxT] = -1;
  }
  __syncthreads();
  for (int i = tid; i < p.T * p.k; i += kThreads) {
    const int t = i / p.k, j = i - t * p.k;
    const int r = rank(s.sel_id[t][j]);
    s.wt[r][t] = s.sel_p[t][j];
    s.row[r][t] = (short)i;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- item stream

template <int FMT>
struct Item {
  uint32_t w[8];                   // 64 codes: MXFP4 16 bytes of row g, of row g+8; NF4 per row 8 bytes of each block
  uint32_t s[FMT == 0 ? 4 : 2];    // MXFP4: scale byte per row; NF4: absmax [row][block]
};

// A tile's row g of this lane and its scales; the second row lies `hi` rows further.
struct Rows {
  const uint8_t* w;
  const uint8_t* s;
};

template <int FMT>
__device__ __forceinline__ void load_item(Item<FMT>& it, const Rows& r, size_t w_hi, size_t s_hi, int d, int K, int t) {
  if (FMT == 1) {
    const bool ok = d * kDK + 32 * t < K;
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    it.s[0] = it.s[1] = 0u;
    if (ok) {
      const uint8_t* w = r.w + (size_t)d * (kDK / 2) + 16 * t;
      const uint8_t* s = r.s + 4 * d + t;
      a = ldg_nc_u128(w);
      b = ldg_nc_u128(w + w_hi);
      it.s[0] = __ldg(s);
      it.s[1] = __ldg(s + s_hi);
    }
    it.w[0] = a.x, it.w[1] = a.y, it.w[2] = a.z, it.w[3] = a.w;
    it.w[4] = b.x, it.w[5] = b.y, it.w[6] = b.z, it.w[7] = b.w;
  } else {
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      const bool ok = d * kDK + 64 * blk < K;
      uint2 a = make_uint2(0u, 0u), b = a;
      it.s[blk] = it.s[2 + blk] = 0u;
      if (ok) {
        const uint8_t* w = r.w + (size_t)d * (kDK / 2) + 32 * blk + 8 * t;
        const uint8_t* s = r.s + (size_t)(2 * d + blk) * 4;
        a = ldg_nc_u64(w);
        b = ldg_nc_u64(w + w_hi);
        it.s[blk] = __ldg(reinterpret_cast<const unsigned*>(s));
        it.s[2 + blk] = __ldg(reinterpret_cast<const unsigned*>(s + s_hi));
      }
      it.w[2 * blk] = a.x, it.w[2 * blk + 1] = a.y;
      it.w[4 + 2 * blk] = b.x, it.w[5 + 2 * blk] = b.y;
    }
  }
}

// acc += the item's 16 x 128 weights times the lane's activations (chunk c = two MMAs).
template <int FMT>
__device__ __forceinline__ void multiply(float (&acc)[4], const Item<FMT>& it, const uint4 (&x)[4], uint32_t lanesel) {
  const uint32_t xp[16] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w,
                           x[2].x, x[2].y, x[2].z, x[2].w, x[3].x, x[3].y, x[3].z, x[3].w};
  if (FMT == 1) {
    const uint32_t s0 = e8m0_to_bf16x2(it.s[0]), s1 = e8m0_to_bf16x2(it.s[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // bytes 2j, 2j+1 of both rows
      const uint32_t b = 2u * (uint32_t)(j & 1);
      const uint32_t a0 = bf16x2_mul(lookup(it.w[j >> 1], lanesel, b), s0);
      const uint32_t a1 = bf16x2_mul(lookup(it.w[4 + (j >> 1)], lanesel, b), s1);
      const uint32_t a2 = bf16x2_mul(lookup(it.w[j >> 1], lanesel, b + 1u), s0);
      const uint32_t a3 = bf16x2_mul(lookup(it.w[4 + (j >> 1)], lanesel, b + 1u), s1);
      mma_bf16_16816(acc, a0, a1, a2, a3, xp[2 * j], xp[2 * j + 1]);
    }
  } else {
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 4 * blk; j < 4 * blk + 4; ++j) {
        const uint32_t b = 2u * (uint32_t)(j & 1);
        mma_bf16_16816(d, lookup(it.w[j >> 1], lanesel, b), lookup(it.w[4 + (j >> 1)], lanesel, b),
                       lookup(it.w[j >> 1], lanesel, b + 1u), lookup(it.w[4 + (j >> 1)], lanesel, b + 1u), xp[2 * j],
                       xp[2 * j + 1]);
      }
      const float s0 = __uint_as_float(it.s[blk]), s1 = __uint_as_float(it.s[2 + blk]);
      acc[0] = fmaf(s0, d[0], acc[0]);
      acc[1] = fmaf(s0, d[1], acc[1]);
      acc[2] = fmaf(s1, d[2], acc[2]);
      acc[3] = fmaf(s1, d[3], acc[3]);
    }
  }
}

// One phase's view of its item sequence: unit u = items [u * per, (u + 1) * per).
template <int FMT, int PHASE>
struct Stream {
  const MoeDecodeArgs& p;
  const Tables& s;
  const uint4* xs;  // shared x in fragment order (phase 2)
  int g, t, K, nd, per, cols;  // nd: items of one expert; cols: units of an expert (phase 2)
  size_t w_hi, s_hi, wrow, srow;

  __device__ __forceinline__ Stream(const MoeDecodeArgs& p_, const Tables& s_, const uint4* xs_, int lane)
      : p(p_), s(s_), xs(xs_), g(lane >> 2), t(lane & 3) {
    K = PHASE == 2 ? p.H : p.I;
    nd = (K + kDK - 1) / kDK;
    cols = p.I / 8;
    per = PHASE == 2 ? nd : nd * s.nhit;
    wrow = (size_t)(K / 2);
    srow = FMT == 0 ? (size_t)(K / 64) * 4 : (size_t)(K / 32);
    const size_t hi = PHASE == 2 ? (size_t)p.I : 8;
    w_hi = hi * wrow;
    s_hi = hi * srow;
  }
  __device__ __forceinline__ Rows rows(int unit, int ei) const {
    // phase 2: unit = (hit expert, 8 columns); phase 3: unit = 16 output rows, ei = hit expert
    const int e = PHASE == 2 ? s.expert[unit / cols] : s.expert[ei];
    const size_t n = PHASE == 2 ? (size_t)e * (2 * (size_t)p.I) + 8 * (size_t)(unit % cols) + g
                                : (size_t)e * (size_t)p.H + 16 * (size_t)unit + g;
    const uint8_t* w = PHASE == 2 ? p.w1 : p.w2;
    const void* sc = PHASE == 2 ? p.s1 : p.s2;
    return Rows{w + n * wrow, static_cast<const uint8_t*>(sc) + n * srow};
  }
  __device__ __forceinline__ void load_x(uint4 (&x)[4], int ei, int d) const {
    if (PHASE == 2) {
      if (g < p.T) {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = xs[(size_t)(d * 4 + c) * (4 * p.T) + 4 * g + t];
      }
    } else {
      const int r = g < p.T ? s.row[ei][g] : -1;
      const uint4* h = reinterpret_cast<const uint4*>(p.hbuf) + ((size_t)max(r, 0) * nd + d) * 16 + t;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool ok = r >= 0 && d * kDK + chunk_k<FMT>(t, c) < K;
        x[c] = ok ? __ldcg(h + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
};

// Position in the item sequence.
struct Cursor {
  int unit, ei, d;
};
template <int PHASE>
__device__ __forceinline__ Cursor cursor_at(int item, int per, int nd) {
  Cursor c;
  c.unit = item / per;
  const int q = item - c.unit * per;
  c.ei = PHASE == 2 ? 0 : q / nd;
  c.d = PHASE == 2 ? q : q - c.ei * nd;
  return c;
}
// Advances by one item; true if the tile's rows change.
template <int PHASE>
__device__ __forceinline__ bool advance(Cursor& c, int nd, int nhit) {
  if (++c.d < nd) return false;
  c.d = 0;
  if (PHASE == 2) {
    ++c.unit;
  } else if (++c.ei == nhit) {
    c.ei = 0;
    ++c.unit;
  }
  return true;
}

// Streams the CTA's items [a, b): `ready` runs once the first loads are in
// flight (a barrier may hide behind them), `emit(unit, acc, whole)` is called
// by one full warp per unit of the range, whole = all of its items were here.
// Returns false if `ready` did.
template <int FMT, int PHASE, class Ready, class Emit>
__device__ __forceinline__ bool run_stream(const Stream<FMT, PHASE>& st, Tables& s, int a, int b, uint32_t lanesel,
                                           int warp, int lane, Ready ready, Emit emit) {
  const int n = b - a, per = st.per, nd = st.nd, nhit = s.nhit;
  auto split = [&](int w) { return a + (int)((long long)n * w / kWarps); };
  const int lo = split(warp), hi = split(warp + 1);
  Item<FMT> it[kStages];
  Cursor ld = cursor_at<PHASE>(lo, per, nd);
  Rows rows{nullptr, nullptr};
  int next = lo;
  if (lo < hi) rows = st.rows(ld.unit, ld.ei);
  auto fetch = [&](Item<FMT>& dst) {
    if (next < hi) {
      load_item<FMT>(dst, rows, st.w_hi, st.s_hi, ld.d, st.K, st.t);
      ++next;
      if (advance<PHASE>(ld, nd, nhit) && next < hi) rows = st.rows(ld.unit, ld.ei);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) fetch(it[i]);
  if (!ready()) return false;

  Cursor cur = cursor_at<PHASE>(lo, per, nd);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  float one[4] = {0.f, 0.f, 0.f, 0.f};  // phase 3: the current expert's part
  uint4 x[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) x[c] = make_uint4(0u, 0u, 0u, 0u);
  bool tail = false;  // a unit begun by this warp and not finished by it
  for (int i = lo; i < hi; i += kStages) {
#pragma unroll
    for (int j = 0; j < kStages; ++j) {
      const int item = i + j;
      if (item < hi) {
        st.load_x(x, cur.ei, cur.d);
        multiply<FMT>(PHASE == 3 ? one : acc, it[j], x, lanesel);
        fetch(it[j]);
        const int unit = cur.unit, ei = cur.ei;
        const bool turn = advance<PHASE>(cur, nd, nhit);
        if (PHASE == 3 && (turn || item + 1 == hi)) {
          // columns of tokens that did not choose the expert are dropped, not
          // added as zeros: 0 times a NaN or infinite weight is NaN
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[q] += s.row[ei][2 * st.t + (q & 1)] >= 0 ? one[q] : 0.f;
            one[q] = 0.f;
          }
        }
        if (cur.unit != unit || item + 1 == hi) {
          const int first = max(unit * per, a), last = min((unit + 1) * per, b);  // the unit's items in this CTA
          if (lo <= first && last <= hi) {
            emit(unit, acc, last - first == per);
          } else {
            tail = lo <= first;
            *reinterpret_cast<float4*>(&s.part[warp][tail ? 1 : 0][lane][0]) =
                make_float4(acc[0], acc[1], acc[2], acc[3]);
          }
          acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
        }
      }
    }
  }
  __syncthreads();
  if (tail) {  // the unit of this warp's last item: add the parts of the warps after it
    const int unit = (hi - 1) / per;
    const int first = max(unit * per, a), last = min((unit + 1) * per, b);
    float4 v = *reinterpret_cast<const float4*>(&s.part[warp][1][lane][0]);
    for (int w = warp + 1; w < kWarps && split(w) < last; ++w) {
      if (split(w) == split(w + 1)) continue;
      const float4 o = *reinterpret_cast<const float4*>(&s.part[w][0][lane][0]);
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    float sum[4] = {v.x, v.y, v.z, v.w};
    emit(unit, sum, last - first == per);
  }
  return true;
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) moe_decode_kernel(MoeDecodeArgs p, uint32_t table_at, uint32_t smem_end) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t base = smem_u32(smem_raw);
  const uint32_t x_bytes = (uint32_t)((p.H + kDK - 1) / kDK) * 256u * (uint32_t)p.T;
  // guards against a shared window placed otherwise than the host assumed
  if (base + x_bytes > table_at || table_at + (uint32_t)kLut256Bytes + sizeof(Tables) > base + smem_end) {
    if (tid == 0) atomicOr(p.err, GNF4_DEVERR_INTERNAL);
    return;
  }
  uint4* xs = reinterpret_cast<uint4*>(smem_raw);
  Tables& s = *reinterpret_cast<Tables*>(smem_raw + (table_at - base) + (uint32_t)kLut256Bytes);
  build_table<FMT>(reinterpret_cast<uint32_t*>(smem_raw + (table_at - base)), tid);
  const uint32_t lanesel = (uint32_t)lane * 4u | (table_at & 0x00FF0000u);
  {  // x in fragment order, zero past H
    const int nd = (p.H + kDK - 1) / kDK;
    for (int i = tid; i < nd * 16 * p.T; i += kThreads) {
      const int l = i % (4 * p.T), c = (i / (4 * p.T)) & 3, d = i / (16 * p.T);
      const int k = d * kDK + chunk_k<FMT>(l & 3, c);
      xs[i] = k < p.H ? ldg_u128(p.x + (size_t)(l >> 2) * p.H + k) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (tid < kMaxExperts / 32) s.hit[tid] = 0u;
  if (p.router_w != nullptr) {
    router_product(p, s, tid);
    if (!grid_barrier(&p.sync[0], p.err, &s.ok)) return;
  }
  __syncthreads();
  if (warp < p.T) select_topk(p, s, warp, lane);
  __syncthreads();
  list_hits(p, s, tid);

  const float inv_gain = FMT == 0 ? 1.0f / kNf4Gain : 1.0f;
  {  // gate_up + SwiGLU; h times its router weight goes to the workspace in fragment order
    const Stream<FMT, 2> st(p, s, xs, lane);
    const long long units = (long long)s.nhit * st.cols;
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
    const int nd2 = (p.I + kDK - 1) / kDK;
    run_stream<FMT, 2>(
        st, s, u0 * st.per, u1 * st.per, lanesel, warp, lane, [] { return true; },
        [&](int unit, const float(&acc)[4], bool) {
          const int ei = unit / st.cols, col = 8 * (unit % st.cols);
          const int d = col / kDK, q = col % kDK;  // the 8 columns are one chunk
          const int tt = FMT == 0 ? (q & 63) >> 4 : q >> 5;
          const int c = FMT == 0 ? 2 * (q >> 6) + ((q >> 3) & 1) : (q >> 3) & 3;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tok = 2 * t + i;
            const int r = tok < p.T ? s.row[ei][tok] : -1;
            if (r < 0) continue;
            const float v = silu_mul(acc[i] * inv_gain, acc[2 + i] * inv_gain) * s.wt[ei][tok];
            p.hbuf[(((size_t)r * nd2 + d) * 16 + 4 * c + tt) * 8 + g] = __float2bfloat16_rn(v);
          }
        });
  }
  {  // down + combine
    const Stream<FMT, 3> st(p, s, xs, lane);
    const long long items = (long long)(p.H / 16) * st.per;
    const long long G = items < gridDim.x ? items : gridDim.x;
    const bool mine = (long long)blockIdx.x < G;
    const int a = mine ? (int)(items * blockIdx.x / G) : 0, b = mine ? (int)(items * (blockIdx.x + 1) / G) : 0;
    auto store = [&](int unit, const float(&acc)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 2 * t + (i & 1);
        if (tok < p.T) p.out[(size_t)tok * p.H + 16 * unit + g + 8 * (i >> 1)] = __float2bfloat16_rn(acc[i] * inv_gain);
      }
    };
    const bool ok = run_stream<FMT, 3>(
        st, s, a, b, lanesel, warp, lane, [&] { return grid_barrier(&p.sync[1], p.err, &s.ok); },
        [&](int unit, const float(&acc)[4], bool whole) {
          if (whole) {
            store(unit, acc);
            return;
          }
          // the CTAs of the unit's first and last item; all between them hold a part
          const long long q0 = (long long)unit * st.per, q1 = q0 + st.per - 1;
          const int c0 = (int)(((q0 + 1) * G - 1) / items), c1 = (int)(((q1 + 1) * G - 1) / items);
          float4* part = reinterpret_cast<float4*>(p.part);
          part[((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0 ? 1 : 0)) * 32 + lane] =
              make_float4(acc[0], acc[1], acc[2], acc[3]);
          __threadfence();
          __syncwarp();
          int last = 0;
          if (lane == 0) {
            last = atomicAdd(p.unit_count + unit, 1u) == (unsigned)(c1 - c0);
            if (last) p.unit_count[unit] = 0u;
            __threadfence();
          }
          last = __shfl_sync(0xffffffffu, last, 0);
          __syncwarp();
          if (!last) return;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          for (int c = c0; c <= c1; ++c) {
            const float4 v = __ldcg(part + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * 32 + lane);
            sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
          }
          store(unit, sum);
        });
    if (!ok) return;
  }
  // the last CTA to leave zeroes the barrier words
  if (tid == 0) {
    if (atomicAdd(&p.sync[2], 1u) == gridDim.x - 1) {
      p.sync[0] = p.sync[1] = p.sync[2] = 0u;
    }
  }
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t moe_decode_workspace(int T, int k, int H, int I, size_t* count_at, size_t* part_at, size_t* h_at) {
  size_t n = kSyncBytes;
  *count_at = n;
  n = align256(n + (size_t)(H / 16) * sizeof(unsigned));
  *part_at = n;
  n += (size_t)kMaxGrid * 2 * 32 * sizeof(float4);
  *h_at = n;
  return align256(n + (size_t)T * k * ((I + kDK - 1) / kDK) * kDK * 2);
}

template <int FMT>
static cudaError_t launch_t(const MoeDecodeArgs& p, int num_sms, cudaStream_t stream) {
  static std::atomic<bool> configured[64];
  constexpr int kMaxSmem = 227 * 1024;
  cudaError_t e = set_smem_limit_once(moe_decode_kernel<FMT>, kMaxSmem, configured);
  if (e != cudaSuccess) return e;
  const uint32_t x_bytes = (uint32_t)((p.H + kDK - 1) / kDK) * 256u * (uint32_t)p.T;
  const uint32_t table_at = kWindow + x_bytes <= 0x10000u ? 0x10000u : 0x20000u;
  const uint32_t smem = table_at - kWindow + (uint32_t)kLut256Bytes + (uint32_t)sizeof(Tables);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_sms < kMaxGrid ? num_sms : kMaxGrid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the grid barriers need every CTA resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_decode_kernel<FMT>, p, table_at, smem);
}

cudaError_t launch_moe_decode(int fmt, const MoeDecodeArgs& p, int num_sms, cudaStream_t stream) {
  return fmt == 0 ? launch_t<0>(p, num_sms, stream) : launch_t<1>(p, num_sms, stream);
}

}  // namespace gnf4
