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
//   2 gate_up + SwiGLU: work unit = 16 gate rows and the 16 matching up rows
//     of a hit expert, two m16 tiles of 8 + 8, so a lane ends with both halves
//     of a value;
//   3 down + combine: work unit = 32 output rows over ALL hit experts: the
//     router weight is folded into h, so the weighted sum over the experts is
//     the same fp32 accumulator and no per-expert output exists.
// A unit's K (phase 3: hit experts x K) is cut in items of 32 rows x 128 k
// (2 KB of codes); the item sequence of a CTA is divided evenly over its 16
// warps and each warp streams a contiguous range.  A warp that covers a whole
// unit finishes it in registers; split units are added through shared memory
// in warp order.  In phase 3 the item sequence is also divided evenly over the
// CTAs (whole units would leave up to half of the SMs idle); a unit split
// between CTAs is added by the last CTA to finish it, in CTA order, from
// partial sums in the workspace.  Every sum has a fixed order: outputs do not
// depend on timing.
//
// Loads: every warp has its own ring of TMA boxes (one instruction per item)
// and issues them itself; nothing is shared between warps, so the ring needs
// no empty barriers.  Plain loads of the same tiles are bound by the L1: 8
// rows x 64 bytes touch 8 lines per instruction, and what shared memory leaves
// of the L1 (28 KB) caps the bytes in flight (1.8 TB/s at T = 8, H = 7168).
// Scales come by plain loads, one row per lane and four items at a time.
//
// MMA mapping (m16n8k16, fp16 operands, fp32 sums): A = weight codes, B =
// activations.  A lane's codes of one scale block feed two (MXFP4) or four
// (NF4) MMAs whose result is multiplied in fp32 by the activations' unit and the
// scale, so scales are neither rounded nor multiplied into the weights one by
// one, and sums have the range of fp32.  e2m1 is exact in fp16, NF4 codes are
// within 2^-12.  Activations are scaled by the power of two
// that puts the largest of a token's x (of a (token, expert) pair's h) in
// [2^14, 2^15): 8-bit significands of x stay exact down to 2^-28 of it, h is
// rounded to 11 bits.  The largest of h is known when phase 2 ends (an integer
// maximum in the workspace), so phase 2 leaves h in fp32 and phase 3 rounds it.
//   Phase 2: the MMA's 8 columns are the T tokens, whichever expert they
// chose; products of tokens that did not choose it are computed (the MMA has
// the columns anyway) and dropped.  x lies in shared memory in fragment order.
//   Phase 3: columns as in phase 2; h lies in shared memory where there is room,
// else a lane fetches its part for the next item while it works on this one.
//
// Decode: MXFP4 converts a byte to an fp16 pair with one instruction
// (cvt.rn.f16x2.e2m1x2: half a cycle per SM, measured).  NF4 looks a byte up in
// the per-lane pair table of the grouped GEMV (one PRMT and one shared load).
// Rounded to 16 bits apart from that: out, once.
//
// Bound: 16 to 23 us of a call are latency: the meetings of the grid (one behind
// the router product, one behind phase 2, one more where h is too large for
// shared memory), two pipeline starts, the cross-CTA tail.  In the loops MXFP4
// is bound by HBM (5.0-5.4 TB/s; the loads alone 6.6), NF4 by shared memory (122
// cycles per item, of which 64 are lookups: 5.3 TB/s; measured 4.4-5).  Calls:
// OLMoE shape T = 1 25 us, T = 8 60 us; 7168 / 2048, 48 experts, T = 8, MXFP4
// 182 to 190 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
constexpr int kItemBytes = 32 * kDK / 2;           // one TMA box
constexpr int kMaxStages = 2;                      // items in flight per warp (4: 5.1 instead of 6.6 TB/s, loads alone)
constexpr uint32_t kMaxWindow = 227 * 1024;        // dynamic shared memory of a CTA

struct Route {
  short row[kMaxPairs][kMaxT];  // pair = row of h of (hit expert, token); ~(a pair of the expert) if not routed
  short expert[kMaxPairs];      // hit expert ids, ascending
  uint32_t hit[kMaxExperts / 32];   // bit per expert
  uint32_t tokens[kMaxExperts / 4]; // byte per expert: the tokens that chose it
  short sel_id[kMaxPairs];      // by pair
  float sel_p[kMaxPairs];
};
struct Work {
  uint64_t full[kWarps][kMaxStages];
  float red[kWarps][kMaxT];     // router products per warp
  uint32_t xmax[kMaxT];         // largest finite |x| of a token (fp32 bits)
  float hscale[kMaxPairs];      // scale of a pair's fp16 h
  int nhit;
  int ok;
  int abort;
};
// fp32 bits of the largest |v| -> the scale 2^(14 - e), e at least 15 - 127; and the inverse of a power of two.
__device__ __forceinline__ float scale_up(uint32_t top) { return __uint_as_float((268u - max(top >> 23, 15u)) << 23); }
__device__ __forceinline__ float inverse_of(float pow2) { return __uint_as_float(0x7F000000u - __float_as_uint(pow2)); }

// Offsets in the dynamic shared window.  x in fragment order (in phase 3: h,
// where there is room), Route, Work and MXFP4's scale scratch first; NF4's pair table at a 64 KB boundary (0x10000, or
// 0x20000 where x needs the room); then the rings.
struct Plan {
  uint32_t route, work, scratch, table, ring, total;
  uint32_t act;  // bytes for activations at the start
  int stages;
};

constexpr uint32_t kWindow = 0x400;  // start of the dynamic shared window that the host's layout assumes
// A warp's scratch: the fp32 scales of four items.  MXFP4 [4][32 rows][4], 2 KB of its own; NF4 [4][32][2] in the
// unused upper halves of eight entries of the pair table, 16 rows to an entry.
constexpr int kScratchStride = 2048, kScratchItem = 512;  // per warp, per item
template <int FMT>
__device__ __forceinline__ constexpr int scratch_row(int r) {
  return FMT == 0 ? (r >> 4) * 256 + (r & 15) * 8 : 16 * r;
}
// Workspace words: [0] parity of the call, [1 + b + 3 * parity] arrivals at grid barrier b.  A call uses the counters
// (and the hmax) of its parity and zeroes the other ones, which the call before it used; no CTA has to wait for the
// others to leave.
constexpr int kSyncBytes = 256;
constexpr int kHmaxStep = 32;  // words: a line for every pair's maximum, so that the warps' updates do not queue (6 us at T = 8)

// NF4 pairs as fp16, one copy per lane, 256 bytes per entry.
__device__ __forceinline__ void build_table(uint32_t* lut, int tid) {
  for (int i = tid; i < 256 * 8; i += kThreads) {
    const uint32_t b = (uint32_t)i >> 3;
    __half2 h = __floats2half2_rn(kNf4Code[b >> 4], kNf4Code[b & 15u]);
    const uint32_t v = *reinterpret_cast<uint32_t*>(&h);
    *reinterpret_cast<uint4*>(lut + b * 64u + 4u * ((uint32_t)i & 7u)) = make_uint4(v, v, v, v);
  }
}

// D (16x8 fp32) = A (16x16 f16, row) x B (16x8 f16, col), or += in the second form.
__device__ __forceinline__ void mma_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte j of `word` selects the entry; `lanesel` holds 4*lane in byte 0 and the table's 64 KB base in byte 2.
__device__ __forceinline__ uint32_t lookup(uint32_t word, uint32_t lanesel, uint32_t j) {
  uint32_t v;
  asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(prmt_b32(word, lanesel, 0x7604u | (j << 4))));
  return v;
}

// Eight e2m1 codes to four fp16 pairs (k0,k1) .. (k6,k7), exactly.
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&p)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
      : "r"(w));
}
// Fragment order of activations: chunk c (0..3) of lane column t holds 8
// consecutive k of a 128-k item, starting at chunk_k; chunk_of is the inverse.
template <int FMT>
__device__ __forceinline__ int chunk_k(int t, int c) {
  return FMT == 0 ? 64 * (c >> 1) + 16 * t + 8 * (c & 1) : 32 * c + 8 * t;
}
template <int FMT>  // k inside the item, a multiple of 8 -> 4 * c + t
__device__ __forceinline__ int chunk_of(int k) {
  return FMT == 0 ? 4 * (2 * (k >> 6) + ((k >> 3) & 1)) + ((k & 63) >> 4) : 4 * (k >> 5) + ((k >> 3) & 3);
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ unsigned atom_add_acq_rel(unsigned* p, unsigned v) {
  unsigned o;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(o) : "l"(p), "r"(v) : "memory");
  return o;
}

// All CTAs of the grid meet (cooperative launch: they are all resident).  The
// release is cumulative over the block barrier before it, the acquire over the
// one after it (a full fence on either side cost 1 to 4 us).
__device__ __forceinline__ void grid_arrive(unsigned* ctr) {
  __syncthreads();
  if (threadIdx.x == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(ctr) : "memory");
}
// Bounded: false after the wait limit, with the timeout flagged.
__device__ __forceinline__ bool grid_wait(unsigned* ctr, unsigned* err, int* ok) {
  if (threadIdx.x == 0) {
    const long long t0 = clock64();
    int good = 1;
    while (true) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
      if (v >= gridDim.x) break;
      __nanosleep(40);  // 148 pollers on one line delay the arrivals (4% of a T = 8 call)
      if (clock64() - t0 > kSpinLimitCycles) {
        atomicOr(err, GNF4_DEVERR_TIMEOUT);
        good = 0;
        break;
      }
    }
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

// The CTA's experts are blockIdx + i * grid, each the work of `wpe` warps (E <= 1024: at most 7 a CTA).
struct RouterPart {
  int wpe, e, first;
  uint4 w;  // this thread's first chunk, loaded early
  __device__ __forceinline__ RouterPart(const MoeDecodeArgs& p, int tid) {
    const int per_cta = (p.E + (int)gridDim.x - 1) / (int)gridDim.x, warp = tid >> 5;
    wpe = per_cta <= 1 ? 16 : per_cta <= 2 ? 8 : per_cta <= 4 ? 4 : 2;
    e = blockIdx.x + (warp / wpe) * (int)gridDim.x;
    first = (warp % wpe) * 32 + (tid & 31);
    w = make_uint4(0u, 0u, 0u, 0u);
    if (p.router_w != nullptr && e < p.E && first < p.H / 8)
      w = ldg_nc_u128(reinterpret_cast<const uint4*>(p.router_w) + (size_t)e * (p.H / 8) + first);
  }
};

// logits of the CTA's experts (TP >= T tokens).
template <int TP>
__device__ __forceinline__ void router_product(const MoeDecodeArgs& p, Work& s, const RouterPart& part, int tid) {
  const int warp = tid >> 5, lane = tid & 31, H8 = p.H / 8, wpe = part.wpe, e = part.e;
  const uint4* x = reinterpret_cast<const uint4*>(p.x);
  float acc[TP];
#pragma unroll
  for (int t = 0; t < TP; ++t) acc[t] = 0.f;
  if (e < p.E) {
    const uint4* w = reinterpret_cast<const uint4*>(p.router_w) + (size_t)e * H8;
#pragma unroll 1
    for (int i = part.first; i < H8; i += wpe * 32) {
      const uint4 wv = i == part.first ? part.w : ldg_nc_u128(w + i);
      uint4 xv[TP];
#pragma unroll
      for (int t = 0; t < TP; ++t) xv[t] = __ldg(x + (size_t)min(t, p.T - 1) * H8 + i);
#pragma unroll
      for (int t = 0; t < TP; ++t) acc[t] = dot8(wv, xv[t], acc[t]);
    }
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1)
#pragma unroll
    for (int t = 0; t < TP; ++t) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], d);
  if (lane == 0)
#pragma unroll
    for (int t = 0; t < TP; ++t) s.red[warp][t] = acc[t];
  __syncthreads();
  if (e < p.E && warp % wpe == 0 && lane < p.T) {
    float v = 0.f;
    for (int i = 0; i < wpe; ++i) v += s.red[warp + i][lane];
    p.logits[(size_t)lane * p.E + e] = v;
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
// lower expert, NaN last) and the softmax of their raw logits, as the router
// epilogue of the routing call.  A lane holds the keys of N experts.
template <int N>
__device__ __forceinline__ void select_topk(const MoeDecodeArgs& p, Route& s, int t, int lane,
                                            float* logit) {
  const float* logits = p.logits + (size_t)t * p.E;
  uint32_t key[N];
  float raw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * 32 + lane;
    raw[i] = e < p.E ? __ldcg(logits + e) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < p.E ? score_key(p.bias != nullptr ? raw[i] + __ldg(p.bias + e) : raw[i]) : 0u;
  }
  int mine = 0;
  float l = -INFINITY;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = key[0];
    float value = raw[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (key[i] > best) {
        best = key[i];
        value = raw[i];
        at = i;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t who = __ballot_sync(0xffffffffu, best == top);
    int owner = __ffs((int)who) - 1;
    if (who & (who - 1u))  // equal scores: the lowest expert
      owner = (int)(__reduce_min_sync(0xffffffffu, best == top ? (unsigned)(at * 32 + lane) : 0xFFFFFFFFu) & 31u);
    const float v = __shfl_sync(0xffffffffu, value, owner);
    const int row = __shfl_sync(0xffffffffu, at, owner);
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = owner == lane && i == at ? 0u : key[i];
    if (lane == j) {
      mine = row * 32 + owner;
      l = v;
    }
  }
  if (lane < p.k) {
    s.sel_id[t * p.k + lane] = (short)mine;
    atomicOr(&s.hit[mine >> 5], 1u << (mine & 31));
    atomicOr(&s.tokens[mine >> 2], 1u << (8 * (mine & 3) + t));
    if (blockIdx.x == 0) p.topk_ids[t * p.k + lane] = mine;
  }
  *logit = l;
}

// The weights of the selected logits: the other half of select_topk, off the path to the first loads.
__device__ __forceinline__ void weigh_topk(const MoeDecodeArgs& p, Route& s, int t, int lane, float l) {
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
    s.sel_p[t * p.k + lane] = ex / sum;
    if (blockIdx.x == 0) p.topk_weights[t * p.k + lane] = ex / sum;
  }
}

// Hit experts in ascending order, and the pair of every (hit expert, token).  All threads; a barrier before and after.
__device__ __forceinline__ void list_hits(const MoeDecodeArgs& p, Route& s, int* nhit, int tid) {
  if (tid >= kThreads - 32) {
    const int n = __reduce_add_sync(0xffffffffu, (unsigned)__popc(s.hit[tid & 31]));
    if (tid == kThreads - 32) *nhit = n;
  }
  if (tid < p.T * p.k) {  // pairs <= 256
    const int e = s.sel_id[tid], tok = tid / p.k;
    int r = __popc(s.hit[e >> 5] & ((1u << (e & 31)) - 1u));  // rank: set bits below e
    for (int i = 0; i < (e >> 5); ++i) r += __popc(s.hit[i]);
    const uint32_t toks = (s.tokens[e >> 2] >> (8 * (e & 3))) & 255u;
    s.row[r][tok] = (short)tid;
    if (tok == __ffs((int)toks) - 1) {  // the expert's first token fills in for those that did not choose it
      s.expert[r] = (short)e;
#pragma unroll
      for (int t = 0; t < kMaxT; ++t)
        if (!((toks >> t) & 1u)) s.row[r][t] = (short)~tid;
    }
  }
}

// ---------------------------------------------------------------- item stream

__device__ __forceinline__ uint2 lds_u64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Scales of four consecutive items (512 k) of one row, as loaded: the 16-byte
// blocks that hold them.  Rows are K/32 bytes (MXFP4) or K/16 (NF4) apart and
// aligned to nothing, 4 bytes.  One row per lane: every load touches 32 lines,
// so they are as wide as they can be (4-byte loads kept the L1 busy for 160
// cycles per item).
template <int FMT>
struct ScaleGroup {
  uint4 q[FMT == 0 ? 3 : 2];
  uint32_t off;  // the first scale's byte in q
};

// The 16-byte block at b, whose bytes outside [lo, hi) are not read: 0.
__device__ __noinline__ uint4 load_edge(uintptr_t b, uintptr_t lo, uintptr_t hi) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  for (int i = 0; i < 16; ++i)
    if (b + i >= lo && b + i < hi) w[i >> 2] |= (uint32_t)__ldg(reinterpret_cast<const uint8_t*>(b + i)) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// row: the row's first scale; bytes: of the row; group: 512-k group; [lo, hi): the array.  Blocks without a byte of
// the group are not read.  EDGES: an array that begins at no 16-byte boundary shares its first and its last block
// with other memory; blocks that stick out are read byte by byte.
template <int FMT, bool EDGES>
__device__ __forceinline__ void load_scales(ScaleGroup<FMT>& s, const uint8_t* row, int bytes, int group,
                                            const void* lo, const void* hi) {
  constexpr int kBytes = FMT == 0 ? 32 : 16, kBlocks = FMT == 0 ? 3 : 2;
  const uintptr_t a = reinterpret_cast<uintptr_t>(row) + (size_t)group * kBytes;
  const uintptr_t down = a & ~(uintptr_t)15, first = reinterpret_cast<uintptr_t>(lo), end = reinterpret_cast<uintptr_t>(hi);
  s.off = (uint32_t)(a & 15);
  const int need = (int)s.off + min(bytes - group * kBytes, kBytes);
  if (!EDGES || (down >= first && down + ((need + 15) & ~15) <= end)) {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
      s.q[i] = 16 * i < need ? ldg_u128(reinterpret_cast<const void*>(down + 16 * i)) : make_uint4(0u, 0u, 0u, 0u);
  } else {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i)
      s.q[i] = 16 * i < need ? load_edge(down + 16 * i, first, end) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// The group as fp32 in the warp's scratch (this lane's row).  left: scales from the group on (a scale past K is
// written as 0 or 2^-127: its codes and activations are zero).
template <int FMT>
__device__ __forceinline__ void scales_to_scratch(const ScaleGroup<FMT>& s, int left, uint32_t scratch, int lane) {
  constexpr int kWords = FMT == 0 ? 8 : 5;
  uint32_t in[FMT == 0 ? 12 : 8], w[kWords];
#pragma unroll
  for (int i = 0; i < (FMT == 0 ? 3 : 2); ++i)
    in[4 * i] = s.q[i].x, in[4 * i + 1] = s.q[i].y, in[4 * i + 2] = s.q[i].z, in[4 * i + 3] = s.q[i].w;
  const uint32_t o = s.off >> 2;
  const bool shifted = __any_sync(0xffffffffu, s.off != 0u);
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    w[i] = in[i];
    if (shifted) w[i] = o == 0u ? in[i] : o == 1u ? in[i + 1] : o == 2u ? in[i + 2] : in[i + 3];
  }
  if (FMT == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(scratch + kScratchItem * j + scratch_row<FMT>(lane)),
                   "r"(2 * j < left ? w[2 * j] : 0u), "r"(2 * j + 1 < left ? w[(2 * j + 1) % kWords] : 0u)
                   : "memory");
  } else {
    uint32_t v[4], nan = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = shifted ? __funnelshift_r(w[j % kWords], w[(j + 1) % kWords], 8u * (s.off & 3u)) : w[j % kWords];
      nan |= (~v[j] - 0x01010101u) & v[j];
    }
    if (left < 16)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] &= left <= 4 * j ? 0u : left >= 4 * j + 4 ? 0xFFFFFFFFu : (1u << (8 * (left - 4 * j))) - 1u;
    const bool any_nan = (nan & 0x80808080u) != 0u;  // a byte may be 255
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // 2^(e - 127): the exponent field, the subnormal 2^-127 for 0, NaN for 255
      uint32_t f[4] = {(v[j] << 23) & 0x7F800000u, (v[j] << 15) & 0x7F800000u, (v[j] << 7) & 0x7F800000u,
                       (v[j] >> 1) & 0x7F800000u};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = max(f[i], 0x00400000u);
      if (any_nan)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (f[i] == 0x7F800000u) f[i] = 0x7FC00000u;
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(scratch + kScratchItem * j + scratch_row<FMT>(lane)),
                   "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3])
                   : "memory");
    }
  }
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// acc += scale of the row * d, d brought back to true units (of its column) first: a sum in units of the scaled
// activations overflows 2^(14 - e) times before the true sum does.  Two values per instruction: 48 experts of 7168 /
// 2048, T = 8, MXFP4: 187 us, one by one 190, without the step 183.
__device__ __forceinline__ void add_scaled(float (&acc)[4], const float (&d)[4], float sa, float sb,
                                           const float (&unit)[2]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const float sc = i < 2 ? sa : sb;
    asm("{\n\t.reg .b64 d, u, a, s;\n\t"
        "mov.b64 d, {%2, %3};\n\tmov.b64 u, {%4, %5};\n\tmov.b64 s, {%6, %6};\n\tmov.b64 a, {%0, %1};\n\t"
        "mul.rn.f32x2 d, d, u;\n\tfma.rn.f32x2 a, d, s, a;\n\tmov.b64 {%0, %1}, a;\n\t}\n"
        : "+f"(acc[i]), "+f"(acc[i + 1])
        : "f"(d[i]), "f"(d[i + 1]), "f"(unit[0]), "f"(unit[1]), "f"(sc));
  }
}

// acc[tile] += the item's weights (shared memory) times the lane's activations: chunk c at x + c * x_step in shared
// memory (HERE), else own[c].
// Tile k holds item rows r0 + 8 STEP_T k (its first 8) and 8 STEP_H further.
template <int FMT, bool HERE, int STEP_T, int STEP_H>
__device__ __forceinline__ void multiply(float (&acc)[2][4], uint32_t item, uint32_t scratch, uint32_t x,
                                         uint32_t x_step, const uint4 (&own)[4], const float (&unit)[2], int r0, int t,
                                         uint32_t lanesel) {
  uint4 v[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) v[b] = HERE ? lds_u128(x + b * x_step) : own[b];
  const uint32_t key = (uint32_t)(r0 >> 1) & 3u;  // the box's 64-byte swizzle: 16-byte chunk ^= (row / 2) % 4
  if (FMT == 1) {
    const uint32_t at = item + 64 * r0 + 4 * t + (key << 4);
    scratch += 16 * r0;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const int ra = 8 * STEP_T * tile, rb = ra + 8 * STEP_H;
      const uint4 qa = lds_u128(scratch + scratch_row<FMT>(ra)), qb = lds_u128(scratch + scratch_row<FMT>(rb));
      const float sa[4] = {__uint_as_float(qa.x), __uint_as_float(qa.y), __uint_as_float(qa.z), __uint_as_float(qa.w)};
      const float sb[4] = {__uint_as_float(qb.x), __uint_as_float(qb.y), __uint_as_float(qb.z), __uint_as_float(qb.w)};
#pragma unroll
      for (int b = 0; b < 4; ++b) {  // one 32-block: this lane's 8 codes of each row
        const uint32_t q = at ^ ((uint32_t)b << 4);
        uint32_t lo[4], hi[4];
        e2m1_to_f16(lds_u32(q + 64 * ra), lo);
        e2m1_to_f16(lds_u32(q + 64 * rb), hi);
        float d[4];
        mma_new(d, lo[0], hi[0], lo[1], hi[1], v[b].x, v[b].y);
        mma_add(d, lo[2], hi[2], lo[3], hi[3], v[b].z, v[b].w);
        add_scaled(acc[tile], d, sa[b], sb[b], unit);
      }
    }
  } else {
    const uint32_t at = item + 64 * r0 + 8 * (t & 1);
    scratch += 8 * r0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {  // one 64-block: 16 codes of each row
      const uint32_t q = at + (((uint32_t)(2 * b + (t >> 1)) ^ key) << 4);
      const uint4 v0 = v[2 * b], v1 = v[2 * b + 1];
#pragma unroll
      for (int tile = 0; tile < 2; ++tile) {
        const int ra = 8 * STEP_T * tile, rb = ra + 8 * STEP_H;
        const uint2 va = lds_u64(q + 64 * ra), vb = lds_u64(q + 64 * rb);
        const float sa = lds_f32(scratch + scratch_row<FMT>(ra) + 4 * b), sb = lds_f32(scratch + scratch_row<FMT>(rb) + 4 * b);
        float d[4];
        mma_new(d, lookup(va.x, lanesel, 0), lookup(vb.x, lanesel, 0), lookup(va.x, lanesel, 1),
                lookup(vb.x, lanesel, 1), v0.x, v0.y);
        mma_add(d, lookup(va.x, lanesel, 2), lookup(vb.x, lanesel, 2), lookup(va.x, lanesel, 3),
                lookup(vb.x, lanesel, 3), v0.z, v0.w);
        mma_add(d, lookup(va.y, lanesel, 0), lookup(vb.y, lanesel, 0), lookup(va.y, lanesel, 1),
                lookup(vb.y, lanesel, 1), v1.x, v1.y);
        mma_add(d, lookup(va.y, lanesel, 2), lookup(vb.y, lanesel, 2), lookup(va.y, lanesel, 3),
                lookup(vb.y, lanesel, 3), v1.z, v1.w);
        add_scaled(acc[tile], d, sa, sb, unit);
      }
    }
  }
}

// `total` things divided evenly over `parts`: part c holds [begin(c), begin(c + 1)).
struct Share {
  int base, extra;  // the first `extra` parts hold one more
  __device__ __forceinline__ Share(int total, unsigned parts) : base(total / (int)parts), extra(total % (int)parts) {}
  __device__ __forceinline__ int begin(int c) const { return c * base + min(c, extra); }
  __device__ __forceinline__ int owner(int i) const {
    const int big = extra * (base + 1);
    return i < big ? i / (base + 1) : extra + (i - big) / base;
  }
};

// Position in the item sequence.
struct Cursor {
  int unit, ei, d;
};

// One phase's view of its item sequence: unit u = items [u * per, (u + 1) * per).
template <int FMT, int PHASE>
struct Stream {
  const MoeDecodeArgs& p;
  const Route& s;
  const Work& wk;
  const CUtensorMap* map;
  int g, t, lane, nd, per, cols, nhit;  // nd: items of one expert; cols: units of an expert (phase 2)
  int ns, srow;                         // scales and scale bytes of a row

  __device__ __forceinline__ Stream(const MoeDecodeArgs& p_, const Route& s_, const Work& wk_, const CUtensorMap* map_,
                                    int lane_)
      : p(p_), s(s_), wk(wk_), map(map_), g(lane_ >> 2), t(lane_ & 3), lane(lane_), nhit(wk_.nhit) {
    const int K = PHASE == 2 ? p.H : p.I;
    nd = (K + kDK - 1) / kDK;
    cols = p.I / 16;
    per = PHASE == 2 ? nd : nd * nhit;
    ns = FMT == 0 ? K / 64 : K / 32;
    srow = ns * (FMT == 0 ? 4 : 1);
  }
  __device__ __forceinline__ Cursor at(int item) const {
    Cursor c;
    c.unit = item / per;
    const int q = item - c.unit * per;
    c.ei = PHASE == 2 ? c.unit / cols : q / nd;
    c.d = PHASE == 2 ? q : q - c.ei * nd;
    return c;
  }
  // Advances by one item; true if the tile's rows change.
  __device__ __forceinline__ bool advance(Cursor& c) const {
    if (++c.d < nd) return false;
    c.d = 0;
    if (PHASE == 2) {
      c.ei = ++c.unit / cols;
    } else if (++c.ei == nhit) {
      c.ei = 0;
      ++c.unit;
    }
    return true;
  }
  // One box: phase 2: 16 gate rows, then the 16 up rows; phase 3: 32 rows.
  __device__ __forceinline__ void load_box(void* dst, uint64_t* bar, const Cursor& c) const {
    mbar_arrive_expect_tx(bar, kItemBytes);
    const int e = s.expert[c.ei];
    if (PHASE == 2)
      tma_load_4d(dst, map, bar, (kDK / 2) * c.d, 16 * (c.unit - c.ei * cols), 0, e);
    else
      tma_load_3d(dst, map, bar, (kDK / 2) * c.d, 32 * c.unit, e);
  }
  __device__ __forceinline__ const void* scales() const { return PHASE == 2 ? p.s1 : p.s2; }
  __device__ __forceinline__ const void* scales_end() const { return PHASE == 2 ? p.s1_end : p.s2_end; }
  // First scale of item row `lane`.
  __device__ __forceinline__ const uint8_t* scale_row(const Cursor& c) const {
    const size_t e = (size_t)s.expert[c.ei];
    const size_t n = PHASE == 2 ? e * (2 * (size_t)p.I) + 16 * (size_t)(c.unit - c.ei * cols) + (lane & 15) +
                                      (lane < 16 ? 0 : (size_t)p.I)
                                : e * (size_t)p.H + 32 * (size_t)c.unit + lane;
    return static_cast<const uint8_t*>(scales()) + n * (size_t)srow;
  }
  // Phase 3: the pair whose h this lane multiplies (a column without the token takes another: its sums are dropped).
  __device__ __forceinline__ int pair(int ei) const {
    const int r = s.row[ei][g];
    return r < 0 ? ~r : r;
  }
  // Phase 3 with h in global memory: this lane's fp16 h of an item.
  __device__ __forceinline__ void load_h(uint4 (&h)[4], const Cursor& c) const {
    const uint4* q = p.h16 + ((size_t)pair(c.ei) * nd + c.d) * 16 + t;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __ldcg(q + 4 * i);
  }
  // 1 / the scale of column q (0, 1) of this lane; 0 for a phase 3 column whose token did not choose expert ei.
  __device__ __forceinline__ float unit_of(int ei, int q) const {
    const int col = 2 * t + q;
    if (PHASE == 2) return inverse_of(scale_up(wk.xmax[col]));
    const int r = s.row[ei][col];
    return r < 0 ? 0.f : inverse_of(wk.hscale[r]);
  }
};

// A warp's ring of boxes: slot and phase of the next box to issue and to read.
struct Ring {
  uint32_t base;   // shared address
  uint8_t* ptr;
  uint64_t* full;
  int stages;
  int put, get;
  uint32_t parity;
  __device__ __forceinline__ void pushed() { put = put + 1 == stages ? 0 : put + 1; }
  __device__ __forceinline__ void popped() {
    if (++get == stages) {
      get = 0;
      parity ^= 1u;
    }
  }
};

// The second look at a box, by the whole warp: kept out of the loop.  False, in all lanes, if it gives up: *abort is
// set then.
__device__ __noinline__ bool box_wait_slow(uint64_t* bar, uint32_t parity, unsigned* err, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, abort)) != 0;
}

// The `n` boxes that the warp has issued and not read land (or a bounded wait each runs out).
__device__ __noinline__ void drain_boxes(uint64_t* full, int stages, int get, uint32_t parity, int n) {
  for (int i = 0; i < n; ++i) {
    mbar_drain(full + get, parity);
    if (++get == stages) {
      get = 0;
      parity ^= 1u;
    }
  }
}

// A warp's way through its items [lo, hi) of the CTA's [a, b).
template <int FMT>
struct Walk {
  int a, b, lo, hi;
  int next;         // next item to issue
  Cursor cur, ld;   // next item to multiply, next item to issue
  const uint8_t* row;   // this lane's scales of the rows at cur (of the group loaded last)
  ScaleGroup<FMT> sc;   // the scale group after the one in the scratch
};

template <int FMT, int PHASE>
__device__ __forceinline__ void issue_box(const Stream<FMT, PHASE>& st, Ring& ring, Walk<FMT>& w) {
  if (w.next < w.hi) {
    if (st.lane == 0) st.load_box(ring.ptr + ring.put * kItemBytes, ring.full + ring.put, w.ld);
    ring.pushed();
    ++w.next;
    st.advance(w.ld);
  }
}

// The first boxes and scales on their way.
template <int FMT, int PHASE, bool EDGES>
__device__ __forceinline__ void start_stream(const Stream<FMT, PHASE>& st, Ring& ring, Walk<FMT>& w, int a, int b,
                                             int warp) {
  const int n = b - a;
  w.a = a, w.b = b;
  w.lo = a + n * warp / kWarps;
  w.hi = a + n * (warp + 1) / kWarps;
  w.next = w.lo;
  w.cur = w.ld = st.at(w.lo);
  // earlier generic accesses to the ring (partial sums) before the boxes
  fence_proxy_async_smem();
  __syncwarp();
  for (int i = 0; i < ring.stages; ++i) issue_box(st, ring, w);
  if (w.lo < w.hi) {
    w.row = st.scale_row(w.cur);
    load_scales<FMT, EDGES>(w.sc, w.row, st.srow, w.cur.d >> 2, st.scales(), st.scales_end());
  }
}

// The loaded scale group (the one of item `item` at cur) to the scratch, and the one after it on its way.
template <int FMT, int PHASE, bool EDGES>
__device__ __forceinline__ void next_scales(const Stream<FMT, PHASE>& st, Walk<FMT>& w, int item, uint32_t scratch) {
  const int group = w.cur.d >> 2;
  scales_to_scratch<FMT>(w.sc, st.ns - group * (FMT == 0 ? 8 : 16), scratch, st.lane);
  const int skip = min(4 - (w.cur.d & 3), st.nd - w.cur.d);
  if (item + skip >= w.hi) return;  // no other group belongs to this warp
  if (w.cur.d + skip < st.nd) {
    load_scales<FMT, EDGES>(w.sc, w.row, st.srow, group + 1, st.scales(), st.scales_end());
  } else {
    Cursor q = w.cur;
    q.d = st.nd - 1;
    st.advance(q);
    w.row = st.scale_row(q);
    load_scales<FMT, EDGES>(w.sc, w.row, st.srow, 0, st.scales(), st.scales_end());
  }
}

// Multiplies the warp's items.  The first scale group lies in the scratch;
// phase 3: h holds the first item's activations.  `emit(unit, acc, whole)` is
// called by one full warp per unit of the CTA's range, whole = all of its items
// were here.  x: phase 2 this lane's x in shared memory (items 4 * x_step
// apart); phase 3 this lane's column of h in shared memory (HERE), else h holds
// the first item's.  A wait that gives up flags the timeout and sets
// wk.abort, which ends every warp's items at its next wait: a slot whose box
// may be in flight is neither read nor issued again.  Returns false then, in
// all threads, with no box of the CTA in flight.
template <int FMT, int PHASE, bool EDGES, bool HERE, class Emit>
__device__ __forceinline__ bool run_stream(const Stream<FMT, PHASE>& st, Ring& ring, Walk<FMT>& w, Work& wk,
                                           unsigned* err, uint32_t scratch, uint32_t x, uint32_t x_step,
                                           uint32_t lanesel, uint8_t* rings, int warp, uint4 (&h)[4], Emit emit) {
  const int a = w.a, b = w.b, lo = w.lo, hi = w.hi, per = st.per, lane = st.lane;
  auto split = [&](int i) { return a + (b - a) * i / kWarps; };
  // NF4 reads 8 bytes per lane: this order of the 8 rows keeps each half of the warp on 32 banks
  const int r0 = FMT == 0 ? (st.g & 1) | ((st.g & 2) << 1) | ((st.g & 4) >> 1) : st.g;
  uint4 own[4] = {};  // !HERE: the present item's activations; h: the next one's
  uint32_t column = x;  // phase 3, HERE: the current expert's row of h
  if (PHASE == 3 && HERE && lo < hi) column = x + 256u * (uint32_t)(st.pair(w.cur.ei) * st.nd);
  float acc[2][4] = {};
  float one[2][4] = {};   // phase 3: the current expert's part
  float head[2][4] = {};  // a unit begun by an earlier warp
  float unit2[2] = {0.f, 0.f};  // of the lane's two columns; phase 3: for the current expert
  if (lo < hi) unit2[0] = st.unit_of(w.cur.ei, 0), unit2[1] = st.unit_of(w.cur.ei, 1);
  bool tail = false;  // a unit begun by this warp and not finished by it
  for (int item = lo; item < hi; ++item) {
    const int unit = w.cur.unit, d = w.cur.d;
    if ((d & 3) == 0 && item > lo) next_scales<FMT, PHASE, EDGES>(st, w, item, scratch);
    const bool turn = st.advance(w.cur), more = item + 1 < hi;
    if (!HERE) {
#pragma unroll
      for (int i = 0; i < 4; ++i) own[i] = h[i];
      if (more) st.load_h(h, w.cur);
    }
    if (!__all_sync(0xffffffffu, mbar_try_wait(ring.full + ring.get, ring.parity)) &&
        !box_wait_slow(ring.full + ring.get, ring.parity, err, &wk.abort)) {
      drain_boxes(ring.full, ring.stages, ring.get, ring.parity, w.next - item);
      break;
    }
    __syncwarp();
    multiply<FMT, HERE, PHASE == 2 ? 1 : 2, PHASE == 2 ? 2 : 1>(
        PHASE == 3 ? one : acc, ring.base + ring.get * kItemBytes, scratch + (d & 3) * kScratchItem,
        column + 4 * x_step * d, x_step, own, unit2, r0, st.t, lanesel);
    ring.popped();
    __syncwarp();  // every lane has read the box and the scratch
    issue_box(st, ring, w);
    if (!turn && more) continue;
    if (PHASE == 3) {
      // columns of tokens that did not choose the expert are dropped, not
      // added as zeros: 0 times a NaN or infinite weight is NaN
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool chosen = unit2[q] != 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          acc[k][q] += chosen ? one[k][q] : 0.f;
          acc[k][q + 2] += chosen ? one[k][q + 2] : 0.f;
          one[k][q] = one[k][q + 2] = 0.f;
        }
        if (more) unit2[q] = st.unit_of(w.cur.ei, q);
      }
      if (HERE) column = x + 256u * (uint32_t)(st.pair(w.cur.ei) * st.nd);
    }
    if (more && w.cur.unit == unit) continue;
    const int first = max(unit * per, a), last = min((unit + 1) * per, b);  // the unit's items in this CTA
    if (lo <= first && last <= hi) {
      emit(unit, acc, last - first == per, r0);
    } else if (lo <= first) {
      tail = true;  // stays in acc: this was the last item
      break;
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) head[k][i] = acc[k][i];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
  }
  // the ring is idle: its first KB takes the head part
  auto part = [&](int i) { return reinterpret_cast<float4*>(rings + (size_t)i * ring.stages * kItemBytes) + lane; };
#pragma unroll
  for (int k = 0; k < 2; ++k) part(warp)[32 * k] = make_float4(head[k][0], head[k][1], head[k][2], head[k][3]);
  __syncthreads();
  if (wk.abort) return false;
  if (tail) {  // add the parts of the warps after this one
    const int unit = (hi - 1) / per;
    const int first = max(unit * per, a), last = min((unit + 1) * per, b);
    // a warp without items has an empty head part: the sum runs over four warps' parts at a time
#pragma unroll 1
    for (int i = warp + 1; i < kWarps && split(i) < last; i += 4) {
      float4 v[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) v[j][k] = part(min(i + j, kWarps - 1))[32 * k];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + j >= kWarps || split(i + j) >= last) break;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          acc[k][0] += v[j][k].x, acc[k][1] += v[j][k].y, acc[k][2] += v[j][k].z, acc[k][3] += v[j][k].w;
        }
      }
    }
    emit(unit, acc, last - first == per, r0);
  }
  return true;
}

// x as fp16 scaled per token, in fragment order, zero past H.  All threads;
// a token belongs to 16 / TP warps (TP: T up to a power of two).
template <int FMT>
__device__ __forceinline__ void stage_x(const MoeDecodeArgs& p, Work& s, uint4* xs, int tid) {
  const int nd = (p.H + kDK - 1) / kDK, H8 = p.H / 8;
  const int wpt = p.T == 1 ? 16 : p.T == 2 ? 8 : p.T <= 4 ? 4 : 2;
  const int tok = (tid >> 5) / wpt, first = ((tid >> 5) % wpt) * 32 + (tid & 31), step = wpt * 32;
  const uint4* x = reinterpret_cast<const uint4*>(p.x) + (size_t)tok * H8;
  if (tok < p.T) {
    uint32_t m = 0;
#pragma unroll 4
    for (int i = first; i < H8; i += step) {
      const uint4 v = __ldg(x + i);
      const uint32_t q = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
      if (__vcmpgeu2(q, 0x7F807F80u) != 0u) {  // an infinity or a NaN stays out
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t a = (w[j >> 1] >> (16 * (j & 1))) & 0x7FFFu;
          m = max(m, a >= 0x7F80u ? 0u : a);
        }
      } else {
        m = max(m, max(q & 0xFFFFu, q >> 16));
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) atomicMax(&s.xmax[tok], m << 16);
  }
  __syncthreads();
  if (tok >= p.T) return;
  const float sc = scale_up(s.xmax[tok]);
#pragma unroll 4
  for (int i = first; i < nd * 16; i += step) {
    uint4 v = i < H8 ? __ldg(x + i) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __half2 h = __floats2half2_rn(__uint_as_float(w[j] << 16) * sc, __uint_as_float(w[j] & 0xFFFF0000u) * sc);
      w[j] = *reinterpret_cast<uint32_t*>(&h);
    }
    const int at = chunk_of<FMT>(8 * (i & 15));  // 4 * c + t
    xs[((i >> 4) * 4 + (at >> 2)) * 4 * p.T + 4 * tok + (at & 3)] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int FMT, bool EDGES>
__global__ void __launch_bounds__(kThreads, 1)
    moe_decode_kernel(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map2,
                      const MoeDecodeArgs p, const Plan plan) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes
  const int g = lane >> 2, t = lane & 3;
  if (smem_u32(smem_raw) != kWindow) {  // the plan's alignments assume it
    if (tid == 0) atomicOr(p.err, GNF4_DEVERR_INTERNAL);
    return;
  }
  uint4* xs = reinterpret_cast<uint4*>(smem_raw);
  Route& rt = *reinterpret_cast<Route*>(smem_raw + plan.route);
  Work& wk = *reinterpret_cast<Work*>(smem_raw + plan.work);
  const uint32_t scratch = kWindow + plan.scratch + (uint32_t)(warp * kScratchStride);
  uint8_t* rings = smem_raw + plan.ring;
  Ring ring{};
  ring.ptr = rings + (size_t)warp * plan.stages * kItemBytes;
  ring.base = smem_u32(ring.ptr);
  ring.full = wk.full[warp];
  ring.stages = plan.stages;

  if (tid < kMaxExperts / 32) rt.hit[tid] = 0u;
  if (tid < kMaxExperts / 4) rt.tokens[tid] = 0u;
  if (tid < kMaxT) wk.xmax[tid] = 0u;
  if (tid == 0) {
    wk.abort = 0;
    prefetch_tmap(&map1);
    prefetch_tmap(&map2);
  }
  if (lane < plan.stages) mbar_init(ring.full + lane, 1);
  fence_mbar_init();
  const unsigned parity = __ldcg(p.sync) & 1u;
  unsigned* const barrier = p.sync + 1 + 3 * parity;
  unsigned* const hmax = p.hmax + kMaxPairs * kHmaxStep * parity;
  // the table is laid out while the router's first weights arrive, x while the CTAs meet
  const RouterPart part(p, tid);
  __syncthreads();
  if (FMT == 0) build_table(reinterpret_cast<uint32_t*>(smem_raw + plan.table), tid);
  if (p.router_w != nullptr) {
    if (p.T == 1) router_product<1>(p, wk, part, tid);
    else if (p.T == 2) router_product<2>(p, wk, part, tid);
    else if (p.T <= 4) router_product<4>(p, wk, part, tid);
    else router_product<8>(p, wk, part, tid);
    grid_arrive(barrier);
  }
  stage_x<FMT>(p, wk, xs, tid);
  const int nd2 = (p.I + kDK - 1) / kDK;
  if (p.I % kDK != 0) {  // the last item of every row of h: zero past I
    const int pad = (nd2 * kDK - p.I) / 8;  // chunks
    for (int row = blockIdx.x; row < p.T * p.k; row += gridDim.x)
      for (int i = tid; i < 2 * pad; i += kThreads) {
        const int c = chunk_of<FMT>(p.I % kDK + 8 * (i >> 1));
        reinterpret_cast<float4*>(p.hbuf)[(((size_t)row * nd2 + nd2 - 1) * 16 + c) * 2 + (i & 1)] =
            make_float4(0.f, 0.f, 0.f, 0.f);
      }
  }
  if (blockIdx.x == gridDim.x - 1) {  // what the call before this one used
    if (tid < 3) p.sync[1 + 3 * (1u - parity) + tid] = 0u;
    if (tid < kMaxPairs) p.hmax[kHmaxStep * (kMaxPairs * (1u - parity) + tid)] = 0u;
  }
  if (p.router_w != nullptr) {
    if (!grid_wait(barrier, p.err, &wk.ok)) return;
  } else {
    __syncthreads();
  }
  float logit = 0.f;  // warp t, lane j: the j-th selected logit of token t
  if (warp < p.T) {
    if (p.E <= 64) select_topk<2>(p, rt, warp, lane, &logit);
    else if (p.E <= 128) select_topk<4>(p, rt, warp, lane, &logit);
    else if (p.E <= 384) select_topk<12>(p, rt, warp, lane, &logit);
    else select_topk<kMaxExperts / 32>(p, rt, warp, lane, &logit);
  }
  __syncthreads();
  list_hits(p, rt, &wk.nhit, tid);
  __syncthreads();
  const uint32_t lanesel = (uint32_t)lane * 4u | ((kWindow + plan.table) & 0x00FF0000u);
  Walk<FMT> w;
  uint4 h[4];  // phase 3: the next item's activations on their way

  {  // gate_up + SwiGLU; h times its router weight goes to the workspace in fragment order
    const Stream<FMT, 2> st(p, rt, wk, &map1, lane);
    const Share sh(wk.nhit * st.cols, gridDim.x);
    start_stream<FMT, 2, EDGES>(st, ring, w, sh.begin(blockIdx.x) * st.per, sh.begin(blockIdx.x + 1) * st.per, warp);
    if (warp < p.T) weigh_topk(p, rt, warp, lane, logit);  // while the first weights arrive
    if (w.lo < w.hi) next_scales<FMT, 2, EDGES>(st, w, w.lo, scratch);
    __syncthreads();
    // columns past T repeat the last token and are never stored
    const uint32_t x = kWindow + 16u * (4 * min(g, p.T - 1) + t), x_step = 64u * p.T;
    auto emit = [&](int unit, const float(&acc)[2][4], bool, int r0) {
      const int ei = unit / st.cols;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int tok = 2 * t + i, r = rt.row[ei][tok];
        const float w = r < 0 ? 0.f : rt.sel_p[r];
        uint32_t top = 0u;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = 16 * (unit - ei * st.cols) + 8 * k;  // 8 columns = one chunk
          const size_t chunk = (size_t)(col / kDK) * 16 + chunk_of<FMT>(col % kDK);
          if (r < 0) continue;
          const float v = silu_mul(acc[k][i], acc[k][2 + i]) * w;
          p.hbuf[((size_t)r * nd2 * 16 + chunk) * 8 + r0] = v;
          const uint32_t m = __float_as_uint(v) & 0x7FFFFFFFu;
          top = max(top, m >= 0x7F800000u ? 0u : m);
        }
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (r >= 0 && g == 0) atomicMax(hmax + kHmaxStep * r, top);
      }
    };
    if (!run_stream<FMT, 2, EDGES, true>(st, ring, w, wk, p.err, scratch, x, x_step, lanesel, rings, warp, h, emit))
      return;  // the other CTAs wait at the next meeting until their own limit
  }
  {  // down + combine
    const Stream<FMT, 3> st(p, rt, wk, &map2, lane);
    const Share sh((p.H / 32) * st.per, gridDim.x);
    auto store = [&](int unit, const float(&acc)[2][4], int r0) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 2 * t + (i & 1);
          if (tok < p.T) p.out[(size_t)tok * p.H + 32 * unit + 16 * k + r0 + 8 * (i >> 1)] = __float2bfloat16_rn(acc[k][i]);
        }
    };
    auto emit = [&](int unit, const float(&acc)[2][4], bool whole, int r0) {
      if (whole) {
        store(unit, acc, r0);
        return;
      }
      // the CTAs of the unit's first and last item; all between them hold a part
      const int c0 = sh.owner(unit * st.per), c1 = sh.owner((unit + 1) * st.per - 1);
      float4* part = reinterpret_cast<float4*>(p.part) + lane;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        part[(((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0 ? 1 : 0)) * 2 + k) * 32] =
            make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
      __syncwarp();
      int last = 0;
      if (lane == 0) {
        last = atom_add_acq_rel(p.unit_count + unit, 1u) == (unsigned)(c1 - c0);
        if (last) p.unit_count[unit] = 0u;
      }
      last = __shfl_sync(0xffffffffu, last, 0);
      __syncwarp();
      if (!last) return;
      float sum[2][4] = {};
#pragma unroll 4
      for (int c = c0; c <= c1; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 v = __ldcg(part + (((size_t)c * 2 + (c == c0 ? 1 : 0)) * 2 + k) * 32);
          sum[k][0] += v.x, sum[k][1] += v.y, sum[k][2] += v.z, sum[k][3] += v.w;
        }
      store(unit, sum, r0);
    };
    grid_arrive(barrier + 1);
    // the weights do not wait for the other CTAs
    start_stream<FMT, 3, EDGES>(st, ring, w, sh.begin(blockIdx.x), sh.begin(blockIdx.x + 1), warp);
    if (w.lo < w.hi) next_scales<FMT, 3, EDGES>(st, w, w.lo, scratch);
    if (!grid_wait(barrier + 1, p.err, &wk.ok)) {
      // copies in flight land before the CTA leaves
      drain_boxes(ring.full, ring.stages, ring.get, ring.parity, w.next - w.lo);
      return;
    }
    if (blockIdx.x == 0 && tid == 0) p.sync[0] = 1u - parity;  // every CTA has read it
    const int pairs = p.T * p.k;  // <= 256
    // h to fp16: all of it into every CTA's shared memory, or, where that is
    // too small, each CTA a share in global memory and one more barrier
    const float4* src = reinterpret_cast<const float4*>(p.hbuf);
    const int chunks = pairs * nd2 * 16;  // of 8 values
    const bool here = (uint32_t)chunks * 16u <= plan.act;
    const int c0 = here ? tid : (int)(blockIdx.x * kThreads) + tid, cs = here ? kThreads : (int)gridDim.x * kThreads;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;  // the first chunk comes along with the maxima
    if (c0 < chunks) u = __ldcg(src + 2 * c0), v = __ldcg(src + 2 * c0 + 1);
    if (tid < pairs) wk.hscale[tid] = scale_up(__ldcg(hmax + kHmaxStep * tid));
    __syncthreads();
#pragma unroll 1
    for (int i = c0; i < chunks;) {
      const float sc = wk.hscale[i / (nd2 * 16)];
      __half2 q[4] = {__floats2half2_rn(u.x * sc, u.y * sc), __floats2half2_rn(u.z * sc, u.w * sc),
                      __floats2half2_rn(v.x * sc, v.y * sc), __floats2half2_rn(v.z * sc, v.w * sc)};
      const int to = i;
      i += cs;
      if (i < chunks) u = __ldcg(src + 2 * i), v = __ldcg(src + 2 * i + 1);
      *(here ? reinterpret_cast<uint4*>(smem_raw) + to : p.h16 + to) = *reinterpret_cast<uint4*>(q);
    }
    if (here) {
      __syncthreads();
      const uint32_t x = kWindow + 16u * (uint32_t)t;
      run_stream<FMT, 3, EDGES, true>(st, ring, w, wk, p.err, scratch, x, 64u, lanesel, rings, warp, h, emit);
    } else {
      grid_arrive(barrier + 2);
      if (!grid_wait(barrier + 2, p.err, &wk.ok)) {
        drain_boxes(ring.full, ring.stages, ring.get, ring.parity, w.next - w.lo);
        return;
      }
      if (w.lo < w.hi) st.load_h(h, w.cur);
      run_stream<FMT, 3, EDGES, false>(st, ring, w, wk, p.err, scratch, 0u, 0u, lanesel, rings, warp, h, emit);
    }
  }
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

Plan make_plan(int fmt, int T, int H, int pairs, int I) {
  Plan q{};
  auto up = [](uint32_t n, uint32_t a) { return (n + a - 1) / a * a; };
  const uint32_t x = (uint32_t)((H + kDK - 1) / kDK) * 256u * (uint32_t)T;
  // Room for all of h where that is cheaper than sharing the conversion and meeting once more.  MXFP4: 23 KB (T = 1,
  // k = 4, I = 2880) 31.6 us instead of 33.5, 64 KB (T = 4, k = 8, I = 1024) 39.0 instead of 40.6, but 128 KB (T = 8)
  // 55.4 instead of 53.6.  NF4: 32 KB (T = 4, k = 8, I = 512) 30.0 instead of 30.7, but 64 KB (I = 1024), which moves
  // the table, 44.7 instead of 44.2.  An x that is larger leaves the room anyway.
  const uint32_t h = (uint32_t)pairs * (uint32_t)((I + kDK - 1) / kDK) * 256u;
  const uint32_t limit = fmt == 0 ? 32768u : 65536u;
  q.act = x;
  if (h > q.act && h <= limit) q.act = h;
  q.route = q.act;
  q.work = up(q.route + (uint32_t)sizeof(Route), 16);
  const uint32_t low = up(q.work + (uint32_t)sizeof(Work), 16);
  if (fmt == 0) {
    q.table = (kWindow + low <= 0x10000u ? 0x10000u : 0x20000u) - kWindow;
    if (low > q.table) return q;  // no stages: refused
    q.scratch = q.table + 128;
    q.ring = q.table + kLut256Bytes;
  } else {
    q.scratch = low;
    q.ring = low + kWarps * kScratchStride;
  }
  q.ring = up(kWindow + q.ring, 1024) - kWindow;  // the boxes' swizzle repeats every 512 bytes
  const uint32_t per_stage = kWarps * kItemBytes;
  const uint32_t fit = q.ring < kMaxWindow ? (kMaxWindow - q.ring) / per_stage : 0;
  q.stages = (int)(fit < (uint32_t)kMaxStages ? fit : (uint32_t)kMaxStages);
  q.total = q.ring + (uint32_t)q.stages * per_stage;
  return q;
}

}  // namespace

size_t moe_decode_workspace(int T, int k, int I, size_t* at) {
  size_t n = kSyncBytes;
  at[0] = n;  // hmax
  n = align256(n + 2 * (size_t)kMaxPairs * kHmaxStep * sizeof(unsigned));
  at[1] = n;  // unit_count
  n = align256(n + (size_t)(kMoeDecodeMaxTH / 32) * sizeof(unsigned));  // the same place for every shape: it stays zero
  at[2] = n;  // part
  n += (size_t)kMaxGrid * 2 * 2 * 32 * sizeof(float4);
  at[3] = n;  // hbuf
  n = align256(n + (size_t)T * k * ((I + kDK - 1) / kDK) * kDK * sizeof(float));
  at[4] = n;  // h16
  return align256(n + (size_t)T * k * ((I + kDK - 1) / kDK) * kDK * 2);
}

template <int FMT, bool EDGES>
static cudaError_t launch_t(const CUtensorMap& map1, const CUtensorMap& map2, const MoeDecodeArgs& p, int num_sms,
                            cudaStream_t stream) {
  static std::atomic<bool> configured[64];
  const Plan plan = make_plan(FMT, p.T, p.H, p.T * p.k, p.I);
  const int grid = num_sms < kMaxGrid ? num_sms : kMaxGrid;
  if (plan.stages < 1 || p.E > 8 * grid) return cudaErrorInvalidConfiguration;  // the router: 8 experts a CTA
  cudaError_t e = set_smem_limit_once(moe_decode_kernel<FMT, EDGES>, (int)kMaxWindow, configured);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = plan.total;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the grid barriers need every CTA resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_decode_kernel<FMT, EDGES>, map1, map2, p, plan);
}

cudaError_t launch_moe_decode(int fmt, const CUtensorMap& map1, const CUtensorMap& map2, const MoeDecodeArgs& p,
                              int num_sms, cudaStream_t stream) {
  // Scale arrays that begin at 16-byte boundaries (as allocations do) need no look at their ends, which costs 2 to 5%:
  // NF4, OLMoE shape, T = 8 61.1 us instead of 59.1, MXFP4, 64 experts of 2048 / 1024, T = 4 41.9 instead of 39.4.
  const bool edges = ((reinterpret_cast<uintptr_t>(p.s1) | reinterpret_cast<uintptr_t>(p.s2)) & 15) != 0;
  if (fmt == 0)
    return edges ? launch_t<0, true>(map1, map2, p, num_sms, stream) : launch_t<0, false>(map1, map2, p, num_sms, stream);
  return edges ? launch_t<1, true>(map1, map2, p, num_sms, stream) : launch_t<1, false>(map1, map2, p, num_sms, stream);
}

}  // namespace gnf4
