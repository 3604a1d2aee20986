// router.cu — the MoE router in front of the permute: scores, top-k, routing weights,
// per-expert counts and the balance loss, and the gradient of the logits.
//
// Per token with logits l[e]:
//   softmax   p_e = exp(l_e - max l) / sum exp(l - max l)
//   sigmoid   p_e = 1 / (1 + exp(-l_e))
//   ids       the k experts of the largest l_e (softmax, and sigmoid without a bias: both
//             are increasing in l), or of the largest p_e + bias_e, behind which come those
//             switched off (l_e = -inf); ties to the lowest id
//   weights   scale * p_i, or scale * p_i / (sum of the k chosen p + 1e-20)
// Over the tokens that token_mask keeps, with h_e = p_e (softmax) or
// p_e / (sum of all p + 1e-20) (sigmoid):
//   counts_e = pairs routed to e,  prob_sums_e = sum h_e,  C = sum counts,
//   loss = loss_coef * E * k / C^2 * sum_e counts_e * prob_sums_e
// (for N tokens C = N*k, so this is loss_coef * E * sum f_e * P_e with f_e = counts_e / C
// and P_e = prob_sums_e / N).  counts carries no gradient, so
//   d loss / d h_te = loss_coef * E * k / C^2 * counts_e =: g_e.
// Backward, with P = sum of the chosen p + 1e-20:
//   d p_i += scale * (dw_i - sum_j dw_j p_j / P) / P   (renormalised; else scale * dw_i)
//   softmax: d p_e += g_e;  d l_e = p_e * (d p_e - sum_j d p_j p_j)
//   sigmoid: d p_e += (g_e - sum_j g_j h_j) / (sum of all p + 1e-20);  d l_e = d p_e * p_e * (1 - p_e)
//
// From 129 experts on a warp holds a token: the logits in registers (8 to 32 a lane, 16-byte
// loads of four neighbours), the next token's on their way.  The picks come from a short
// list: the k-th largest of the 32 lanes' maxima bounds the k-th largest value from below, and
// what reaches it (a dozen, typically) is gathered one to a lane, so that a pick is one warp
// maximum and a vote instead of a pass over the row.  With a bias the list is made from fp32
// scores with a margin for their rounding, and only its members are scored in double.
// Up to 128 experts 8 or 16 lanes hold a token and a warp works on four or two.
// All sums are fp32 in a fixed order (per lane over its tokens, at most 256 of them in a launch,
// over the warp's tokens, over the CTA's warps, then over CTAs and launches in double), the
// counts are integers: nothing depends on the order of atomics.
//
// What bounds it: the issue of instructions (ncu at 16384 x 256 with a bias: 67% of the slots in
// both directions), about 820 a token forward and 555 backward.  50021 x 256 fp32 with a bias:
// 56 us forward with statistics, 33 us backward, against 8 and 16 us for the bytes (passing over
// the row for every pick: 130 us).  16384 x 32 BF16, four tokens a warp: 11.3 and 4.7 us (a warp a
// token: 14.5 and 9), of which 5 us are the finishing launch.
#include <cfloat>

#include "abi_checks.h"
#include "cluster.cuh"
#include "common.cuh"
#include "launch.h"

namespace fp8q {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// CTAs that 148 SMs hold at once: four an SM (64 registers a thread) up to 256 experts, two
// above.  A fixed number, so that the order of the sums is the same wherever it runs.
constexpr int resident(int vpl) { return vpl <= 8 ? 4 : 2; }
constexpr int max_blocks(int experts) { return 148 * (experts <= 256 ? resident(8) : resident(16)); }
constexpr int kRouterMaxExperts = 1024;
constexpr int kRouterMaxTopk = 64;
constexpr float kEps = 1e-20f;
constexpr unsigned kAll = 0xFFFFFFFFu;

enum Mode { kSoftmax = 0, kSigmoid = 1, kSigmoidBias = 2 };

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_float<uint16_t>(uint16_t v) {
  return __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Expert i of lane `sub` of the L lanes that hold a token: four neighbours at a time.
template <int L = 32>
__device__ __forceinline__ int expert_of(int sub, int i) {
  return 4 * sub + 4 * L * (i >> 2) + (i & 3);
}

// NaN counts as -inf (a padding row may hold anything), +inf as the largest finite value.
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

// fp32 -> uint32 with the same order (-0 and +0 equal); every value but NaN maps above 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// exp(x), x <= 0, by the hardware base-2 exponential: off by 1.5 |x| + 4 half steps.
__device__ __forceinline__ float exp_neg(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// p = sigmoid(l) and q = 1 - p without cancellation on either side.
__device__ __forceinline__ void sigmoid2(float l, float& p, float& q) {
  const float t = exp_neg(-fabsf(l));
  const float r = rcp(1.0f + t);
  const float s = t * r;
  p = l >= 0.0f ? r : s;
  q = l >= 0.0f ? s : r;
}

// A token's logits as they lie in memory (padding lanes: -inf).  quads: E % 4 == 0, whole and
// aligned quads.
template <int L, int V, typename T>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int sub, bool quads, float (&v)[V]) {
  if (quads) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const int e = expert_of<L>(sub, j);
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) {
        if constexpr (sizeof(T) == 4) {
          f = *reinterpret_cast<const float4*>(row + e);
        } else {
          const uint2 h = *reinterpret_cast<const uint2*>(row + e);
          f = make_float4(__uint_as_float(h.x << 16), __uint_as_float(h.x & 0xFFFF0000u), __uint_as_float(h.y << 16),
                          __uint_as_float(h.y & 0xFFFF0000u));
        }
      }
      v[j] = f.x;
      v[j + 1] = f.y;
      v[j + 2] = f.z;
      v[j + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert_of<L>(sub, i);
      v[i] = e < E ? to_float<T>(row[e]) : -INFINITY;
    }
  }
}
template <int L, int V, typename T>
__device__ __forceinline__ void store_row(T* __restrict__ row, int E, int sub, bool quads, const float (&v)[V]) {
  if (quads) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const int e = expert_of<L>(sub, j);
      if (e < E) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(row + e) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        else
          *reinterpret_cast<uint2*>(row + e) = make_uint2(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = expert_of<L>(sub, i);
      if (e < E) {
        if constexpr (sizeof(T) == 4) row[e] = v[i];
        else row[e] = (T)pack_bf16(v[i], 0.0f);
      }
    }
  }
}
// A warp's row of gradients in shared memory.
template <int L, int V>
__device__ __forceinline__ void read_row(const float* buf, int E, int sub, bool quads, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    if (quads) {
      const int e = expert_of<L>(sub, j);
      const float4 f = e < E ? *reinterpret_cast<const float4*>(buf + e) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      v[j] = f.x;
      v[j + 1] = f.y;
      v[j + 2] = f.z;
      v[j + 3] = f.w;
    } else {
#pragma unroll
      for (int i = j; i < j + 4; ++i) v[i] = expert_of<L>(sub, i) < E ? buf[expert_of<L>(sub, i)] : 0.0f;
    }
  }
}

struct RouterArgs {
  int64_t tokens;
  int E, topk;
  bool renorm, stats;
  float scale;
};
// Where the balance statistics go: the workspace (then router_finish_kernel sums the CTAs'
// parts), or with `fused` (one cluster holds every CTA) straight to the results.
struct StatsOut {
  uint32_t* ws;      // [0]: a counter for the finishing kernel
  float* sums;       // the parts: a row of E sums per CTA (of this launch on)
  int32_t* numbers;  // and of E counts
  int32_t* counts;
  float* prob_sums;
  float* loss;
  float loss_coef;
  bool fused;
};

__device__ __forceinline__ float loss_of(const RouterArgs& a, float loss_coef, double dot, long long c) {
  return c > 0 ? (float)((double)loss_coef * a.E * a.topk / ((double)c * (double)c) * dot) : 0.0f;
}

// The CTA's sums and counts (complete, behind a barrier).
__device__ __forceinline__ void publish(const float* sums, const int* counts, const RouterArgs& a, const StatsOut& out) {
  if (!out.fused) {
    const int64_t at = (int64_t)blockIdx.x * a.E;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      out.sums[at + e] = sums[e];
      out.numbers[at + e] = counts[e];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) out.ws[0] = 0u;
    return;
  }
  __shared__ double dot_sh[kWarps];
  __shared__ long long c_sh[kWarps];
  const uint32_t size = cluster_size();
  __syncthreads();
  cluster_sync();
  if (cluster_rank() == 0) {
    double dot = 0.0;
    long long c = 0;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      double s = 0.0;
      int n = 0;
      for (uint32_t r = 0; r < size; ++r) {  // in rank order
        s += (double)ld_cluster_f32(smem_u32(sums + e), r);
        n += ld_cluster_s32(smem_u32(counts + e), r);
      }
      out.counts[e] = n;
      out.prob_sums[e] = (float)s;
      dot += (double)n * (double)(float)s;
      c += n;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      dot += __shfl_xor_sync(kAll, dot, o);
      c += __shfl_xor_sync(kAll, c, o);
    }
    if ((threadIdx.x & 31) == 0) {
      dot_sh[threadIdx.x >> 5] = dot;
      c_sh[threadIdx.x >> 5] = c;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) {
        dot += dot_sh[w];
        c += c_sh[w];
      }
      *out.loss = loss_of(a, out.loss_coef, dot, c);
    }
  }
  __syncthreads();
  cluster_sync();  // the first CTA has read the others' sums
}

// ------------------------------------------------------------------ selection
struct Pick {
  float l;  // its logit
  int e;
};

// The score that orders experts under a bias, in double (neighbouring scores can be closer
// than an fp32 sum resolves), as the upper and the lower half of a key with the same order.  NaN
// counts as -inf.  An expert that its logit switches off comes below every score; among
// themselves these are ordered by the bias.
constexpr uint32_t kOffKey = 1u;  // (the upper half of -inf's key is 0x000FFFFF)
__device__ __forceinline__ void bias_keys(float l, float bias, uint32_t& hi, uint32_t& lo) {
  if (l == -INFINITY) {
    hi = kOffKey;
    lo = order_key(bias == bias ? bias : -INFINITY);
    return;
  }
  const double s = 1.0 / (1.0 + exp(-(double)l)) + (double)bias;
  const uint64_t b = (uint64_t)__double_as_longlong(s == s ? s + 0.0 : -(double)INFINITY);  // (-0 counts as 0)
  const uint64_t key = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
  hi = (uint32_t)(key >> 32);
  lo = (uint32_t)key;
}

// Any row: each pick passes over the whole row.  Writes the k picks, best first.
template <int VPL, int MODE, typename T>
__device__ __noinline__ void pick_all(const T* row, const float* bias, int E, int K, int lane, Pick* picks) {
  uint32_t key[VPL];
  uint32_t key_lo[MODE == kSigmoidBias ? VPL : 1];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = expert_of(lane, i);
    key[i] = 0u;
    if (MODE == kSigmoidBias) key_lo[i] = 0u;
    if (e < E) {
      const float l = clean(to_float<T>(row[e]));
      if (MODE == kSigmoidBias) bias_keys(l, bias[e], key[i], key_lo[i]);
      else key[i] = order_key(l);
    }
  }
  for (int s = 0; s < K; ++s) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = max(best, key[i]);
    const uint32_t m = __reduce_max_sync(kAll, best);
    uint32_t m_lo = 0u;
    if (MODE == kSigmoidBias) {
      uint32_t b = 0u;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (key[i] == m) b = max(b, key_lo[i]);
      m_lo = __reduce_max_sync(kAll, b);
    }
    uint32_t e = 0xFFFFu;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
      if (key[i] == m && (MODE != kSigmoidBias || key_lo[i] == m_lo)) e = expert_of(lane, i);
    e = __reduce_min_sync(kAll, e);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e == (uint32_t)expert_of(lane, i)) key[i] = 0u;
    if (lane == 0) {
      picks[s].e = (int)e;
      picks[s].l = MODE == kSigmoidBias ? clean(to_float<T>(row[e])) : from_key(m);
    }
  }
  __syncwarp();
}
// How far an fp32 score sigmoid2(l) + bias may be from the exact one: the sigmoid by 2^-21
// (1.5 |l| + 4 half steps of the exponential times s (1 - s), and 4 more, are 5.4 half steps),
// the sum by half a step; the rest covers the arithmetic on the bound itself.
__device__ __forceinline__ float score_error(float score) { return 0x1.4p-21f + 0x1p-23f * fabsf(score); }

constexpr int kListTopk = 16;  // the short list is tried up to this k (it needs k <= 32 lanes)

// From the short list: `order` holds what the row is ordered by (the logits, or fp32 scores
// under a bias), `val` the logits.  false (nothing written) if the list would not fit.
template <int VPL, int MODE>
__device__ __forceinline__ bool pick_listed(const float (&order)[VPL], const float (&val)[VPL],
                                            const float* __restrict__ bias, int K, int lane, Pick* __restrict__ picks) {
  float lm = order[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) lm = fmaxf(lm, order[i]);
  uint32_t cur = order_key(lm), m = 0u;
  for (int s = 0; s < K; ++s) {
    m = __reduce_max_sync(kAll, cur);
    if (lane == __ffs(__ballot_sync(kAll, cur == m)) - 1) cur = 0u;
  }
  float least = from_key(m);
  if (MODE == kSigmoidBias) least -= 2.0f * score_error(least);  // loosened by the errors on either side
  int n = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool in = order[i] >= least;
    const unsigned mask = __ballot_sync(kAll, in);
    const int at = n + __popc(mask & ((1u << lane) - 1u));
    if (in && at < 32) {
      picks[at].l = val[i];
      picks[at].e = expert_of(lane, i);
    }
    n += __popc(mask);
  }
  __syncwarp();
  if (n > 32 || !(least > -INFINITY)) {  // (a bound of -inf, or NaN, lets padding lanes in)
    __syncwarp();
    return false;
  }
  Pick c = {0.0f, 0xFFFF};
  if (lane < n) c = picks[lane];
  __syncwarp();
  uint32_t key = 0u, lo = 0u;
  if (lane < n) {
    if (MODE == kSigmoidBias) bias_keys(c.l, bias[c.e], key, lo);
    else key = order_key(c.l);
  }
  for (int s = 0; s < K; ++s) {
    const uint32_t top = __reduce_max_sync(kAll, key);
    bool won = key == top;
    const unsigned b = __ballot_sync(kAll, won);
    if (b & (b - 1u)) {  // equal upper halves: the lower ones, then the lowest id
      if (MODE == kSigmoidBias) {
        const uint32_t t2 = __reduce_max_sync(kAll, won ? lo : 0u);
        won = won && lo == t2;
      }
      const uint32_t e = __reduce_min_sync(kAll, won ? (uint32_t)c.e : 0xFFFFFFFFu);
      won = won && (uint32_t)c.e == e;
    }
    if (won) {
      picks[s] = c;
      key = 0u;
    }
  }
  __syncwarp();
  return true;
}

// ------------------------------------------------------------------ forward
template <int VPL, int MODE, typename T>
__global__ void __launch_bounds__(kThreads, resident(VPL)) router_kernel(const T* __restrict__ logits, const float* __restrict__ bias,
                                                          const uint8_t* __restrict__ mask, RouterArgs a,
                                                          int32_t* __restrict__ topk_idx, float* __restrict__ weights,
                                                          StatsOut out) {
  constexpr int kSlots = 32 * VPL;
  __shared__ float sums_sh[kSlots];
  __shared__ int counts_sh[kSlots];
  __shared__ Pick picks_sh[kWarps][kRouterMaxTopk];
  pdl_wait_for(logits, bias, mask);
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int E = a.E, K = a.topk;
  const bool quads = (E & 3) == 0, bias_quads = (reinterpret_cast<uintptr_t>(bias) & 15) == 0;
  Pick* picks = picks_sh[wid];
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  if (a.stats) {
    for (int e = threadIdx.x; e < E; e += kThreads) {
      sums_sh[e] = 0.0f;
      counts_sh[e] = 0;
    }
    __syncthreads();
  }
  constexpr bool kAhead = VPL <= 8;  // the next row is loaded while this one is worked on
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  int64_t t = (int64_t)blockIdx.x * kWarps + wid;
  float next[VPL];
  if (kAhead && t < a.tokens) load_row<32, VPL, T>(logits + t * E, E, lane, quads, next);
  for (; t < a.tokens; t += stride) {
    const T* row = logits + t * E;
    const bool live = mask == nullptr || mask[t] != 0;
    float val[VPL];
    if (kAhead) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) val[i] = clean(next[i]);
      if (t + stride < a.tokens) load_row<32, VPL, T>(row + stride * E, E, lane, quads, next);
    } else {
      load_row<32, VPL, T>(row, E, lane, quads, val);
#pragma unroll
      for (int i = 0; i < VPL; ++i) val[i] = clean(val[i]);
    }
    float p[VPL];
    if (MODE != kSoftmax && (MODE == kSigmoidBias || a.stats)) {
      float q;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sigmoid2(val[i], p[i], q);
    }
    // ---- the k picks
    bool done = false;
    if (K <= kListTopk) {
      if (MODE == kSigmoidBias) {
        float order[VPL];
        load_row<32, VPL, float>(bias, E, lane, quads && bias_quads, order);  // (padding lanes: -inf)
        float most = val[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) most = fmaxf(most, val[i]);
        // An expert that is off stays off the list (0 * -inf is NaN), unless all of the row's are.
        const bool some_on = __any_sync(kAll, most > -INFINITY);
#pragma unroll
        for (int i = 0; i < VPL; ++i) order[i] += p[i];
        if (some_on) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) order[i] = __fmaf_rn(val[i], 0.0f, order[i]);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) order[i] = fmaxf(order[i], -INFINITY);  // (NaN counts as -inf)
        done = pick_listed<VPL, MODE>(order, val, bias, K, lane, picks);
      } else {
        done = pick_listed<VPL, MODE>(val, val, bias, K, lane, picks);
      }
    }
    if (!done) pick_all<VPL, MODE, T>(row, bias, E, K, lane, picks);
    Pick mine[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) mine[h] = lane + 32 * h < K ? picks[lane + 32 * h] : Pick{-INFINITY, 0};
    const float top = picks[0].l;
    __syncwarp();
    // ---- probabilities
    float z_inv = 1.0f;  // softmax: 1 / sum exp
    if (MODE == kSoftmax) {
      if (a.stats || !a.renorm) {
        float z = 0.0f;
        const float base = top == -INFINITY ? 0.0f : top;  // a row of -inf has no probability at all
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          p[i] = exp_neg(val[i] - base);
          z += p[i];
        }
        z = warp_sum(z);
        z_inv = z > 0.0f ? rcp(z) : 0.0f;
        if (a.stats && live) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) acc[i] = __fmaf_rn(p[i], z_inv, acc[i]);
        }
      }
    } else if (a.stats) {
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) z += p[i];
      const float share = live ? rcp(warp_sum(z) + kEps) : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = __fmaf_rn(p[i], share, acc[i]);
    }
    float w[2], total = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = 0.0f;
      if (lane + 32 * h < K) {
        if (MODE == kSoftmax) {
          w[h] = top == -INFINITY ? 0.0f : exp_neg(mine[h].l - top);
          if (!a.renorm) w[h] *= z_inv;
        } else {
          float q;
          sigmoid2(mine[h].l, w[h], q);
        }
      }
      total += w[h];
    }
    // The eps is of the size of the probabilities; exp(l - max) exceeds them by the factor
    // z >= 1, for which 1e-20 is as far below fp32 resolution.
    const float factor = a.renorm ? a.scale * rcp(warp_sum(total) + kEps) : a.scale;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int s = lane + 32 * h;
      if (s < K) {
        topk_idx[t * K + s] = mine[h].e;
        weights[t * K + s] = live ? w[h] * factor : 0.0f;
        if (a.stats && live) atomicAdd(&counts_sh[mine[h].e], 1);
      }
    }
  }
  if (!a.stats) return;
  for (int w = 0; w < kWarps; ++w) {  // the warps' sums in order
    if (wid == w) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (expert_of(lane, i) < E) sums_sh[expert_of(lane, i)] += acc[i];
    }
    __syncthreads();
  }
  publish(sums_sh, counts_sh, a, out);
}

// ------------------------------------------------------------------ up to 128 experts
// L lanes (8 or 16) hold a token, 4 or 8 experts a lane, and a warp works on 32 / L tokens at
// once: the rounds of the choice and the sums, which are most of the work, serve them
// together.  Maxima and sums go by shuffles within the L lanes; every lane of the warp takes
// every step, a group past the last token on -inf.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v = min(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

template <int L, int V, int MODE, typename T>
__global__ void __launch_bounds__(kThreads, 4) router_small_kernel(const T* __restrict__ logits,
                                                                   const float* __restrict__ bias,
                                                                   const uint8_t* __restrict__ mask, RouterArgs a,
                                                                   int32_t* __restrict__ topk_idx,
                                                                   float* __restrict__ weights, StatsOut out) {
  constexpr int kGroups = 32 / L;
  __shared__ float sums_sh[L * V];
  __shared__ int counts_sh[L * V];
  __shared__ Pick picks_sh[kWarps][kGroups][kRouterMaxTopk];
  pdl_wait_for(logits, bias, mask);
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, sub = lane & (L - 1), grp = lane / L;
  const int E = a.E, K = a.topk;
  const bool quads = (E & 3) == 0;
  Pick* picks = picks_sh[wid][grp];
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  if (a.stats) {
    for (int e = threadIdx.x; e < E; e += kThreads) {
      sums_sh[e] = 0.0f;
      counts_sh[e] = 0;
    }
    __syncthreads();
  }
  const int64_t stride = (int64_t)gridDim.x * kWarps * kGroups;
  int64_t t = ((int64_t)blockIdx.x * kWarps + wid) * kGroups + grp;
  float next[V];
  auto load = [&](int64_t u) {
    if (u < a.tokens) {
      load_row<L, V, T>(logits + u * E, E, sub, quads, next);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) next[i] = -INFINITY;
    }
  };
  load(t);
  for (; t - grp < a.tokens; t += stride) {  // the warp's first token decides for all
    const bool here = t < a.tokens;
    const bool live = here && (mask == nullptr || mask[t] != 0);
    const T* row = logits + (here ? t : 0) * E;
    float val[V];
    uint32_t key[V], key_lo[MODE == kSigmoidBias ? V : 1];
#pragma unroll
    for (int i = 0; i < V; ++i) val[i] = clean(next[i]);
    load(t + stride);
    // ---- the k picks, by `key` (and under a bias its lower half `key_lo`).  With `check`, one
    // round more: true if two neighbours in the order may be closer than their fp32 errors.
    auto choose = [&](bool check) {
      bool close = false;
      float before = INFINITY;
      for (int s = 0; s < K + (check ? 1 : 0); ++s) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < V; ++i) best = max(best, key[i]);
        const uint32_t m = group_max<L>(best);
        if (check) {
          const float f = from_key(m);
          close |= s > 0 && s < E && !(before - f > 2.0f * score_error(before));
          before = f;
          if (s == K) break;
        }
        uint32_t m_lo = 0u;
        if (MODE == kSigmoidBias && !check) {
          uint32_t b = 0u;
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (key[i] == m) b = max(b, key_lo[i]);
          m_lo = group_max<L>(b);
        }
        uint32_t e = 0xFFFFu;
        float l = 0.0f;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
          if (key[i] == m && (MODE != kSigmoidBias || check || key_lo[i] == m_lo)) {
            e = expert_of<L>(sub, i);
            l = val[i];
          }
        const uint32_t first = group_min<L>(e);
        if (e == first) {  // the lane that holds it
          picks[s].e = (int)e;
          picks[s].l = l;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (first == (uint32_t)expert_of<L>(sub, i)) key[i] = 0u;
      }
      __syncwarp();
      return close;
    };
    if (MODE == kSigmoidBias) {
      // fp32 scores decide where they can; where some token's are too close, the warp's tokens
      // are scored in double (for every token that cost half of the kernel's time).
      // Experts that are off count as -inf there (0 * -inf is NaN), which sets none of them before
      // another; where a whole row is off, its biases do.
      float score[V], most = val[0];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = expert_of<L>(sub, i);
        float p, q;
        sigmoid2(val[i], p, q);
        score[i] = e < E ? p + bias[e] : 0.0f;
        most = fmaxf(most, val[i]);
      }
      const bool some_on = (__ballot_sync(kAll, most > -INFINITY) >> (grp * L) & ((1u << L) - 1u)) != 0u;
      if (__all_sync(kAll, some_on)) {
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] = __fmaf_rn(val[i], 0.0f, score[i]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (some_on && val[i] == -INFINITY) score[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        key[i] = expert_of<L>(sub, i) < E ? order_key(score[i] == score[i] ? score[i] : -INFINITY) : 0u;
      if (__any_sync(kAll, choose(true) && here)) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = expert_of<L>(sub, i);
          key[i] = key_lo[i] = 0u;
          if (e < E) bias_keys(val[i], bias[e], key[i], key_lo[i]);
        }
        choose(false);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = expert_of<L>(sub, i) < E ? order_key(val[i]) : 0u;
      choose(false);
    }
    const float top = picks[0].l;  // (softmax: the row's maximum)
    // ---- probabilities
    float z_inv = 1.0f;
    if (MODE == kSoftmax) {
      if (a.stats || !a.renorm) {
        float p[V], z = 0.0f;
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          p[i] = exp_neg(val[i] - base);
          z += p[i];
        }
        z = group_sum<L>(z);
        z_inv = z > 0.0f ? rcp(z) : 0.0f;
        const float share = live ? z_inv : 0.0f;
        if (a.stats) {
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(p[i], share, acc[i]);
        }
      }
    } else if (a.stats) {
      float p[V], q, z = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sigmoid2(val[i], p[i], q);
        z += p[i];
      }
      z = group_sum<L>(z);
      const float share = live ? rcp(z + kEps) : 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(p[i], share, acc[i]);
    }
    auto weight = [&](float l) {
      float w, q;
      if (MODE == kSoftmax) {
        w = top == -INFINITY ? 0.0f : exp_neg(l - top);
        return a.renorm ? w : w * z_inv;
      }
      sigmoid2(l, w, q);
      return w;
    };
    float total = 0.0f;
    if (a.renorm)
      for (int s = sub; s < K; s += L) total += weight(picks[s].l);
    const float factor = a.renorm ? a.scale * rcp(group_sum<L>(total) + kEps) : a.scale;
    if (here) {
      for (int s = sub; s < K; s += L) {
        const Pick p = picks[s];
        topk_idx[t * K + s] = p.e;
        weights[t * K + s] = live ? weight(p.l) * factor : 0.0f;
        if (a.stats && live) atomicAdd(&counts_sh[p.e], 1);
      }
    }
    __syncwarp();
  }
  if (!a.stats) return;
#pragma unroll
  for (int o = L; o < 32; o <<= 1)  // over the warp's tokens
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = __fadd_rn(acc[i], __shfl_xor_sync(kAll, acc[i], o));
  for (int w = 0; w < kWarps; ++w) {  // the warps' sums in order
    if (wid == w && grp == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (expert_of<L>(sub, i) < E) sums_sh[expert_of<L>(sub, i)] += acc[i];
    }
    __syncthreads();
  }
  publish(sums_sh, counts_sh, a, out);
}

// Sums the CTAs' partial results: a cluster of CTAs per 32 experts, its warps sharing the
// rows (10 each at most, all on their way at once), the CTAs' sums joined in rank order; the
// last cluster to finish (the counter was zeroed by the kernel before) forms the loss.
constexpr int kFinishCluster = 8;
__global__ void __launch_bounds__(kThreads) router_finish_kernel(int blocks, RouterArgs a, StatsOut out) {
  __shared__ double sum_sh[kWarps][32];
  __shared__ int cnt_sh[kWarps][32];
  __shared__ bool last;
  pdl_wait_for(out.ws, out.sums, out.numbers, out.counts, out.prob_sums);
  pdl_trigger();
  const int E = a.E;
  uint32_t* ws = out.ws;
  int32_t* counts = out.counts;
  float* prob_sums = out.prob_sums;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int e = blockIdx.x / size * 32 + lane;
  const float* part = out.sums;
  const int32_t* part_n = out.numbers;
  double s = 0.0;
  int n = 0;
  if (e < E) {
#pragma unroll 10
    for (int b = rank * kWarps + wid; b < blocks; b += size * kWarps) {
      s += (double)part[(int64_t)b * E + e];
      n += part_n[(int64_t)b * E + e];
    }
  }
  sum_sh[wid][lane] = s;
  cnt_sh[wid][lane] = n;
  __syncthreads();
  if (wid == 0) {
    for (int w = 1; w < kWarps; ++w) {
      s += sum_sh[w][lane];
      n += cnt_sh[w][lane];
    }
    sum_sh[0][lane] = s;
    cnt_sh[0][lane] = n;
  }
  if (size > 1) {
    __syncwarp();
    cluster_sync();
    if (rank == 0 && wid == 0) {
      double ps[kFinishCluster];
      int pn[kFinishCluster];
#pragma unroll
      for (uint32_t r = 1; r < kFinishCluster; ++r) {  // all on their way, then added in rank order
        ps[r] = r < size ? ld_cluster_f64(smem_u32(&sum_sh[0][lane]), r) : 0.0;
        pn[r] = r < size ? ld_cluster_s32(smem_u32(&cnt_sh[0][lane]), r) : 0;
      }
#pragma unroll
      for (uint32_t r = 1; r < kFinishCluster; ++r) {
        s += ps[r];
        n += pn[r];
      }
    }
    __syncwarp();
    cluster_sync();  // the peers' sums were read: they may end
  }
  if (rank != 0 || wid != 0) return;
  if (e < E) {
    counts[e] = n;
    prob_sums[e] = (float)s;
  }
  double dot = 0.0;
  long long c = 0;
  if (E <= 32) {  // one cluster: everything is here
    c = n;
    dot = (double)n * (double)(float)s;
  } else {
    __threadfence();
    __syncwarp();
    if (lane == 0) last = atomicAdd(ws, 1u) == gridDim.x / size - 1;
    __syncwarp();
    if (!last) return;
    __threadfence();
#pragma unroll 4
    for (int i = lane; i < E; i += 32) {
      const int32_t ci = __ldcg(counts + i);
      dot += (double)ci * (double)__ldcg(prob_sums + i);
      c += ci;
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    dot += __shfl_xor_sync(kAll, dot, o);
    c += __shfl_xor_sync(kAll, c, o);
  }
  if (lane == 0) *out.loss = loss_of(a, out.loss_coef, dot, c);
}

// ------------------------------------------------------------------ backward
// g_e of every expert into shared memory; ends with a barrier.
__device__ __forceinline__ void balance_slopes(const int32_t* counts, const RouterArgs& a, float loss_coef,
                                               const float* grad_loss, float* g_sh) {
  __shared__ long long c_sh[kWarps];
  long long c = 0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) c += counts[e];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) c += __shfl_xor_sync(kAll, c, o);
  if ((threadIdx.x & 31) == 0) c_sh[threadIdx.x >> 5] = c;
  __syncthreads();
  c = 0;
  for (int w = 0; w < kWarps; ++w) c += c_sh[w];
  const double f = c > 0 ? (double)*grad_loss * (double)loss_coef * a.E * a.topk / ((double)c * (double)c) : 0.0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) g_sh[e] = (float)(f * (double)counts[e]);
  __syncthreads();
}

template <int VPL, bool SIGMOID, typename T>
__global__ void __launch_bounds__(kThreads, resident(VPL)) router_bwd_kernel(const T* __restrict__ logits,
                                                              const uint8_t* __restrict__ mask, RouterArgs a,
                                                              const int32_t* __restrict__ topk_idx,
                                                              const float* __restrict__ grad_weights,
                                                              const int32_t* __restrict__ row_id_map, int64_t rows,
                                                              const int32_t* __restrict__ counts, float loss_coef,
                                                              const float* __restrict__ grad_loss,
                                                              T* __restrict__ grad, int* status) {
  extern __shared__ __align__(16) float sh[];  // g_e, then a row per warp
  pdl_wait_for(logits, mask, topk_idx, grad_weights, row_id_map, counts, grad_loss);
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int E = a.E, K = a.topk;
  const bool balance = grad_loss != nullptr;
  float* g_sh = sh;
  const int pitch = (E + 3) & ~3;  // rows on 16 bytes
  float* buf = sh + (1 + wid) * pitch;
  if (balance) balance_slopes(counts, a, loss_coef, grad_loss, g_sh);
  float g[VPL];  // this lane's g_e
#pragma unroll
  for (int i = 0; i < VPL; ++i) g[i] = balance && expert_of(lane, i) < E ? g_sh[expert_of(lane, i)] : 0.0f;
  const bool quads = (E & 3) == 0;
  // A row of zeros per warp, into which the chosen experts' gradients are put and taken out
  // again.
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (expert_of(lane, i) < E) buf[expert_of(lane, i)] = 0.0f;
  __syncwarp();
  constexpr bool kAhead = VPL <= 8;
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  int64_t t = (int64_t)blockIdx.x * kWarps + wid;
  float next[VPL];
  if (kAhead && t < a.tokens) load_row<32, VPL, T>(logits + t * E, E, lane, quads, next);
  int next_id[2] = {-1, -1};  // this lane's slots of the next token: expert (or -1), gradient
  float next_dw[2] = {0.0f, 0.0f};
  auto load_slots = [&](int64_t u) {
    if (grad_weights == nullptr || (mask != nullptr && mask[u] == 0)) return;  // (a masked token's are not used)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int s = lane + 32 * h;
      if (s < K) {
        const int e = topk_idx[u * K + s];
        int64_t at = u * K + s;
        bool ok = e >= 0 && e < E;
        if (row_id_map != nullptr) {
          at = row_id_map[at];
          ok = ok && at >= 0 && at < rows;
        }
        next_id[h] = ok ? e : -1;
        next_dw[h] = ok ? grad_weights[at] : 0.0f;
        if (!ok) record_status(status, FP8Q_ERR_DEVICE);
      }
    }
  };
  if (t < a.tokens) load_slots(t);
  for (; t < a.tokens; t += stride) {
    const T* row = logits + t * E;
    float p[VPL];
    if (kAhead) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] = clean(next[i]);
      if (t + stride < a.tokens) load_row<32, VPL, T>(row + stride * E, E, lane, quads, next);
    } else {
      load_row<32, VPL, T>(row, E, lane, quads, p);
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] = clean(p[i]);
    }
    if (mask != nullptr && mask[t] == 0) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] = 0.0f;
      store_row<32, VPL, T>(grad + t * E, E, lane, quads, p);
      if (t + stride < a.tokens) load_slots(t + stride);
      continue;
    }
    // ---- the slots: lane s (and 32 + s) holds slot s
    int id[2];
    float dw[2], ps[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      id[h] = next_id[h];
      dw[h] = next_dw[h];
      ps[h] = id[h] >= 0 ? clean(to_float<T>(row[id[h]])) : 0.0f;
    }
    if (t + stride < a.tokens) load_slots(t + stride);
    // ---- probabilities (softmax: not yet divided by their sum) and the row's sums
    float q[SIGMOID ? VPL : 1], unused;
    if (SIGMOID) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) sigmoid2(p[i], p[i], q[i]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (id[h] >= 0) sigmoid2(ps[h], ps[h], unused);
      }
    } else {
      float m = p[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) m = fmaxf(m, p[i]);
      m = from_key(__reduce_max_sync(kAll, order_key(m)));
      const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] = exp_neg(p[i] - base);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (id[h] >= 0) ps[h] = exp_neg(ps[h] - base);
    }
    float z = 0.0f, gp = 0.0f, total = ps[0] + ps[1], dot = dw[0] * ps[0] + dw[1] * ps[1];
#pragma unroll
    for (int i = 0; i < VPL; ++i) z += p[i];
    if (balance) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) gp = __fmaf_rn(g[i], p[i], gp);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {  // four independent sums a step
      z = __fadd_rn(z, __shfl_xor_sync(kAll, z, o));
      gp = __fadd_rn(gp, __shfl_xor_sync(kAll, gp, o));
      total = __fadd_rn(total, __shfl_xor_sync(kAll, total, o));
      dot = __fadd_rn(dot, __shfl_xor_sync(kAll, dot, o));
    }
    const float z_inv = SIGMOID ? rcp(z + kEps) : (z > 0.0f ? rcp(z) : 0.0f);
    // Softmax probabilities carry the factor z_inv: in P = sum of the chosen p + 1e-20, and
    // in mean = sum dw p / P.
    const float unit = SIGMOID ? 1.0f : z_inv;
    const float inv = a.renorm ? rcp(total * unit + kEps) : 1.0f;
    const float mean = a.renorm ? dot * unit * inv : 0.0f;
    const float own = a.scale * inv;
    // ---- the chosen experts' part, through the warp's row
    if (grad_weights != nullptr) {
      // Ids are distinct in a row the router wrote; should a caller repeat one, the slots are
      // added one by one, in slot order.
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (id[h] >= 0) buf[id[h]] = __int_as_float(1 + lane + 32 * h);
      __syncwarp();
      bool repeated = false;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        repeated |= id[h] >= 0 && __float_as_int(buf[id[h]]) != 1 + lane + 32 * h;
      __syncwarp();
      if (!__any_sync(kAll, repeated)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (id[h] >= 0) buf[id[h]] = own * (dw[h] - mean);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (id[h] >= 0) buf[id[h]] = 0.0f;
        __syncwarp();
        for (int s = 0; s < K; ++s) {
          const int e = s < 32 ? id[0] : id[1];
          if (lane == (s & 31) && e >= 0) buf[e] += own * ((s < 32 ? dw[0] : dw[1]) - mean);
          __syncwarp();
        }
      }
      __syncwarp();
    }
    float d[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
    if (grad_weights != nullptr) {
      read_row<32, VPL>(buf, E, lane, quads, d);
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (id[h] >= 0) buf[id[h]] = 0.0f;
    }
    // ---- through the scores
    if (SIGMOID) {
      if (balance) {
        const float base = gp * z_inv;
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = __fmaf_rn(g[i] - base, z_inv, d[i]);
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] *= p[i] * q[i];
    } else {
      // sum d p: the balance part over all experts, and the slots' own * (dw - mean) p
      const float all = __fmaf_rn(own * unit, dot - mean * total, gp * unit);
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] = (p[i] * unit) * ((balance ? d[i] + g[i] : d[i]) - all);
    }
    store_row<32, VPL, T>(grad + t * E, E, lane, quads, d);
    __syncwarp();
  }
}

// Up to 128 experts: L lanes a token, as in router_small_kernel.
template <int L, int V, bool SIGMOID, typename T>
__global__ void __launch_bounds__(kThreads, 4) router_small_bwd_kernel(
    const T* __restrict__ logits, const uint8_t* __restrict__ mask, RouterArgs a, const int32_t* __restrict__ topk_idx,
    const float* __restrict__ grad_weights, const int32_t* __restrict__ row_id_map, int64_t rows,
    const int32_t* __restrict__ counts, float loss_coef, const float* __restrict__ grad_loss, T* __restrict__ grad,
    int* status) {
  constexpr int kGroups = 32 / L;
  __shared__ float g_sh[L * V];
  __shared__ __align__(16) float buf_sh[kWarps][kGroups][L * V];
  pdl_wait_for(logits, mask, topk_idx, grad_weights, row_id_map, counts, grad_loss);
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, sub = lane & (L - 1), grp = lane / L;
  const int E = a.E, K = a.topk;
  const bool balance = grad_loss != nullptr, quads = (E & 3) == 0;
  float* buf = buf_sh[wid][grp];
  if (balance) balance_slopes(counts, a, loss_coef, grad_loss, g_sh);
  float g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert_of<L>(sub, i);
    g[i] = balance && e < E ? g_sh[e] : 0.0f;
    buf[e] = 0.0f;
  }
  __syncwarp();
  const int64_t stride = (int64_t)gridDim.x * kWarps * kGroups;
  for (int64_t t = ((int64_t)blockIdx.x * kWarps + wid) * kGroups + grp; t - grp < a.tokens; t += stride) {
    const bool here = t < a.tokens;
    const bool live = here && (mask == nullptr || mask[t] != 0);
    const T* row = logits + (here ? t : 0) * E;
    float p[V], q[SIGMOID ? V : 1], unused;
    if (live) {
      load_row<L, V, T>(row, E, sub, quads, p);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = -INFINITY;
    }
    float base = 0.0f;
    if (SIGMOID) {
#pragma unroll
      for (int i = 0; i < V; ++i) sigmoid2(clean(p[i]), p[i], q[i]);
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = clean(p[i]);
        m = fmaxf(m, p[i]);
      }
#pragma unroll
      for (int o = L / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
      base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = exp_neg(p[i] - base);
    }
    // Slot s of a live token: its expert (-1: to be skipped) and its weight's gradient.
    auto slot = [&](int s, float& dw) {
      const int e = topk_idx[t * K + s];
      int64_t at = t * K + s;
      bool ok = e >= 0 && e < E;
      if (row_id_map != nullptr) {
        at = row_id_map[at];
        ok = ok && at >= 0 && at < rows;
      }
      dw = ok ? grad_weights[at] : 0.0f;
      return ok ? e : -1;
    };
    const bool slots = live && grad_weights != nullptr;
    float z = 0.0f, gp = 0.0f, total = 0.0f, dot = 0.0f, dw;
    if (slots) {
      for (int s = sub; s < K; s += L) {
        const int e = slot(s, dw);
        if (e < 0) {
          record_status(status, FP8Q_ERR_DEVICE);
          continue;
        }
        float ps = clean(to_float<T>(row[e]));
        if (SIGMOID) sigmoid2(ps, ps, unused);
        else ps = exp_neg(ps - base);
        total += ps;
        dot = __fmaf_rn(dw, ps, dot);
        buf[e] = __int_as_float(1 + s);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z += p[i];
      gp = __fmaf_rn(g[i], p[i], gp);
    }
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) {
      z = __fadd_rn(z, __shfl_xor_sync(kAll, z, o));
      gp = __fadd_rn(gp, __shfl_xor_sync(kAll, gp, o));
      total = __fadd_rn(total, __shfl_xor_sync(kAll, total, o));
      dot = __fadd_rn(dot, __shfl_xor_sync(kAll, dot, o));
    }
    const float z_inv = SIGMOID ? rcp(z + kEps) : (z > 0.0f ? rcp(z) : 0.0f);
    const float unit = SIGMOID ? 1.0f : z_inv;  // as in router_bwd_kernel
    const float inv = a.renorm ? rcp(total * unit + kEps) : 1.0f;
    const float mean = a.renorm ? dot * unit * inv : 0.0f;
    const float own = a.scale * inv;
    bool repeated = false;
    __syncwarp();
    if (slots)
      for (int s = sub; s < K; s += L) {
        const int e = slot(s, dw);
        repeated |= e >= 0 && __float_as_int(buf[e]) != 1 + s;
      }
    __syncwarp();
    if (!__any_sync(kAll, repeated)) {
      if (slots)
        for (int s = sub; s < K; s += L) {
          const int e = slot(s, dw);
          if (e >= 0) buf[e] = own * (dw - mean);
        }
    } else {  // ids that a caller repeated: one slot after the other
      if (slots)
        for (int s = sub; s < K; s += L) {
          const int e = slot(s, dw);
          if (e >= 0) buf[e] = 0.0f;
        }
      __syncwarp();
      for (int s = 0; s < K; ++s) {
        if (slots && sub == (s & (L - 1))) {
          const int e = slot(s, dw);
          if (e >= 0) buf[e] += own * (dw - mean);
        }
        __syncwarp();
      }
    }
    __syncwarp();
    float d[V];
    read_row<L, V>(buf, E, sub, quads, d);
    __syncwarp();
    if (slots)
      for (int s = sub; s < K; s += L) {
        const int e = slot(s, dw);
        if (e >= 0) buf[e] = 0.0f;
      }
    if (SIGMOID) {
      if (balance) {
        const float shared = gp * z_inv;
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = __fmaf_rn(g[i] - shared, z_inv, d[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] *= p[i] * q[i];
    } else {
      const float all = __fmaf_rn(own * unit, dot - mean * total, gp * unit);
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = (p[i] * unit) * (d[i] + g[i] - all);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = live ? d[i] : 0.0f;
    if (here) store_row<L, V, T>(grad + t * E, E, sub, quads, d);
    __syncwarp();
  }
}

// Routing weights to their destination rows: the rows are set to zero by one launch, then
// one thread per pair stores its weight.
__global__ void __launch_bounds__(256) zero_rows_kernel(float* __restrict__ row_weights, int64_t rows) {
  pdl_wait_for(row_weights);
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < rows) row_weights[i] = 0.0f;
}
__global__ void __launch_bounds__(256) scatter_weights_kernel(const float* __restrict__ weights,
                                                              const int32_t* __restrict__ row_id_map, int64_t pairs,
                                                              int64_t rows, float* __restrict__ row_weights,
                                                              int* status) {
  pdl_wait_for(weights, row_id_map);
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= pairs) return;
  const int64_t r = row_id_map[i];
  if (r < 0 || r >= rows) {
    record_status(status, FP8Q_ERR_DEVICE);
    return;
  }
  row_weights[r] = weights[i];
}

// Tokens a CTA takes at a time, and the CTAs of a forward launch.
int tokens_per_cta(int experts) { return kWarps * (experts <= 64 ? 4 : experts <= 128 ? 2 : 1); }
int router_blocks(int64_t tokens, int experts) {
  const int64_t b = (tokens + tokens_per_cta(experts) - 1) / tokens_per_cta(experts);
  return (int)(b < 1 ? 1 : b < max_blocks(experts) ? b : max_blocks(experts));
}
// A lane adds its tokens' shares one after the other.  With statistics a launch takes 256 of them a
// lane at most (1.2 million tokens from 129 experts on, 2.4 or 4.8 million below): one share added
// 74000 times over, by a router that has not learned yet, would be off by 1e-3.
constexpr int kRounds = 256;
int64_t tokens_per_launch(int experts) { return (int64_t)kRounds * tokens_per_cta(experts) * max_blocks(experts); }
// CTAs of all launches.
int64_t stats_rows(int64_t tokens, int experts) {
  const int64_t most = tokens_per_launch(experts);
  if (tokens <= most) return router_blocks(tokens, experts);
  return tokens / most * max_blocks(experts) + (tokens % most ? router_blocks(tokens % most, experts) : 0);
}
// Few tokens: up to eight CTAs, two rounds each, joined as one cluster - no second launch (64
// tokens to 32 experts: 5.4 us on the GPU; four rounds, 1000 tokens, took 11.6 us, as much as
// the second launch costs).
constexpr int kFusedCtas = 8;
bool fused(int64_t tokens, int experts) { return tokens <= (int64_t)2 * kFusedCtas * tokens_per_cta(experts); }

struct FwdPtrs {
  const float* bias;
  const uint8_t* mask;
  int32_t* idx;
  float* weights;
};

template <typename T>
cudaError_t launch_fwd(int mode, const T* logits, const FwdPtrs& p, const RouterArgs& a, const StatsOut& out, int blocks,
                       cudaStream_t st) {
  using Kernel = void (*)(const T*, const float*, const uint8_t*, RouterArgs, int32_t*, float*, StatsOut);
#define FP8Q_BY_MODE(name, ...) \
  (mode == kSoftmax ? (Kernel)name<__VA_ARGS__, kSoftmax, T> \
                    : mode == kSigmoid ? (Kernel)name<__VA_ARGS__, kSigmoid, T> : (Kernel)name<__VA_ARGS__, kSigmoidBias, T>)
  const Kernel k = a.E <= 32    ? FP8Q_BY_MODE(router_small_kernel, 8, 4)
                   : a.E <= 64  ? FP8Q_BY_MODE(router_small_kernel, 8, 8)
                   : a.E <= 128 ? FP8Q_BY_MODE(router_small_kernel, 16, 8)
                   : a.E <= 256 ? FP8Q_BY_MODE(router_kernel, 8)
                   : a.E <= 512 ? FP8Q_BY_MODE(router_kernel, 16)
                                : FP8Q_BY_MODE(router_kernel, 32);
#undef FP8Q_BY_MODE
  return launch_clusters_after(k, (unsigned)blocks, out.fused ? (unsigned)blocks : 1u, kThreads, 0, st, logits, p.bias,
                               p.mask, a, p.idx, p.weights, out);
}

struct BwdPtrs {
  const uint8_t* mask;
  const int32_t* idx;
  const float* gw;
  const int32_t* map;
  int64_t rows;
  const int32_t* counts;
  float loss_coef;
  const float* grad_loss;
};

template <typename T>
cudaError_t launch_bwd(bool sigmoid, const T* logits, const RouterArgs& a, const BwdPtrs& p, T* grad, int* status,
                       cudaStream_t st) {
  using Kernel = void (*)(const T*, const uint8_t*, RouterArgs, const int32_t*, const float*, const int32_t*, int64_t,
                          const int32_t*, float, const float*, T*, int*);
#define FP8Q_BY_MODE(name, ...) (sigmoid ? (Kernel)name<__VA_ARGS__, true, T> : (Kernel)name<__VA_ARGS__, false, T>)
  const Kernel k = a.E <= 32    ? FP8Q_BY_MODE(router_small_bwd_kernel, 8, 4)
                   : a.E <= 64  ? FP8Q_BY_MODE(router_small_bwd_kernel, 8, 8)
                   : a.E <= 128 ? FP8Q_BY_MODE(router_small_bwd_kernel, 16, 8)
                   : a.E <= 256 ? FP8Q_BY_MODE(router_bwd_kernel, 8)
                   : a.E <= 512 ? FP8Q_BY_MODE(router_bwd_kernel, 16)
                                : FP8Q_BY_MODE(router_bwd_kernel, 32);
#undef FP8Q_BY_MODE
  // The larger kernel's g_e and a row per warp: at most 36 KB.
  const size_t smem = a.E <= 128 ? 0 : (size_t)(kWarps + 1) * ((a.E + 3) & ~3) * sizeof(float);
  return launch_after(k, dim3((unsigned)router_blocks(a.tokens, a.E)), kThreads, smem, st, logits, p.mask, a, p.idx, p.gw,
                      p.map, p.rows, p.counts, p.loss_coef, p.grad_loss, grad, status);
}

constexpr uint32_t kKnownFlags = FP8Q_ROUTER_SIGMOID | FP8Q_ROUTER_RENORM | FP8Q_ROUTER_BF16;

// Sizes shared by both directions.
fp8q_status check_router(int64_t tokens, int32_t num_experts, uint32_t flags, int32_t topk) {
  if (num_experts < 1 || num_experts > kRouterMaxExperts || topk < 1 || topk > kRouterMaxTopk || topk > num_experts ||
      (flags & ~kKnownFlags))
    return FP8Q_ERR_ARG;
  if (tokens < 0 || tokens > kMaxInt32 / topk) return FP8Q_ERR_SHAPE;
  return FP8Q_OK;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" {

size_t fp8q_router_workspace_bytes(int64_t tokens, int32_t num_experts) {
  if (tokens < 0 || num_experts < 1 || num_experts > kRouterMaxExperts) return 0;
  if (fused(tokens, num_experts)) return 16;
  return 16 + (size_t)stats_rows(tokens, num_experts) * num_experts * 8;
}

fp8q_status fp8q_router_topk(const void* logits, int64_t tokens, int32_t num_experts, uint32_t flags,
                             const float* bias, const uint8_t* token_mask, int32_t topk, float scale, float loss_coef,
                             int32_t* topk_idx, float* weights, int32_t* counts, float* prob_sums, float* loss,
                             void* workspace, size_t workspace_bytes, fp8q_stream_t stream) {
  const fp8q_status c = check_router(tokens, num_experts, flags, topk);
  if (c != FP8Q_OK) return c;
  if (bias && !(flags & FP8Q_ROUTER_SIGMOID)) return FP8Q_ERR_ARG;
  const bool stats = counts != nullptr;
  if (stats != (prob_sums != nullptr) || stats != (loss != nullptr)) return FP8Q_ERR_ARG;
  if (tokens == 0 && !stats) return FP8Q_OK;
  if (tokens > 0 && (!logits || !topk_idx || !weights)) return FP8Q_ERR_NULL;
  if (!aligned_to(logits, 16) || !aligned_to(topk_idx, 4) || !aligned_to(weights, 4) || !aligned_to(bias, 4) ||
      !aligned_to(counts, 4) || !aligned_to(prob_sums, 4) || !aligned_to(loss, 4))
    return FP8Q_ERR_ALIGN;
  if (stats) {
    if (!workspace) return FP8Q_ERR_NULL;
    if (!aligned_to(workspace, 16)) return FP8Q_ERR_ALIGN;
    if (workspace_bytes < fp8q_router_workspace_bytes(tokens, num_experts)) return FP8Q_ERR_ARG;
  }
  DeviceInfo dev;
  if (device_info(&dev) != FP8Q_OK) return FP8Q_ERR_CUDA;
  RouterArgs a = {tokens, num_experts, topk, (flags & FP8Q_ROUTER_RENORM) != 0, stats, scale};
  const int mode = !(flags & FP8Q_ROUTER_SIGMOID) ? kSoftmax : bias ? kSigmoidBias : kSigmoid;
  cudaStream_t st = to_stream(stream);
  const bool one = stats && fused(tokens, num_experts);
  // Workspace: 16 bytes, then all CTAs' rows of sums, then of counts.
  const int64_t rows = stats ? stats_rows(tokens, num_experts) : 0;
  float* sums = stats ? static_cast<float*>(workspace) + 4 : nullptr;
  int32_t* numbers = stats ? reinterpret_cast<int32_t*>(sums + rows * num_experts) : nullptr;
  StatsOut out = {static_cast<uint32_t*>(workspace), sums, numbers, counts, prob_sums, loss, loss_coef, one};
  const int64_t most = stats ? tokens_per_launch(num_experts) : tokens;
  for (int64_t t = 0; t == 0 || t < tokens; t += most) {
    a.tokens = tokens - t < most ? tokens - t : most;
    int blocks = router_blocks(a.tokens, num_experts);
    if (one && blocks > kFusedCtas) blocks = kFusedCtas;
    const FwdPtrs p = {bias, token_mask ? token_mask + t : nullptr, topk_idx + t * topk, weights + t * topk};
    const cudaError_t rc =
        (flags & FP8Q_ROUTER_BF16)
            ? launch_fwd(mode, static_cast<const uint16_t*>(logits) + t * num_experts, p, a, out, blocks, st)
            : launch_fwd(mode, static_cast<const float*>(logits) + t * num_experts, p, a, out, blocks, st);
    if (rc != cudaSuccess) return FP8Q_ERR_CUDA;
    if (stats) {
      out.sums += (int64_t)blocks * num_experts;
      out.numbers += (int64_t)blocks * num_experts;
    }
  }
  if (!stats || one) return FP8Q_OK;
  out.sums = sums;
  out.numbers = numbers;
  // Few rows need no cluster: 64 are one or two a warp.
  const unsigned size = rows > 64 ? kFinishCluster : rows > kWarps ? 2 : 1;
  return launch_clusters_after(router_finish_kernel, (unsigned)((num_experts + 31) / 32) * size, size, kThreads, 0, st,
                               (int)rows, a, out) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

fp8q_status fp8q_router_topk_bwd(const void* logits, int64_t tokens, int32_t num_experts, uint32_t flags,
                                 const uint8_t* token_mask, int32_t topk, float scale, const int32_t* topk_idx,
                                 const float* grad_weights, const int32_t* row_id_map, int64_t grad_rows,
                                 const int32_t* counts, float loss_coef, const float* grad_loss, void* grad_logits,
                                 fp8q_stream_t stream) {
  const fp8q_status c = check_router(tokens, num_experts, flags, topk);
  if (c != FP8Q_OK) return c;
  if ((row_id_map && !grad_weights) || grad_rows < 0 || grad_rows > kMaxInt32) return FP8Q_ERR_ARG;
  if (tokens == 0) return FP8Q_OK;
  if (!logits || !grad_logits || (grad_weights && !topk_idx) || (grad_loss && !counts)) return FP8Q_ERR_NULL;
  if (!aligned_to(logits, 16) || !aligned_to(grad_logits, 16) || !aligned_to(topk_idx, 4) ||
      !aligned_to(grad_weights, 4) || !aligned_to(row_id_map, 4) || !aligned_to(counts, 4) || !aligned_to(grad_loss, 4))
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (device_info(&dev) != FP8Q_OK) return FP8Q_ERR_CUDA;
  const RouterArgs a = {tokens, num_experts, topk, (flags & FP8Q_ROUTER_RENORM) != 0, false, scale};
  const BwdPtrs p = {token_mask, topk_idx, grad_weights, row_id_map, grad_rows, counts, loss_coef, grad_loss};
  const bool sigmoid = (flags & FP8Q_ROUTER_SIGMOID) != 0;
  const cudaError_t rc = (flags & FP8Q_ROUTER_BF16)
                             ? launch_bwd(sigmoid, static_cast<const uint16_t*>(logits), a, p,
                                          static_cast<uint16_t*>(grad_logits), dev.status, to_stream(stream))
                             : launch_bwd(sigmoid, static_cast<const float*>(logits), a, p,
                                          static_cast<float*>(grad_logits), dev.status, to_stream(stream));
  return rc == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA;
}

fp8q_status fp8q_permute_row_weights(const float* weights, const int32_t* row_id_map, int64_t pairs, int64_t rows,
                                     float* row_weights, fp8q_stream_t stream) {
  if (pairs < 0 || pairs > kMaxInt32 || rows < 0 || rows > kMaxInt32) return FP8Q_ERR_SHAPE;
  if ((rows > 0 && !row_weights) || (pairs > 0 && (!weights || !row_id_map))) return FP8Q_ERR_NULL;
  if (!aligned_to(weights, 4) || !aligned_to(row_id_map, 4) || !aligned_to(row_weights, 4)) return FP8Q_ERR_ALIGN;
  if (rows == 0 && pairs == 0) return FP8Q_OK;
  DeviceInfo dev;
  if (device_info(&dev) != FP8Q_OK) return FP8Q_ERR_CUDA;
  if (rows > 0 && launch_after(zero_rows_kernel, dim3((unsigned)((rows + 255) / 256)), 256, 0, to_stream(stream),
                               row_weights, rows) != cudaSuccess)
    return FP8Q_ERR_CUDA;
  if (pairs == 0) return FP8Q_OK;
  return launch_after(scatter_weights_kernel, dim3((unsigned)((pairs + 255) / 256)), 256, 0, to_stream(stream), weights,
                      row_id_map, pairs, rows, row_weights, dev.status) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

}  // extern "C"
