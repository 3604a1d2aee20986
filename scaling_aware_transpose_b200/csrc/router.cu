// router.cu — the MoE router in front of the permute: scores, top-k, routing weights,
// per-expert counts and the balance loss, and the gradient of the logits.
//
// Per token with logits l[e]:
//   softmax   p_e = exp(l_e - max l) / sum exp(l - max l)
//   sigmoid   p_e = 1 / (1 + exp(-l_e))
//   ids       the k experts of the largest l_e (softmax, and sigmoid without a bias: both
//             are increasing in l), or of the largest p_e + bias_e; ties to the lowest id
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
// One warp per token, the token's logits in registers (expert e = lane + 32 i).  Each pick
// is a warp maximum of the order-preserving integer image of the key.  All sums are fp32
// in a fixed order (per lane over the warp's tokens, over the CTA's warps, then over CTAs
// in double), the counts are integers: nothing depends on the order of atomics.
#include <cfloat>

#include "abi_checks.h"
#include "common.cuh"
#include "launch.h"

namespace fp8q {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxBlocks = 592;  // a fixed cap, so that the order of the sums is the same on every device
constexpr int kRouterMaxExperts = 1024;
constexpr int kRouterMaxTopk = 64;
constexpr float kEps = 1e-20f;
constexpr unsigned kAll = 0xFFFFFFFFu;

enum Mode { kSoftmax = 0, kSigmoid = 1, kSigmoidBias = 2 };

__device__ __forceinline__ float load_logit(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_logit(const uint16_t* p, int64_t i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}
__device__ __forceinline__ void store_grad(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, int64_t i, float v) {
  uint16_t r;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
  p[i] = r;
}

// NaN counts as -inf (a padding row may hold anything), +inf as the largest finite value;
// adding +0 turns -0 into +0, so that the two tie.
__device__ __forceinline__ float clean(float l) { return l != l ? -INFINITY : fminf(l + 0.0f, FLT_MAX); }

// fp32 -> uint32 with the same order; every value but NaN maps above 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
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

// p = sigmoid(l) and q = 1 - p without cancellation on either side.
__device__ __forceinline__ void sigmoid2(float l, float& p, float& q) {
  const float t = expf(-fabsf(l));
  const float r = __frcp_rn(1.0f + t);
  const float s = t * r;
  p = l >= 0.0f ? r : s;
  q = l >= 0.0f ? s : r;
}

struct RouterArgs {
  int64_t tokens;
  int E, topk;
  bool renorm, stats;
  float scale;
};

// ------------------------------------------------------------------ forward
// Workspace: [0] a counter for the finishing kernel, then per CTA E sums (fp32), then per
// CTA E counts (int32), from byte 16 on.
template <int VPL, int MODE, typename T>
__global__ void __launch_bounds__(kThreads) router_kernel(const T* __restrict__ logits, const float* __restrict__ bias,
                                                          const uint8_t* __restrict__ mask, RouterArgs a,
                                                          int32_t* __restrict__ topk_idx, float* __restrict__ weights,
                                                          uint32_t* __restrict__ ws) {
  __shared__ float sums_sh[kRouterMaxExperts];
  __shared__ int counts_sh[kRouterMaxExperts];
  pdl_wait_for(logits, bias, mask);
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int E = a.E, K = a.topk;
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
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + wid; t < a.tokens; t += stride) {
    const bool live = mask == nullptr || mask[t] != 0;
    uint32_t key[VPL];
    uint32_t key_lo[MODE == kSigmoidBias ? VPL : 1];
    float val[VPL];  // the logit, then its share of the balance statistics
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      val[i] = -INFINITY;
      key[i] = 0u;
      if (MODE == kSigmoidBias) key_lo[i] = 0u;
      if (e < E) {
        val[i] = clean(load_logit(logits, t * E + e));
        if (MODE == kSigmoidBias) {
          // Neighbouring scores can be closer than an fp32 sum resolves: the score is
          // formed in double and compared as its fp32 value and the remainder.
          const double s = 1.0 / (1.0 + exp(-(double)val[i])) + (double)bias[e];
          const float hi = (float)s;
          key[i] = max(order_key(hi + 0.0f), 1u);
          key_lo[i] = order_key((float)(s - (double)hi) + 0.0f);
        } else {
          key[i] = order_key(val[i]);
        }
      }
    }
    // ---- the k picks: lane s (and 32 + s) keeps pick s
    int pick_e[2] = {0, 0};
    float pick_v[2] = {-INFINITY, -INFINITY};
    float top = -INFINITY;
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
        if (key[i] == m && (MODE != kSigmoidBias || key_lo[i] == m_lo)) e = lane + 32 * i;
      e = __reduce_min_sync(kAll, e);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e == (uint32_t)(lane + 32 * i)) key[i] = 0u;
      if (s == 0 && MODE == kSoftmax) top = from_key(m);
      if (lane == (s & 31)) {
        if (s < 32) {
          pick_e[0] = (int)e;
          pick_v[0] = from_key(m);
        } else {
          pick_e[1] = (int)e;
          pick_v[1] = from_key(m);
        }
      }
    }
    // ---- probabilities
    float z_inv = 1.0f;  // softmax: 1 / sum exp
    if (MODE == kSoftmax) {
      if (a.stats || !a.renorm) {
        float z = 0.0f;
        const float base = top == -INFINITY ? 0.0f : top;  // a row of -inf has no probability at all
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          val[i] = expf(val[i] - base);
          z += val[i];
        }
        z = warp_sum(z);
        z_inv = z > 0.0f ? __frcp_rn(z) : 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) val[i] *= z_inv;
      }
    } else if (a.stats) {
      float z = 0.0f, q;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        sigmoid2(val[i], val[i], q);
        z += val[i];
      }
      z = warp_sum(z) + kEps;
      z_inv = __frcp_rn(z);
#pragma unroll
      for (int i = 0; i < VPL; ++i) val[i] *= z_inv;
    }
    if (a.stats && live) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] += val[i];
    }
    float w[2], total = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool on = lane + 32 * h < K;
      w[h] = 0.0f;
      if (on) {
        if (MODE == kSoftmax) {
          w[h] = top == -INFINITY ? 0.0f : expf(pick_v[h] - top);
          if (!a.renorm) w[h] *= z_inv;
        } else {
          float q;
          const float l = MODE == kSigmoidBias ? clean(load_logit(logits, t * E + pick_e[h])) : pick_v[h];
          sigmoid2(l, w[h], q);
        }
      }
      total += w[h];
    }
    // The eps is of the size of the probabilities; exp(l - max) exceeds them by the factor
    // z >= 1, for which 1e-20 is as far below fp32 resolution.
    const float factor = a.renorm ? a.scale * __frcp_rn(warp_sum(total) + kEps) : a.scale;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int s = lane + 32 * h;
      if (s < K) {
        topk_idx[t * K + s] = pick_e[h];
        weights[t * K + s] = live ? w[h] * factor : 0.0f;
        if (a.stats && live) atomicAdd(&counts_sh[pick_e[h]], 1);
      }
    }
  }
  if (!a.stats) return;
  for (int w = 0; w < kWarps; ++w) {  // the warps' sums in order
    if (wid == w) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < E) sums_sh[lane + 32 * i] += acc[i];
    }
    __syncthreads();
  }
  float* part = reinterpret_cast<float*>(ws + 4);
  int32_t* part_n = reinterpret_cast<int32_t*>(part + (int64_t)gridDim.x * E);
  for (int e = threadIdx.x; e < E; e += kThreads) {
    part[(int64_t)blockIdx.x * E + e] = sums_sh[e];
    part_n[(int64_t)blockIdx.x * E + e] = counts_sh[e];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) ws[0] = 0u;
}

// Sums the CTAs' partial results: a CTA per 32 experts, a warp per every 32nd CTA's row;
// the last CTA to finish (the counter was zeroed by the kernel before) forms the loss.
__global__ void __launch_bounds__(1024) router_finish_kernel(int blocks, int E, int topk, float loss_coef,
                                                             uint32_t* __restrict__ ws, int32_t* __restrict__ counts,
                                                             float* __restrict__ prob_sums, float* __restrict__ loss) {
  __shared__ double sum_sh[32][33];
  __shared__ int cnt_sh[32][33];
  __shared__ bool last;
  pdl_wait_for(ws, counts, prob_sums);
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  const float* part = reinterpret_cast<const float*>(ws + 4);
  const int32_t* part_n = reinterpret_cast<const int32_t*>(part + (int64_t)blocks * E);
  double s = 0.0;
  int n = 0;
  if (e < E) {
#pragma unroll 4
    for (int b = wid; b < blocks; b += 32) {
      s += (double)part[(int64_t)b * E + e];
      n += part_n[(int64_t)b * E + e];
    }
  }
  sum_sh[wid][lane] = s;
  cnt_sh[wid][lane] = n;
  __syncthreads();
  if (wid == 0 && e < E) {
    for (int w = 1; w < 32; ++w) {
      s += sum_sh[w][lane];
      n += cnt_sh[w][lane];
    }
    counts[e] = n;
    prob_sums[e] = (float)s;
    __threadfence();
  }
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(ws, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last || wid != 0) return;
  __threadfence();
  double dot = 0.0;
  long long c = 0;
  for (int i = lane; i < E; i += 32) {
    const int32_t ci = __ldcg(counts + i);
    dot += (double)ci * (double)__ldcg(prob_sums + i);
    c += ci;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    dot += __shfl_xor_sync(kAll, dot, o);
    c += __shfl_xor_sync(kAll, c, o);
  }
  if (lane == 0) *loss = c > 0 ? (float)((double)loss_coef * E * topk / ((double)c * (double)c) * dot) : 0.0f;
}

// ------------------------------------------------------------------ backward
template <int VPL, bool SIGMOID, typename T>
__global__ void __launch_bounds__(kThreads) router_bwd_kernel(const T* __restrict__ logits,
                                                              const uint8_t* __restrict__ mask, RouterArgs a,
                                                              const int32_t* __restrict__ topk_idx,
                                                              const float* __restrict__ grad_weights,
                                                              const int32_t* __restrict__ row_id_map, int64_t rows,
                                                              const int32_t* __restrict__ counts, float loss_coef,
                                                              const float* __restrict__ grad_loss,
                                                              T* __restrict__ grad, int* status) {
  extern __shared__ float sh[];  // [E] g_e, then per warp [E]
  __shared__ long long c_sh[kWarps];
  pdl_wait_for(logits, mask, topk_idx, grad_weights, row_id_map, counts, grad_loss);
  pdl_trigger();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int E = a.E, K = a.topk;
  const bool balance = grad_loss != nullptr;
  float* g_sh = sh;
  float* buf = sh + E + wid * E;
  if (balance) {
    long long c = 0;
    for (int e = threadIdx.x; e < E; e += kThreads) c += counts[e];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) c += __shfl_xor_sync(kAll, c, o);
    if (lane == 0) c_sh[wid] = c;
    __syncthreads();
    c = 0;
    for (int w = 0; w < kWarps; ++w) c += c_sh[w];
    const double f = c > 0 ? (double)*grad_loss * (double)loss_coef * E * K / ((double)c * (double)c) : 0.0;
    for (int e = threadIdx.x; e < E; e += kThreads) g_sh[e] = (float)(f * (double)counts[e]);
    __syncthreads();
  }
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + wid; t < a.tokens; t += stride) {
    if (mask != nullptr && mask[t] == 0) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < E) store_grad(grad, t * E + lane + 32 * i, 0.0f);
      continue;
    }
    float p[VPL], q[SIGMOID ? VPL : 1];
    float z = 0.0f;
    if (SIGMOID) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        sigmoid2(e < E ? clean(load_logit(logits, t * E + e)) : -INFINITY, p[i], q[i]);
        z += p[i];
      }
      z = warp_sum(z) + kEps;
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        p[i] = e < E ? clean(load_logit(logits, t * E + e)) : -INFINITY;
        m = fmaxf(m, p[i]);
      }
      m = from_key(__reduce_max_sync(kAll, order_key(m)));
      const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        p[i] = expf(p[i] - base);
        z += p[i];
      }
      z = warp_sum(z);
      const float z_inv = z > 0.0f ? __frcp_rn(z) : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) p[i] *= z_inv;
    }
    float d[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
    if (grad_weights != nullptr) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < E) buf[lane + 32 * i] = p[i];
      __syncwarp();
      int id[2];
      float dw[2], ps[2], total = 0.0f, dot = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int s = lane + 32 * h;
        id[h] = -1;
        dw[h] = ps[h] = 0.0f;
        if (s < K) {
          const int e = topk_idx[t * K + s];
          int64_t at = t * K + s;
          bool ok = e >= 0 && e < E;
          if (row_id_map != nullptr) {
            at = row_id_map[at];
            ok = ok && at >= 0 && at < rows;
          }
          if (ok) {
            id[h] = e;
            dw[h] = grad_weights[at];
            ps[h] = buf[e];
          } else {
            record_status(status, FP8Q_ERR_DEVICE);
          }
        }
        total += ps[h];
        dot += dw[h] * ps[h];
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < E) buf[lane + 32 * i] = 0.0f;
      __syncwarp();
      float inv = 1.0f, mean = 0.0f;
      if (a.renorm) {
        inv = __frcp_rn(warp_sum(total) + kEps);
        mean = warp_sum(dot) * inv;
      }
      // Ids are distinct for a row the router wrote, so the stores do not meet; should a
      // caller repeat one, the slots are added one by one, in slot order.
      bool repeated = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned same = __match_any_sync(kAll, id[h] >= 0 ? id[h] : -1 - lane);
        repeated |= __popc(same) > 1;
      }
      if (K > 32) {
        for (int o = 0; o < 32; ++o) {
          const int other = __shfl_sync(kAll, id[0], o);
          repeated |= id[1] >= 0 && other == id[1];
        }
      }
      if (!__any_sync(kAll, repeated)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (id[h] >= 0) buf[id[h]] = a.scale * inv * (dw[h] - mean);
      } else {
        for (int s = 0; s < K; ++s) {
          if (lane == (s & 31)) {
            const int h = s >> 5;
            const int e = h ? id[1] : id[0];
            const float v = h ? dw[1] : dw[0];
            if (e >= 0) buf[e] += a.scale * inv * (v - mean);
          }
          __syncwarp();
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (lane + 32 * i < E) d[i] = buf[lane + 32 * i];
      __syncwarp();
    }
    if (SIGMOID) {
      if (balance) {
        const float z_inv = __frcp_rn(z);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (lane + 32 * i < E) dot = __fmaf_rn(g_sh[lane + 32 * i], p[i], dot);
        dot = warp_sum(dot) * z_inv;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (lane + 32 * i < E) d[i] = __fmaf_rn(g_sh[lane + 32 * i] - dot, z_inv, d[i]);
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] *= p[i] * q[i];
    } else {
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (balance && lane + 32 * i < E) d[i] += g_sh[lane + 32 * i];
        dot = __fmaf_rn(d[i], p[i], dot);
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] = p[i] * (d[i] - dot);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i < E) store_grad(grad, t * E + lane + 32 * i, d[i]);
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

int router_blocks(int64_t tokens) {
  const int64_t b = (tokens + kWarps - 1) / kWarps;
  return (int)(b < 1 ? 1 : b < kMaxBlocks ? b : kMaxBlocks);
}

template <int VPL, typename T>
cudaError_t launch_fwd(int mode, int blocks, const T* logits, const float* bias, const uint8_t* mask,
                       const RouterArgs& a, int32_t* idx, float* weights, uint32_t* ws, cudaStream_t st) {
  auto k = mode == kSoftmax ? router_kernel<VPL, kSoftmax, T>
                            : mode == kSigmoid ? router_kernel<VPL, kSigmoid, T> : router_kernel<VPL, kSigmoidBias, T>;
  return launch_after(k, dim3((unsigned)blocks), kThreads, 0, st, logits, bias, mask, a, idx, weights, ws);
}

template <typename T>
cudaError_t launch_fwd_for(int mode, int blocks, const void* logits, const float* bias, const uint8_t* mask,
                           const RouterArgs& a, int32_t* idx, float* weights, uint32_t* ws, cudaStream_t st) {
  const T* l = static_cast<const T*>(logits);
  if (a.E <= 32) return launch_fwd<1>(mode, blocks, l, bias, mask, a, idx, weights, ws, st);
  if (a.E <= 64) return launch_fwd<2>(mode, blocks, l, bias, mask, a, idx, weights, ws, st);
  if (a.E <= 128) return launch_fwd<4>(mode, blocks, l, bias, mask, a, idx, weights, ws, st);
  if (a.E <= 256) return launch_fwd<8>(mode, blocks, l, bias, mask, a, idx, weights, ws, st);
  if (a.E <= 512) return launch_fwd<16>(mode, blocks, l, bias, mask, a, idx, weights, ws, st);
  return launch_fwd<32>(mode, blocks, l, bias, mask, a, idx, weights, ws, st);
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

template <int VPL, typename T>
cudaError_t launch_bwd(bool sigmoid, const T* logits, const RouterArgs& a, const BwdPtrs& p, T* grad, int* status,
                       cudaStream_t st) {
  auto k = sigmoid ? router_bwd_kernel<VPL, true, T> : router_bwd_kernel<VPL, false, T>;
  const size_t smem = (size_t)(kWarps + 1) * a.E * sizeof(float);  // at most 36 KB
  return launch_after(k, dim3((unsigned)router_blocks(a.tokens)), kThreads, smem, st, logits, p.mask, a, p.idx, p.gw,
                      p.map, p.rows, p.counts, p.loss_coef, p.grad_loss, grad, status);
}

template <typename T>
cudaError_t launch_bwd_for(bool sigmoid, const void* logits, const RouterArgs& a, const BwdPtrs& p, void* grad,
                           int* status, cudaStream_t st) {
  const T* l = static_cast<const T*>(logits);
  T* g = static_cast<T*>(grad);
  if (a.E <= 32) return launch_bwd<1>(sigmoid, l, a, p, g, status, st);
  if (a.E <= 64) return launch_bwd<2>(sigmoid, l, a, p, g, status, st);
  if (a.E <= 128) return launch_bwd<4>(sigmoid, l, a, p, g, status, st);
  if (a.E <= 256) return launch_bwd<8>(sigmoid, l, a, p, g, status, st);
  if (a.E <= 512) return launch_bwd<16>(sigmoid, l, a, p, g, status, st);
  return launch_bwd<32>(sigmoid, l, a, p, g, status, st);
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
  return 16 + (size_t)router_blocks(tokens) * num_experts * 8;
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
  const RouterArgs a = {tokens, num_experts, topk, (flags & FP8Q_ROUTER_RENORM) != 0, stats, scale};
  const int mode = !(flags & FP8Q_ROUTER_SIGMOID) ? kSoftmax : bias ? kSigmoidBias : kSigmoid;
  const int blocks = router_blocks(tokens);
  uint32_t* ws = stats ? static_cast<uint32_t*>(workspace) : nullptr;
  cudaStream_t st = to_stream(stream);
  const cudaError_t rc =
      (flags & FP8Q_ROUTER_BF16)
          ? launch_fwd_for<uint16_t>(mode, blocks, logits, bias, token_mask, a, topk_idx, weights, ws, st)
          : launch_fwd_for<float>(mode, blocks, logits, bias, token_mask, a, topk_idx, weights, ws, st);
  if (rc != cudaSuccess) return FP8Q_ERR_CUDA;
  if (!stats) return FP8Q_OK;
  return launch_after(router_finish_kernel, dim3((unsigned)((num_experts + 31) / 32)), 1024, 0, st, blocks,
                      (int)num_experts, (int)topk, loss_coef, ws, counts, prob_sums, loss) == cudaSuccess
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
                             ? launch_bwd_for<uint16_t>(sigmoid, logits, a, p, grad_logits, dev.status, to_stream(stream))
                             : launch_bwd_for<float>(sigmoid, logits, a, p, grad_logits, dev.status, to_stream(stream));
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
