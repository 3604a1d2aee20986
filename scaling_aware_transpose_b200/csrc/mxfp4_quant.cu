// mxfp4_quant.cu — BF16 rows -> MXFP4 (see mxfp4.cuh), and the same fused with the MoE
// permute, for the products of mxfp4_matmul.cu.
//
// Two lanes per 32-element tile, 16 elements (two 16-byte loads) each: a tile's amax takes
// one shuffle, and eight lanes hold a 128-element unit whose four scale bytes leave as one
// word of the tiled layout.  2 B are read and 0.53 B written per element: bound by HBM (8192
// x 7168: 24.6 us, 6.05 TB/s; 65536 rows: 6.6 TB/s; 4096 x 7168 to 8 of 32 experts: 44 us, of
// which the routing kernels take 8).
#include <algorithm>

#include "abi_checks.h"
#include "launch.h"
#include "mxfp4.cuh"
#include "permute_common.cuh"

namespace fp8q {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;  // 128-element units per eight lanes

struct Unit {
  uint2 codes;     // this lane's 16 codes
  uint32_t scales; // the unit's four scale bytes (in every lane of the eight)
};

// Lane `sub` of eight holds elements 16 sub .. 16 sub + 15 of the unit.
__device__ __forceinline__ Unit quantize_unit(const uint4& a, const uint4& b, int sub) {
  uint32_t m = maxabs_bf16x2(maxabs_bf16x2(maxabs_bf16x2(a.x, a.y), maxabs_bf16x2(a.z, a.w)),
                             maxabs_bf16x2(maxabs_bf16x2(b.x, b.y), maxabs_bf16x2(b.z, b.w)));
  m = maxabs_bf16x2(m, __byte_perm(m, 0u, 0x1032)) & 0x7FFFu;
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  const int e = mxfp4_tile_exponent(m);
  const float s = exp2_neg(e);
  Unit u;
  u.codes = make_uint2(encode8_e2m1(a, s), encode8_e2m1(b, s));
  u.scales = (uint32_t)(e + 127) << (8 * (sub >> 1));
  u.scales |= __shfl_xor_sync(0xFFFFFFFFu, u.scales, 2);
  u.scales |= __shfl_xor_sync(0xFFFFFFFFu, u.scales, 4);
  return u;
}

// Row of unit u and its position in the row; 32-bit where every unit fits.
__device__ __forceinline__ void split_unit(int64_t u, int k128, bool small, int64_t& row, int64_t& c4) {
  row = small ? (int64_t)((uint32_t)u / (uint32_t)k128) : u / k128;
  c4 = u - row * k128;
}

// Rows up to the next multiple of 128 get scale bytes (127) and no codes.
__global__ void __launch_bounds__(kThreads) quantize_mxfp4_kernel(const uint4* __restrict__ x, int64_t rows,
                                                                  int k128, int64_t n_units, uint2* __restrict__ q,
                                                                  uint8_t* __restrict__ sf) {
  pdl_wait_for(x);
  pdl_trigger();
  const int sub = threadIdx.x & 7;
  const int64_t first = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 3;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 8);
  uint4 a[kUnits], b[kUnits];
  const int64_t live = rows * k128;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = first + i * step;
    a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (u < live) {
      a[i] = ld_stream(x + u * 16 + 2 * sub);
      b[i] = ld_stream(x + u * 16 + 2 * sub + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = first + i * step;
    const Unit v = quantize_unit(a[i], b[i], sub);
    if (u < live) q[u * 8 + sub] = v.codes;
    if (u < n_units && sub == 0) {
      int64_t r, c4;
      split_unit(u, k128, (n_units >> 32) == 0, r, c4);
      *reinterpret_cast<uint32_t*>(sf + sf_word_offset(r, c4, k128)) = v.scales;
    }
  }
}

// The first of a thread's units; its others follow in steps of four, a warp's neighbours.
__device__ __forceinline__ int64_t first_unit() {
  return (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * (4 * kUnits) + ((threadIdx.x & 31) >> 3);
}
__device__ __forceinline__ void quantize_units(const uint4* __restrict__ x, int64_t n_units, int64_t first, Unit (&v)[kUnits]) {
  const int sub = threadIdx.x & 7;
  uint4 a[kUnits], b[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = first + 4 * i;
    a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
    if (u < n_units) {
      a[i] = ld_stream(x + u * 16 + 2 * sub);
      b[i] = ld_stream(x + u * 16 + 2 * sub + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) v[i] = quantize_unit(a[i], b[i], sub);
}
// Units to their tokens' rows: rows[token * topk + slot], in global or shared memory.
__device__ __forceinline__ void store_units(const Unit (&v)[kUnits], int64_t n_units, int64_t first, int k128, int topk,
                                            const int32_t* rows, int64_t max_rows, uint2* __restrict__ q,
                                            uint8_t* __restrict__ sf) {
  const int sub = threadIdx.x & 7;
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = first + 4 * i;
    int64_t t, c4;
    split_unit(u, k128, (n_units >> 32) == 0, t, c4);
    // Eight destinations at a time: lane `sub` reads one's row, stores its scales and hands the
    // row to the other lanes, which all store codes.
    for (int k0 = 0; k0 < topk; k0 += 8) {
      int32_t mine = -1;
      if (u < n_units && k0 + sub < topk) {
        const int32_t r = rows[t * topk + k0 + sub];
        if (r >= 0 && r < max_rows) {  // (never out of range for a consistent routing)
          mine = r;
          *reinterpret_cast<uint32_t*>(sf + sf_word_offset(r, c4, k128)) = v[i].scales;
        }
      }
      const int n = min(8, topk - k0);
      for (int k = 0; k < n; ++k) {
        const int32_t r = __shfl_sync(0xFFFFFFFFu, mine, k, 8);
        if (r >= 0) q[((int64_t)r * k128 + c4) * 8 + sub] = v[i].codes;
      }
    }
  }
}

// Rows start .. end - 1: codes 0, scale bytes 127.
__device__ __forceinline__ void pad_rows_mxfp4(int64_t start, int64_t end, int k128, uint2* __restrict__ q,
                                               uint8_t* __restrict__ sf) {
  if (start < 0 || start >= end) return;
  for (int64_t i = threadIdx.x; i < (end - start) * k128 * 8; i += kThreads) q[start * k128 * 8 + i] = make_uint2(0u, 0u);
  for (int64_t i = threadIdx.x; i < (end - start) * k128; i += kThreads) {
    const int64_t r = i / k128;
    *reinterpret_cast<uint32_t*>(sf + sf_word_offset(start + r, i - r * k128, k128)) = 0x7F7F7F7Fu;
  }
}

// The permute's payload: each unit is quantized once and written to the token's top-k
// destination rows; the trailing CTAs fill the padding rows (codes 0, scale bytes 127).
__global__ void __launch_bounds__(kThreads) scatter_mxfp4_kernel(const uint4* __restrict__ x, int64_t tokens, int k128,
                                                                 const int32_t* __restrict__ row_id_map, int topk,
                                                                 uint2* __restrict__ q, uint8_t* __restrict__ sf,
                                                                 int64_t scatter_ctas, int pad_slots,
                                                                 const int32_t* __restrict__ offsets,
                                                                 const int32_t* __restrict__ totals,
                                                                 int64_t max_rows) {
  if ((int64_t)blockIdx.x >= scatter_ctas) {
    pdl_wait_for(offsets, totals);
    const int64_t c = (int64_t)blockIdx.x - scatter_ctas;
    const int e = (int)(c / pad_slots);
    const int64_t start = (int64_t)offsets[e] + totals[e] + (c - (int64_t)e * pad_slots) * kPadRowsPerCta;
    const int64_t end = min(min(start + kPadRowsPerCta, (int64_t)offsets[e + 1]), max_rows);
    pad_rows_mxfp4(start, end, k128, q, sf);
    return;
  }
  const int64_t n_units = tokens * k128, first = first_unit();
  Unit v[kUnits];
  quantize_units(x, n_units, first, v);
  pdl_wait_for(row_id_map);  // the row ids: everything above overlaps the routing
  store_units(v, n_units, first, k128, topk, row_id_map, max_rows, q, sf);
}

// The whole permute in one launch, for few pairs: every CTA ranks all of them (a warp takes 128,
// counts its experts, and ranks them from the experts' offsets on, as the routing kernels do:
// stable in (token, slot) order) while its part of x is on its way, then stores its units or
// its padding rows (148 CTAs share those: 592 took 10.6 us for the first size below).  The first
// CTA stores the offsets and the row ids.  On the GPU and as a call from Python: one token of 7168
// to 8 of 32 experts 7.0 / 8.2 us against 8.6 / 11.6 by three launches, 512 tokens of 2048 to 2 of
// 8 5.0 / 8.2 against 6.0 / 11.5.  With 256 experts ranking costs as much as the launches: 1024
// tokens of 2048 took 21.3 us against 20.4.
constexpr int kSmallPairs = 1024, kSmallExperts = 128, kSmallWarps = kThreads / 32;
constexpr int kSmallPadCtas = 148;
inline size_t small_smem(int E) { return ((size_t)(kSmallWarps + 2) * E + 1) * sizeof(int32_t); }
__global__ void __launch_bounds__(kThreads) permute_small_mxfp4_kernel(
    const uint4* __restrict__ x, int64_t tokens, int k128, const int32_t* __restrict__ idx, int topk, int E, int align,
    uint2* __restrict__ q, uint8_t* __restrict__ sf, int64_t scatter_ctas, int pad_slots, int32_t* __restrict__ offsets,
    int32_t* __restrict__ row_id_map, int64_t max_rows, int* status) {
  extern __shared__ int32_t sh[];  // counts [warp][expert] | totals [expert] | offsets [expert + 1]
  __shared__ int32_t rows[kSmallPairs];
  int32_t *s_tot = sh + kSmallWarps * E, *s_off = s_tot + E;
  pdl_wait_for(x, idx);
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int pairs = (int)tokens * topk;
  constexpr int kPer = kSmallPairs / kThreads;
  int32_t ids[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = (w * kPer + i) * 32 + lane;
    ids[i] = p < pairs ? ld_g(idx + p) : -1;
  }
  const bool payload = (int64_t)blockIdx.x < scatter_ctas;
  const int64_t n_units = tokens * k128, first = first_unit();
  Unit v[kUnits];
  if (payload) quantize_units(x, n_units, first, v);
  int32_t* mine = sh + w * E;
  for (int e = tid; e < kSmallWarps * E; e += kThreads) sh[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = (w * kPer + i) * 32 + lane;
    const bool ok = ids[i] >= 0 && ids[i] < E;
    if (p < pairs && !ok && blockIdx.x == 0) record_status(status, FP8Q_ERR_DEVICE);
    const unsigned same = __match_any_sync(0xFFFFFFFFu, ok ? ids[i] : -1 - lane);
    if (ok && lane == __ffs(same) - 1) mine[ids[i]] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = tid; e < E; e += kThreads) {
    int32_t t = 0;
#pragma unroll
    for (int i = 0; i < kSmallWarps; ++i) t += sh[i * E + e];
    s_tot[e] = t;
  }
  __syncthreads();
  if (w == 0) {
    int32_t run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int32_t padded = e0 + lane < E ? (s_tot[e0 + lane] + align - 1) / align * align : 0;
      int32_t incl = padded;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += u;
      }
      if (e0 + lane < E) s_off[e0 + lane] = run + incl - padded;
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) s_off[E] = run;
  }
  __syncthreads();
  if (!payload) {
    for (int c = blockIdx.x - (int)scatter_ctas; c < E * pad_slots; c += gridDim.x - (int)scatter_ctas) {
      const int e = c / pad_slots;
      const int64_t start = (int64_t)s_off[e] + s_tot[e] + (c - e * pad_slots) * kPadRowsPerCta;
      pad_rows_mxfp4(start, min(min(start + kPadRowsPerCta, (int64_t)s_off[e + 1]), max_rows), k128, q, sf);
    }
    return;
  }
  for (int e = tid; e < E; e += kThreads) {
    int32_t r = s_off[e];
#pragma unroll
    for (int i = 0; i < kSmallWarps; ++i) {
      const int32_t n = sh[i * E + e];
      sh[i * E + e] = r;
      r += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = (w * kPer + i) * 32 + lane;
    const bool ok = ids[i] >= 0 && ids[i] < E;
    const unsigned same = __match_any_sync(0xFFFFFFFFu, ok ? ids[i] : -1 - lane);
    const int32_t base = ok ? mine[ids[i]] : 0;
    __syncwarp();
    const int32_t r = ok ? base + __popc(same & ((1u << lane) - 1u)) : -1;
    if (ok && lane == __ffs(same) - 1) mine[ids[i]] = base + __popc(same);
    rows[p] = r;
    if (blockIdx.x == 0 && p < pairs) row_id_map[p] = r;
    __syncwarp();
  }
  if (blockIdx.x == 0)
    for (int e = tid; e <= E; e += kThreads) offsets[e] = s_off[e];
  __syncthreads();
  store_units(v, n_units, first, k128, topk, rows, max_rows, q, sf);
}

// A launch that waits for the kernel before it to end.
template <typename... KArgs, typename... Args>
cudaError_t launch_plain(void (*kernel)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" {

size_t fp8q_mxfp4_sf_bytes(int64_t rows, int64_t k) {
  if (rows <= 0 || k <= 0) return 0;
  return (size_t)((rows + 127) / 128) * (size_t)((k + 127) / 128) * kSfTileBytes;
}

fp8q_status fp8q_quantize_rowwise_mxfp4(const void* x, int64_t rows, int64_t cols, uint8_t* q, uint8_t* sf,
                                        fp8q_stream_t stream) {
  if (rows < 0 || cols < 0 || cols % 128 || rows > kMaxInt32 || cols > kMaxInt32) return FP8Q_ERR_SHAPE;
  if (rows == 0 || cols == 0) return FP8Q_OK;
  if (!x || !q || !sf) return FP8Q_ERR_NULL;
  if (!aligned_to(x, 16) || !aligned_to(q, 16) || !aligned_to(sf, 16)) return FP8Q_ERR_ALIGN;
  const int k128 = (int)(cols / 128);
  const int64_t n_units = (rows + 127) / 128 * 128 * k128;
  const int64_t ctas = (n_units + kUnits * (kThreads / 8) - 1) / (kUnits * (kThreads / 8));
  if (ctas > kMaxInt32) return FP8Q_ERR_SHAPE;
  return launch_after(quantize_mxfp4_kernel, dim3((unsigned)ctas), kThreads, 0, to_stream(stream),
                      static_cast<const uint4*>(x), rows, k128, n_units, reinterpret_cast<uint2*>(q), sf) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

fp8q_status fp8q_permute_pad_mxfp4(const void* x, int64_t tokens, int64_t hidden, const int32_t* topk_idx,
                                   int32_t topk, int32_t num_experts, int32_t align, uint8_t* q, uint8_t* sf,
                                   int64_t max_out_rows, int32_t* expert_offsets, int32_t* row_id_map, void* workspace,
                                   size_t workspace_bytes, fp8q_stream_t stream) {
  if (tokens < 0 || hidden < 0 || hidden % 128 || hidden > kMaxInt32) return FP8Q_ERR_SHAPE;
  if (topk < 1 || topk > 64 || num_experts < 1 || num_experts > kMaxExperts || align < 1 || align > 4096)
    return FP8Q_ERR_ARG;
  if (tokens > kMaxInt32 / topk) return FP8Q_ERR_SHAPE;
  if (max_out_rows < tokens * topk + (int64_t)num_experts * (align - 1) || max_out_rows > kMaxInt32) return FP8Q_ERR_ARG;
  if (!expert_offsets) return FP8Q_ERR_NULL;
  if (!aligned_to(expert_offsets, 4)) return FP8Q_ERR_ALIGN;
  cudaStream_t st = to_stream(stream);
  if (tokens > 0) {
    if (!topk_idx || !row_id_map || !workspace) return FP8Q_ERR_NULL;
    if (!aligned_to(workspace, 16) || !aligned_to(topk_idx, 4) || !aligned_to(row_id_map, 4)) return FP8Q_ERR_ALIGN;
    if (workspace_bytes < fp8q_permute_workspace_bytes(tokens, topk, num_experts)) return FP8Q_ERR_ARG;
    if (hidden > 0) {
      if (!x || !q || !sf) return FP8Q_ERR_NULL;
      if (!aligned_to(x, 16) || !aligned_to(q, 16) || !aligned_to(sf, 16)) return FP8Q_ERR_ALIGN;
    }
  }
  DeviceInfo dev;
  if (device_info(&dev) != FP8Q_OK) return FP8Q_ERR_CUDA;
  if (tokens == 0)
    return cudaMemsetAsync(expert_offsets, 0, (size_t)(num_experts + 1) * sizeof(int32_t), st) == cudaSuccess
               ? FP8Q_OK
               : FP8Q_ERR_CUDA;
  const int k128 = (int)(hidden / 128);
  const int64_t n_units = tokens * k128;
  const int64_t per = (kThreads / 32) * 4 * kUnits;
  const int64_t scatter_ctas = (n_units + per - 1) / per;
  const int pad_slots = (align - 1 + kPadRowsPerCta - 1) / kPadRowsPerCta;  // 0 when align == 1
  const int64_t ctas = scatter_ctas + (int64_t)num_experts * pad_slots;
  if (ctas > kMaxInt32) return FP8Q_ERR_SHAPE;
  const int64_t pad_ctas = std::min<int64_t>((int64_t)num_experts * pad_slots, kSmallPadCtas);
  if (hidden > 0 && tokens * topk <= kSmallPairs && num_experts <= kSmallExperts)
    // Launched without the dependent-launch attribute: with it the CTAs crowd onto the SMs that
    // a small product before it leaves free (189 tokens through 8 experts of 1920x2560, permute
    // and product by turns: 22.1 us a pair with it, 14.2 without).
    return launch_plain(permute_small_mxfp4_kernel, dim3((unsigned)(scatter_ctas + pad_ctas)), kThreads,
                        small_smem(num_experts), st, static_cast<const uint4*>(x), tokens, k128, topk_idx, (int)topk,
                        (int)num_experts, (int)align, reinterpret_cast<uint2*>(q), sf, scatter_ctas, pad_slots,
                        expert_offsets, row_id_map, max_out_rows, dev.status) == cudaSuccess
               ? FP8Q_OK
               : FP8Q_ERR_CUDA;
  const fp8q_status rs =
      route_pairs(dev, tokens, topk_idx, topk, num_experts, align, false, expert_offsets, row_id_map, workspace, st);
  if (rs != FP8Q_OK || hidden == 0) return rs;
  const int32_t* totals = route_totals(workspace, tokens, topk, num_experts);
  return launch_after(scatter_mxfp4_kernel, dim3((unsigned)ctas), kThreads, 0, st, static_cast<const uint4*>(x), tokens,
                      k128, (const int32_t*)row_id_map, (int)topk, reinterpret_cast<uint2*>(q), sf, scatter_ctas,
                      pad_slots, (const int32_t*)expert_offsets, totals, max_out_rows) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

}  // extern "C"
