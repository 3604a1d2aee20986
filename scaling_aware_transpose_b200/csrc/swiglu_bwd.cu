// swiglu_bwd.cu — backward of the SwiGLU from 8-bit checkpoints of gate and up.
//
// The forward (fp8q_swiglu_quant_stash) keeps g and u as E4M3 codes with a power-of-two
// scale per 1x128 tile instead of BF16.  With s = 1 / (1 + exp(-g)), the row's factor w and
// the incoming gradient dy of y = g * s * u * w:
//   d gate = dy * w * u * s * (1 + g * (1 - s))      d up = dy * w * g * s
//   d w    = sum over the row of dy * g * s * u      y    = g * s * u * w (recomputed)
// The gradients leave as BF16, or as the row-wise E4M3 pairs that the FP8 products and the
// direct transpose take, with y in the same form on request (the products' weight gradient
// needs it, so the forward need not keep it).
//
// Eight lanes per 1x128 tile, 16 elements each (one 16-byte load of either code, two of dy).
// A CTA holds whole rows: 32 / tiles rows of up to 32 tiles, or one row in steps of 32
// tiles, so that d w is summed inside the CTA in a fixed order.  Per element 4 B are read
// and 4 B (BF16) or 2 to 3 B (E4M3) written: the kernel is bound by HBM.
#include "abi_checks.h"
#include "common.cuh"
#include "launch.h"

namespace fp8q {
namespace {

constexpr int kTilesPerCta = 32;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct BwdIn {
  const uint8_t *gq, *gsf, *uq, *usf;
  const uint16_t* dy;
  const float* w;  // row weights or NULL
};
struct BwdOut {
  uint16_t *dg, *du;                            // BF16 form
  uint8_t *dgq, *dgsf, *duq, *dusf, *yq, *ysf;  // E4M3 form; yq/ysf may be NULL
  float* dw;                                    // or NULL
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four codes -> fp32, before the scale.
__device__ __forceinline__ void decode4(uint32_t c, float* v) {
  const uint32_t lo = cvt_f16x2_e4m3x2(c), hi = cvt_f16x2_e4m3x2(c >> 16);
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[0]), "=f"(v[1]) : "r"(lo));
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(v[2]), "=f"(v[3]) : "r"(hi));
}
// 2^(byte - 127); byte 0 is 2^-127, a subnormal.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Row-wise quantization of a tile's eight lanes x 16 values.
__device__ __forceinline__ void quantize_store(float (&v)[16], uint8_t* q, uint8_t* sf, int64_t at, int64_t tile,
                                               int sub, bool live) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
  const int e = tile_exponent(amax);
  const float s = exp2_neg(e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = cvt_e4m3x2_f32(v[4 * i] * s, v[4 * i + 1] * s) | (cvt_e4m3x2_f32(v[4 * i + 2] * s, v[4 * i + 3] * s) << 16);
  if (live) {
    *reinterpret_cast<uint4*>(q + at) = make_uint4(c[0], c[1], c[2], c[3]);
    if (sub == 0) sf[tile] = (uint8_t)(e + 127);
  }
}

template <bool Fp8>
__global__ void __launch_bounds__(256) swiglu_bwd_kernel(BwdIn in, int64_t rows, int tiles, int rows_per_cta,
                                                         BwdOut out) {
  __shared__ float part[kTilesPerCta];
  pdl_wait_for(in.gq, in.gsf, in.uq, in.usf, in.dy, in.w);
  pdl_trigger();
  const int sub = threadIdx.x & 7, slot = threadIdx.x >> 3;
  const int width = min(tiles, kTilesPerCta);  // tile slots per row
  const int rl = slot / width;                 // row within the CTA (>= rows_per_cta: idle lanes)
  const int64_t row = (int64_t)blockIdx.x * rows_per_cta + rl;
  const bool row_ok = rl < rows_per_cta && row < rows;
  const float w = row_ok && in.w != nullptr ? ld_g(in.w + row) : 1.0f;
  float sum = 0.0f;
  for (int t0 = 0; t0 < tiles; t0 += kTilesPerCta) {  // one step unless a row has more than 32 tiles
    const int t = t0 + slot - rl * width;
    const bool live = row_ok && t < tiles;
    const int64_t tile = row * tiles + t;
    const int64_t at = tile * 128 + sub * 16;
    uint4 gc = make_uint4(0u, 0u, 0u, 0u), uc = gc, d0 = gc, d1 = gc;
    uint32_t gs = 127, us = 127;
    if (live) {
      gc = ld_stream(reinterpret_cast<const uint4*>(in.gq + at));
      uc = ld_stream(reinterpret_cast<const uint4*>(in.uq + at));
      d0 = ld_stream(reinterpret_cast<const uint4*>(in.dy + at));
      d1 = ld_stream(reinterpret_cast<const uint4*>(in.dy + at + 8));
      gs = ld_g(in.gsf + tile);
      us = ld_g(in.usf + tile);
    }
    const float sg = scale_of(gs), su = scale_of(us);
    const uint32_t gw[4] = {gc.x, gc.y, gc.z, gc.w}, uw[4] = {uc.x, uc.y, uc.z, uc.w};
    const uint32_t dw[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
    float dg[16], du[16], y[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float g[4], u[4];
      decode4(gw[i], g);
      decode4(uw[i], u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = 4 * i + j;
        const float dyk = __uint_as_float((j & 1) ? dw[k >> 1] & 0xFFFF0000u : dw[k >> 1] << 16);
        const float gv = g[j] * sg, uv = u[j] * su;
        // exp(-g) by the hardware base-2 exponential: its argument is off by at most
        // |g| * 2^-24 * 1.5, far below the outputs' 8 bits; for g > -30 or so s itself
        // stays within 2^-22.  exp overflowing to +inf gives s = 0.
        const float s = rcp(1.0f + ex2(gv * -1.44269504f));
        const float act = gv * s;                                    // silu(g)
        const float slope = s * __fmaf_rn(gv, 1.0f - s, 1.0f);       // silu'(g)
        const float dyw = dyk * w;
        dg[k] = (dyw * slope) * uv;  // slope first: it is 0 where u could overflow the product
        du[k] = dyw * act;
        const float yv = act * uv;
        sum = __fmaf_rn(dyk, yv, sum);
        if (Fp8) y[k] = yv * w;
      }
    }
    if (Fp8) {
      quantize_store(dg, out.dgq, out.dgsf, at, tile, sub, live);
      quantize_store(du, out.duq, out.dusf, at, tile, sub, live);
      if (out.yq != nullptr) quantize_store(y, out.yq, out.ysf, at, tile, sub, live);
    } else if (live) {
      uint4 v[4];
      uint32_t* p = reinterpret_cast<uint32_t*>(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = pack_bf16(dg[2 * i], dg[2 * i + 1]);
        p[8 + i] = pack_bf16(du[2 * i], du[2 * i + 1]);
      }
      *reinterpret_cast<uint4*>(out.dg + at) = v[0];
      *reinterpret_cast<uint4*>(out.dg + at + 8) = v[1];
      *reinterpret_cast<uint4*>(out.du + at) = v[2];
      *reinterpret_cast<uint4*>(out.du + at + 8) = v[3];
    }
  }
  if (out.dw == nullptr) return;  // uniform
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, o));
  if (sub == 0 && slot < kTilesPerCta) part[slot] = sum;
  __syncthreads();
  if ((int)threadIdx.x < rows_per_cta) {
    const int64_t r = (int64_t)blockIdx.x * rows_per_cta + threadIdx.x;
    if (r < rows) {
      float s = 0.0f;
      for (int t = 0; t < width; ++t) s += part[threadIdx.x * width + t];
      out.dw[r] = s;
    }
  }
}

template <bool Fp8>
fp8q_status launch_bwd(const BwdIn& in, int64_t rows, int64_t cols, const BwdOut& out, cudaStream_t stream) {
  const int tiles = (int)(cols / 128);
  const int per = tiles >= kTilesPerCta ? 1 : kTilesPerCta / tiles;  // rows per CTA
  const int width = tiles < kTilesPerCta ? tiles : kTilesPerCta;
  const unsigned threads = (unsigned)((per * width * 8 + 31) / 32 * 32);
  const int64_t ctas = (rows + per - 1) / per;
  return launch_after(swiglu_bwd_kernel<Fp8>, dim3((unsigned)ctas), threads, 0, stream, in, rows, tiles, per, out) ==
                 cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

// Checks shared by both forms; 1 (not a status) when there is nothing to do.
int check_in(const BwdIn& in, int64_t rows, int64_t cols, const float* dw) {
  if (rows < 0 || cols < 0 || cols % 128 || rows > kMaxInt32 || cols > kMaxInt32) return FP8Q_ERR_SHAPE;
  if (dw && !in.w) return FP8Q_ERR_ARG;
  if (rows == 0 || cols == 0) return 0;
  if (!in.gq || !in.gsf || !in.uq || !in.usf || !in.dy) return FP8Q_ERR_NULL;
  if (!aligned_to(in.gq, 16) || !aligned_to(in.uq, 16) || !aligned_to(in.dy, 16) || !aligned_to(in.w, 4) ||
      !aligned_to(dw, 4))
    return FP8Q_ERR_ALIGN;
  return 0;
}

// d w of rows without columns.
fp8q_status empty_rows(int64_t rows, float* dw, cudaStream_t stream) {
  if (rows == 0 || dw == nullptr) return FP8Q_OK;
  return cudaMemsetAsync(dw, 0, (size_t)rows * sizeof(float), stream) == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" {

fp8q_status fp8q_swiglu_bwd(const uint8_t* gq, const uint8_t* gsf, const uint8_t* uq, const uint8_t* usf,
                            const float* row_weights, const void* dy, int64_t rows, int64_t cols, void* dgate,
                            void* dup, float* drow_weights, fp8q_stream_t stream) {
  const BwdIn in = {gq, gsf, uq, usf, static_cast<const uint16_t*>(dy), row_weights};
  const int c = check_in(in, rows, cols, drow_weights);
  if (c) return static_cast<fp8q_status>(c);
  if (rows == 0 || cols == 0) return empty_rows(rows, drow_weights, to_stream(stream));
  if (!dgate || !dup) return FP8Q_ERR_NULL;
  if (!aligned_to(dgate, 16) || !aligned_to(dup, 16)) return FP8Q_ERR_ALIGN;
  BwdOut out = {};
  out.dg = static_cast<uint16_t*>(dgate);
  out.du = static_cast<uint16_t*>(dup);
  out.dw = drow_weights;
  return launch_bwd<false>(in, rows, cols, out, to_stream(stream));
}

fp8q_status fp8q_swiglu_bwd_quant(const uint8_t* gq, const uint8_t* gsf, const uint8_t* uq, const uint8_t* usf,
                                  const float* row_weights, const void* dy, int64_t rows, int64_t cols, uint8_t* dgq,
                                  uint8_t* dgsf, uint8_t* duq, uint8_t* dusf, uint8_t* yq, uint8_t* ysf,
                                  float* drow_weights, fp8q_stream_t stream) {
  const BwdIn in = {gq, gsf, uq, usf, static_cast<const uint16_t*>(dy), row_weights};
  const int c = check_in(in, rows, cols, drow_weights);
  if (c) return static_cast<fp8q_status>(c);
  if ((yq == nullptr) != (ysf == nullptr)) return FP8Q_ERR_ARG;
  if (rows == 0 || cols == 0) return empty_rows(rows, drow_weights, to_stream(stream));
  if (!dgq || !dgsf || !duq || !dusf) return FP8Q_ERR_NULL;
  if (!aligned_to(dgq, 16) || !aligned_to(duq, 16) || !aligned_to(yq, 16)) return FP8Q_ERR_ALIGN;
  BwdOut out = {};
  out.dgq = dgq;
  out.dgsf = dgsf;
  out.duq = duq;
  out.dusf = dusf;
  out.yq = yq;
  out.ysf = ysf;
  out.dw = drow_weights;
  return launch_bwd<true>(in, rows, cols, out, to_stream(stream));
}

}  // extern "C"
