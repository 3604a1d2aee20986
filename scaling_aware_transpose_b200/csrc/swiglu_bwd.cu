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
// A warp per row (two or four rows of one or two tiles): eight lanes per 1x128 tile, 16
// elements each, four tiles a pass, the next pass's loads in flight during this one.  d w is
// then a sum over the warp's lanes in a fixed order, and nothing waits for another warp.
// Per element 4 B are read and 4 B (BF16) or 2 to 3 B (E4M3) written.  The BF16 form moves
// them at 6.2 TB/s (86.6 us at [32768, 2048]); the E4M3 form at 4.9 TB/s (95 us), bound by
// the issue of about 35 instructions an element at 20 warps an SM (ncu: 71% of the slots; 96
// registers: fewer spill more, more leave too few warps; when the form took 97 us, eight
// elements a lane took 108 us, staging through shared memory by bulk copies 140 us, one-shot
// CTAs with the loads in front 119 us).
// The codes' scales stay out of the arithmetic (g = sg g', u = su u' with the raw codes' values
// g', u'; the factors sg, su, w meet once per tile):
//   s = 1 / (1 + 2^(g' * (-sg log2 e))),  a = g' s,  slope = s + (a sg)(1 - s),  x = dy u'
//   d gate = x slope (w su),  d up = dy a (w sg),  y = a u' (w sg su),  d w += x a (sg su).
#include <cfloat>

#include "abi_checks.h"
#include "common.cuh"
#include "launch.h"

namespace fp8q {
namespace {

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
// Pairs of fp32, one instruction each.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 make2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2(F2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
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
__device__ __forceinline__ uint32_t pack_bf16(F2 x) {
  float a, b;
  split2(x, a, b);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Two codes (in the low or high half of c) -> fp32, before the scale.
__device__ __forceinline__ F2 decode2(uint32_t c) {
  const uint32_t h = cvt_f16x2_e4m3x2(c);
  float x, y;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(x), "=f"(y) : "r"(h));
  return make2(x, y);
}
// 2^(byte - 127); byte 0 is 2^-127, a subnormal.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}
// tile_exponent of a finite amax >= 0, shorter: adding 0x1FFFFF carries into the exponent
// field exactly when the mantissa exceeds 1.75 (the 0x600000 of the rule), and whatever is
// subnormal lies far below the clamp.
__device__ __forceinline__ int quick_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  return b == 0u ? 0 : max((int)((b + 0x1FFFFFu) >> 23) - 135, -127);
}
// max(|a|, |b|, |c|) in one instruction.
__device__ __forceinline__ float max3abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Row-wise quantization of v * factor over a tile's eight lanes x 16 values: the factor is applied
// to the tile's maximum, which gives e, and as f = factor * 2^-e to the values.
__device__ __forceinline__ float tile_amax(const F2 (&v)[8]) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) split2(v[i], x[2 * i], x[2 * i + 1]);
  return fmaxf(max3abs(max3abs(x[0], x[1], x[2]), max3abs(x[3], x[4], x[5]), max3abs(x[6], x[7], x[8])),
               max3abs(max3abs(x[9], x[10], x[11]), max3abs(x[12], x[13], x[14]), x[15]));
}
__device__ __forceinline__ void store_codes(const F2 (&v)[8], int e, float f, uint8_t* q, uint8_t* sf, int64_t at,
                                            int64_t tile, int sub) {
  const F2 f2 = make2(f, f);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0, a1, b0, b1;
    split2(mul2(v[2 * i], f2), a0, a1);
    split2(mul2(v[2 * i + 1], f2), b0, b1);
    c[i] = __byte_perm(cvt_e4m3x2_f32(a0, a1), cvt_e4m3x2_f32(b0, b1), 0x5410);
  }
  *reinterpret_cast<uint4*>(q + at) = make_uint4(c[0], c[1], c[2], c[3]);
  if (sub == 0) sf[tile] = (uint8_t)(e + 127);
}
// f has to be finite: times a value of 0 it would be a NaN code.  It is not in a tile of nothing
// but tiny values (saturated gates, gradients near the bottom of BF16) under a factor of 2 and
// more.  2^64 of it go to the values then, exactly: f is at most 448 / 2^-149, or factor * 2^127
// where e stopped at -127.  What is beyond fp32 even so (the factor itself, by the scales of the
// largest gates) counts as the largest value.
__device__ __forceinline__ void shift_up(F2 (&v)[8], float factor, int e, float& f) {
  if (fabsf(f) <= FLT_MAX) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], make2(0x1p64f, 0x1p64f));
  f = fminf(fmaxf(factor * 0x1p-64f * exp2_neg(e), -FLT_MAX), FLT_MAX);
}

constexpr int kThreads = 128;

// What eight lanes need of one tile.
struct TileIn {
  uint4 g, u, d0, d1;
  uint32_t gs, us;
};

template <bool Fp8>
__global__ void __launch_bounds__(kThreads, Fp8 ? 5 : 6) swiglu_bwd_kernel(BwdIn in, int64_t rows, int tiles,
                                                                                  int per_warp, BwdOut out) {
  pdl_wait_for(in.gq, in.gsf, in.uq, in.usf, in.dy, in.w);
  pdl_trigger();
  const int lane = threadIdx.x & 31, sub = lane & 7, group = lane >> 3;
  const int lanes = 32 / per_warp, step = 4 / per_warp;  // lanes and tiles of a pass per row
  const int64_t row = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * per_warp + group / step;
  const bool row_ok = row < rows;
  const float w = row_ok && in.w != nullptr ? ld_g(in.w + row) : 1.0f;
  const int64_t tile0 = row * tiles;
  auto load = [&](int t) {
    TileIn v;
    v.g = v.u = v.d0 = v.d1 = make_uint4(0u, 0u, 0u, 0u);
    v.gs = v.us = 127u;
    if (row_ok && t < tiles) {
      const int64_t at = (tile0 + t) * 128 + sub * 16;
      v.g = ld_stream(reinterpret_cast<const uint4*>(in.gq + at));
      v.u = ld_stream(reinterpret_cast<const uint4*>(in.uq + at));
      v.d0 = ld_stream(reinterpret_cast<const uint4*>(in.dy + at));
      v.d1 = ld_stream(reinterpret_cast<const uint4*>(in.dy + at + 8));
      v.gs = ld_g(in.gsf + tile0 + t);
      v.us = ld_g(in.usf + tile0 + t);
    }
    return v;
  };
  float sum = 0.0f;
  TileIn next = load(group % step);
  for (int t0 = 0; t0 < tiles; t0 += step) {
    const int t = t0 + group % step;
    const bool live = row_ok && t < tiles;
    const TileIn v = next;
    if (t0 + step < tiles) next = load(t + step);
    const int64_t tile = tile0 + t;
    const int64_t at = tile * 128 + sub * 16;
    const uint4 gc = v.g, uc = v.u, d0 = v.d0, d1 = v.d1;
    const uint32_t gs = v.gs, us = v.us;
    const float sg = scale_of(gs), su = scale_of(us);
    const uint32_t gw[4] = {gc.x, gc.y, gc.z, gc.w}, uw[4] = {uc.x, uc.y, uc.z, uc.w};
    const uint32_t dw[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
    // exp(-g) by the hardware base-2 exponential: its argument is off by at most |g| * 2^-23,
    // far below the outputs' 8 bits.  An exponential of +inf gives s = 0.
    const F2 k2 = make2(sg * -1.44269504f, sg * -1.44269504f);
    // In the slope: a sg must not overflow where 1 - s is 0.  Above 2^118 (a stays below 2^9) every
    // gate but 0 has s = 0 or 1, and the cap changes nothing else.
    const float sc = fminf(sg, 0x1p118f);
    const F2 sg2 = make2(sc, sc);
    const F2 one = make2(1.0f, 1.0f), minus = make2(-1.0f, -1.0f);
    F2 dg[8], du[8], y[8], dot = make2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const F2 g = decode2(gw[k >> 1] >> (16 * (k & 1))), u = decode2(uw[k >> 1] >> (16 * (k & 1)));
      const F2 d = make2(__uint_as_float(dw[k] << 16), __uint_as_float(dw[k] & 0xFFFF0000u));
      float e0, e1;
      split2(mul2(g, k2), e0, e1);
      split2(add2(make2(ex2(e0), ex2(e1)), one), e0, e1);
      const F2 s = make2(rcp(e0), rcp(e1));
      const F2 act = mul2(g, s);
      const F2 slope = fma2(mul2(act, sg2), fma2(s, minus, one), s);
      const F2 x = mul2(d, u);
      dg[k] = mul2(x, slope);
      du[k] = mul2(d, act);
      dot = fma2(x, act, dot);
      if (Fp8) y[k] = mul2(act, u);
    }
    {
      float a0, a1;
      split2(dot, a0, a1);
      sum = __fmaf_rn((a0 + a1) * sg, su, sum);
    }
    if (Fp8) {
      // The three together: their maxima's shuffles overlap (one after the other 98.4 us, not
      // 95.6), and one test covers the f's.
      float mg = tile_amax(dg), mu = tile_amax(du), my = tile_amax(y);
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) {
        mg = fmaxf(mg, __shfl_xor_sync(kAll, mg, o));
        mu = fmaxf(mu, __shfl_xor_sync(kAll, mu, o));
        my = fmaxf(my, __shfl_xor_sync(kAll, my, o));
      }
      const float cg = w * su, cu = w * sg, cy = w * sg * su;
      const int eg = quick_exponent(mg * fabsf(cg)), eu = quick_exponent(mu * fabsf(cu)), ey = quick_exponent(my * fabsf(cy));
      float fg = cg * exp2_neg(eg), fu = cu * exp2_neg(eu), fy = cy * exp2_neg(ey);
      if (!(max3abs(fg, fu, fy) <= FLT_MAX)) {
        shift_up(dg, cg, eg, fg);
        shift_up(du, cu, eu, fu);
        shift_up(y, cy, ey, fy);
      }
      if (live) {
        store_codes(dg, eg, fg, out.dgq, out.dgsf, at, tile, sub);
        store_codes(du, eu, fu, out.duq, out.dusf, at, tile, sub);
        if (out.yq != nullptr) store_codes(y, ey, fy, out.yq, out.ysf, at, tile, sub);
      }
    } else if (live) {
      const F2 fg = make2(w * su, w * su), fu = make2(w * sg, w * sg);
      uint32_t p[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = pack_bf16(mul2(dg[i], fg));
        p[8 + i] = pack_bf16(mul2(du[i], fu));
      }
      *reinterpret_cast<uint4*>(out.dg + at) = make_uint4(p[0], p[1], p[2], p[3]);
      *reinterpret_cast<uint4*>(out.dg + at + 8) = make_uint4(p[4], p[5], p[6], p[7]);
      *reinterpret_cast<uint4*>(out.du + at) = make_uint4(p[8], p[9], p[10], p[11]);
      *reinterpret_cast<uint4*>(out.du + at + 8) = make_uint4(p[12], p[13], p[14], p[15]);
    }
  }
  if (out.dw == nullptr) return;  // uniform
  for (int o = lanes >> 1; o >= 1; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, o));
  if (row_ok && (lane & (lanes - 1)) == 0) out.dw[row] = sum;
}

template <bool Fp8>
fp8q_status launch_bwd(const BwdIn& in, int64_t rows, int64_t cols, const BwdOut& out, cudaStream_t stream) {
  const int tiles = (int)(cols / 128);
  const int per_warp = tiles == 1 ? 4 : tiles == 2 ? 2 : 1;
  const int64_t per_cta = (int64_t)per_warp * (kThreads / 32);
  return launch_after(swiglu_bwd_kernel<Fp8>, dim3((unsigned)((rows + per_cta - 1) / per_cta)), kThreads, 0, stream, in,
                      rows, tiles, per_warp, out) == cudaSuccess
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
