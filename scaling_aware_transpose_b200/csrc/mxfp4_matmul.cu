// mxfp4_matmul.cu — products of MXFP4 operands on the tensor cores: out = A * B^T, dense or
// over the expert groups that the permute makes.
//
// A [m, k] and B [n, k] hold E2M1 codes with one E8M0 scale per 32 elements along k (see
// mxfp4.cuh).  out[i, j] = sum over k tiles t of 2^(sa + sb) * sum of the 32 code products:
// tcgen05.mma kind::mxf4 applies both scales itself and accumulates in fp32 (products of
// two codes and their scale are exact), so nothing is decoded in registers.
//
// One persistent CTA per SM walks output tiles of 128 rows x BN columns; a pipeline stage
// is 256 elements of k (128-byte rows under the 128-byte swizzle):
//   warp 0   TMA loads of the A and B codes, and bulk copies of their scale tiles, which
//            the quantizers store in the order the tensor core reads;
//   warp 1   per stage: scales shared -> tensor memory (tcgen05.cp), four MMAs of 64
//            elements, and a commit that frees the stage;
//   warps 2-5  the epilogue: tensor memory -> registers -> BF16 -> global.
// The accumulator is double-buffered in tensor memory, so the epilogue of one tile runs
// under the MMAs of the next.  Scale columns in tensor memory belong to the stage, which
// is refilled only after its MMAs have completed.
//
// Every wait is bounded; a role whose wait expires records FP8Q_ERR_TIMEOUT and leaves its
// loop, the others follow, outstanding copies and MMAs are waited for (again bounded) and
// the tensor memory is freed.
#include <cuda.h>

#include <mutex>

#include "abi_checks.h"
#include "launch.h"
#include "mxfp4.cuh"

namespace fp8q {
namespace {

constexpr int kBM = 128;
constexpr int kBK = 256;          // elements of k per stage
constexpr int kRowBytes = kBK / 2;
constexpr int kThreads = 192;
constexpr int kTmemCols = 512;

template <int BN, int STAGES>
struct Cfg {
  static constexpr int kAtoms = BN > 128 ? BN / 128 : 1;  // 128-row scale tiles per B tile
  static constexpr int kABytes = kBM * kRowBytes;
  static constexpr int kBBytes = BN * kRowBytes;
  static constexpr int kSfaBytes = 2 * kSfTileBytes;
  static constexpr int kSfbBytes = kAtoms * 2 * kSfTileBytes;
  // Codes first: A and B tiles stay on 1024-byte boundaries (the swizzle's period).
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kSfBytes = kSfaBytes + kSfbBytes;
  static constexpr int kSmem = 1024 + STAGES * (kStageBytes + kSfBytes);
  static constexpr int kSfaCols = 8, kSfbCols = 8 * kAtoms;
  static constexpr int kSfCols = kSfaCols + kSfbCols;
  static constexpr int kAcc = 2;
  static_assert(kAcc * BN + STAGES * kSfCols <= kTmemCols, "tensor memory");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct MatmulArgs {
  const uint8_t *a_sf, *b_sf;
  const int32_t* offsets;  // NULL: dense
  uint16_t* out;
  int64_t m, n;            // m: rows (dense) or the capacity (grouped)
  int k, groups;
  int* status;
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_copy_sf(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_load32(uint32_t (&v)[32], uint32_t tmem) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(tmem));
}
__device__ __forceinline__ void tc_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(hi)), "f"(__uint_as_float(lo)));
  return r;
}

// Shared-memory matrix descriptors (K-major, version 1): codes under the 128-byte swizzle,
// eight rows of 128 bytes apart by 1024; scale tiles without swizzle, eight 16-byte rows
// apart by 128.
__device__ __forceinline__ uint64_t desc_codes(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (8ull << 32) | (1ull << 46);
}
// Instruction descriptor of kind::mxf4: E2M1 operands, UE8M0 scales, M = 128, K = 64; the
// scale ids (bits 4-5 of B, 29-30 of A) pick the half of each 4-byte scale word.
__device__ __forceinline__ constexpr uint32_t idesc_mxf4(int n, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | (1u << 27) | (sf_id << 29);
}

// ------------------------------------------------------------------ tiles
struct Tile {
  int64_t row, col;  // of the output
  int64_t b_row;     // row of B under column col
};

// Output tile `t`, column tiles fastest; false for a tile whose group bounds are
// inconsistent (the status word says so) - every role skips the same tiles.
__device__ __forceinline__ bool locate(const MatmulArgs& a, int64_t t, int64_t n_tiles, int bn, Tile& o) {
  o.row = t / n_tiles * kBM;
  o.col = t % n_tiles * bn;
  o.b_row = o.col;
  if (a.offsets == nullptr) return true;
  int lo = 0, hi = a.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)ld_g(a.offsets + mid) <= o.row) lo = mid; else hi = mid;
  }
  const int64_t b = ld_g(a.offsets + lo), e = ld_g(a.offsets + lo + 1);
  o.b_row += lo * a.n;
  return b <= o.row && o.row < e && e <= a.m && ((b | e) & 127) == 0;
}

__device__ __forceinline__ bool wait_or_record(uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_wait_bounded(bar, parity, kWaitTimeoutNs)) return true;
  record_status(status, FP8Q_ERR_TIMEOUT);
  return false;
}

template <int BN, int STAGES>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                        MatmulArgs a) {
  using C = Cfg<BN, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[C::kAcc], acc_empty[C::kAcc], drain;
  __shared__ uint32_t tmem_sh;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kAcc; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 4);
    }
    mbar_init(&drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_sh)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_wait_for(a.a_sf, a.b_sf, a.offsets, a.out);
  pdl_trigger();

  const int64_t n_tiles = (a.n + BN - 1) / BN;
  int64_t rows = a.m;
  if (a.offsets != nullptr) {
    const bool report = blockIdx.x == 0 && threadIdx.x == 0;
    rows = grouped_rows(a.offsets, a.groups, a.m, report ? a.status : nullptr);
    if (blockIdx.x == 0) validate_groups_cta(a.offsets, a.groups, a.status);
  }
  const int64_t tiles = (rows + kBM - 1) / kBM * n_tiles;
  const int k128 = a.k / 128;
  const int steps = (a.k + kBK - 1) / kBK;

  if (warp == 0) {
    if (lane == 0) {
      asm volatile("fence.proxy.async.global;" ::: "memory");
      int s = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        Tile o;
        if (!locate(a, t, n_tiles, BN, o)) continue;
        const int64_t b_rows = a.offsets ? a.n * a.groups : a.n;
        const uint8_t* sfa = a.a_sf + (o.row >> 7) * k128 * kSfTileBytes;
        const uint8_t* sfb = a.b_sf + (o.b_row >> 7) * k128 * kSfTileBytes;
        int atoms = 1;  // scale tiles of B that exist under this tile
        if (C::kAtoms > 1) atoms = (int)min((int64_t)C::kAtoms, (b_rows - o.b_row + 127) >> 7);
        for (int j = 0; j < steps; ++j) {
          if (!wait_or_record(&empty[s], phase ^ 1u, a.status)) {
            ok = false;
            break;
          }
          const uint32_t sf_bytes = min(2, k128 - 2 * j) * kSfTileBytes;
          const uint32_t base = smem + s * C::kStageBytes;
          const uint32_t sf = smem + STAGES * C::kStageBytes + s * C::kSfBytes;
          mbar_expect_tx(&full[s], C::kStageBytes + (1 + atoms) * sf_bytes);
          tma_load_2d(base, &map_a, j * kRowBytes, (int)o.row, &full[s]);
          tma_load_2d(base + C::kABytes, &map_b, j * kRowBytes, (int)o.b_row, &full[s]);
          bulk_load(sf, sfa + (int64_t)j * 2 * kSfTileBytes, sf_bytes, &full[s]);
          for (int i = 0; i < atoms; ++i)
            bulk_load(sf + C::kSfaBytes + i * 2 * kSfTileBytes,
                      sfb + ((int64_t)i * k128 + (int64_t)j * 2) * kSfTileBytes, sf_bytes, &full[s]);
          ++issued;
          if (++s == STAGES) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      // Outstanding fills end before the CTA does: on the regular path each was consumed
      // (its stage was freed); after an expired wait its copies at least have landed.
      for (int i = 0; i < STAGES && issued > 0; ++i, --issued) {
        if (s == 0) {
          s = STAGES;
          phase ^= 1u;
        }
        --s;
        mbar_wait_bounded(ok ? &empty[s] : &full[s], phase, kWaitTimeoutNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int s = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        Tile o;
        if (!locate(a, t, n_tiles, BN, o)) continue;
        ok = wait_or_record(&acc_empty[acc], acc_phase ^ 1u, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int j = 0; j < steps; ++j) {
          ok = wait_or_record(&full[s], phase, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t base = smem + s * C::kStageBytes;
          const uint32_t sf = smem + STAGES * C::kStageBytes + s * C::kSfBytes;
          const uint32_t tm_a = tmem + C::kAcc * BN + s * C::kSfCols;
          const uint32_t tm_b = tm_a + C::kSfaCols;
          const int chunks = min(2, k128 - 2 * j);  // 128 elements of k each
          for (int c = 0; c < chunks; ++c) {
            tc_copy_sf(tm_a + 4 * c, desc_scales(sf + c * kSfTileBytes));
            for (int i = 0; i < C::kAtoms; ++i)
              tc_copy_sf(tm_b + 4 * (c * C::kAtoms + i),
                         desc_scales(sf + C::kSfaBytes + (2 * i + c) * kSfTileBytes));
          }
          // A B tile narrower than a scale tile starts inside it: 32 rows per column.
          const uint32_t shift = BN < 128 ? (uint32_t)(o.b_row & 127) >> 5 : 0u;
          for (int c = 0; c < chunks; ++c) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t off = (2 * c + h) * 32;  // 64 codes
              tc_mma_mxf4(d, desc_codes(base + off), desc_codes(base + C::kABytes + off), idesc_mxf4(BN, 2 * h),
                          tm_a + 4 * c, tm_b + 4 * c * C::kAtoms + shift, (uint32_t)(j + c + h > 0));
            }
          }
          tc_commit(&empty[s]);
          if (++s == STAGES) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(&acc_full[acc]);
        if (++acc == C::kAcc) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) {
        tc_commit(&drain);
        mbar_wait_bounded(&drain, 0u, kWaitTimeoutNs);
      }
    }
    __syncwarp();
  } else {
    const int quad = warp & 3;  // the tensor-memory lanes this warp may read
    int acc = 0;
    uint32_t acc_phase = 0;
    const bool vec = (a.n & 7) == 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
      Tile o;
      if (!locate(a, t, n_tiles, BN, o)) continue;
      if (!__all_sync(0xFFFFFFFFu, wait_or_record(&acc_full[acc], acc_phase, a.status))) break;
      tc_fence_after();
      const int64_t r = o.row + quad * 32 + lane;
      uint16_t* dst = a.out + r * a.n + o.col;
      const int64_t left = a.n - o.col;  // columns of this tile that exist
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t v[32];
        tc_load32(v, tmem + ((uint32_t)(quad * 32) << 16) + acc * BN + c);
        tc_wait_load();
        if (r < rows) {
          if (vec) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + 8 * i < left)
                *reinterpret_cast<uint4*>(dst + c + 8 * i) =
                    make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                               pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i < left) dst[c + i] = (uint16_t)pack_bf16(v[i], 0u);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      if (++acc == C::kAcc) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
  }
}

// ------------------------------------------------------------------ host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::once_flag once;
  static EncodeFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

// Codes [rows, k/2] bytes as boxes of box_rows rows x 128 bytes; rows and bytes past the
// array read as zero.
bool code_map(CUtensorMap* map, const void* q, int64_t rows, int64_t k, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dim[2] = {(cuuint64_t)(k / 2), (cuuint64_t)rows};
  const cuuint64_t stride[1] = {(cuuint64_t)(k / 2)};
  const cuuint32_t box[2] = {kRowBytes, (cuuint32_t)box_rows};
  const cuuint32_t one[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), dim, stride, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int STAGES>
fp8q_status launch_matmul(const DeviceInfo& dev, const uint8_t* aq, const uint8_t* bq, const MatmulArgs& a,
                          cudaStream_t stream) {
  using C = Cfg<BN, STAGES>;
  CUtensorMap ma, mb;
  if (!code_map(&ma, aq, a.m, a.k, kBM) || !code_map(&mb, bq, a.n * a.groups, a.k, BN)) return FP8Q_ERR_CUDA;
  auto kernel = mxfp4_matmul_kernel<BN, STAGES>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return FP8Q_ERR_CUDA;
  const int64_t tiles = (a.m + kBM - 1) / kBM * ((a.n + BN - 1) / BN);
  const unsigned grid = (unsigned)(tiles < dev.num_sms ? tiles : dev.num_sms);
  return launch_after(kernel, dim3(grid), kThreads, (size_t)C::kSmem, stream, ma, mb, a) == cudaSuccess ? FP8Q_OK
                                                                                                  : FP8Q_ERR_CUDA;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_matmul_mxfp4(const uint8_t* aq, const uint8_t* asf, int64_t m, const uint8_t* bq,
                                         const uint8_t* bsf, int64_t n, int64_t k, const int32_t* group_offsets,
                                         int32_t num_groups, void* out, fp8q_stream_t stream) {
  if (m < 0 || n < 0 || k < 0 || k % 128 || m > kMaxInt32 || n > kMaxInt32 || k > kMaxInt32) return FP8Q_ERR_SHAPE;
  if (num_groups < 1 || (!group_offsets && num_groups != 1)) return FP8Q_ERR_ARG;
  if (group_offsets && (n % 128 || n > kMaxInt32 / num_groups)) return FP8Q_ERR_SHAPE;
  if (m == 0 || n == 0) return FP8Q_OK;
  if (k == 0) return FP8Q_ERR_SHAPE;
  if (!aq || !asf || !bq || !bsf || !out) return FP8Q_ERR_NULL;
  if (!aligned_to(aq, 16) || !aligned_to(asf, 16) || !aligned_to(bq, 16) || !aligned_to(bsf, 16) ||
      !aligned_to(out, 16) || !aligned_to(group_offsets, 4))
    return FP8Q_ERR_ALIGN;
  DeviceInfo dev;
  if (device_info(&dev) != FP8Q_OK) return FP8Q_ERR_CUDA;
  const MatmulArgs a = {asf, bsf, group_offsets, static_cast<uint16_t*>(out), m, n, (int)k, num_groups, dev.status};
  return launch_matmul<128, 6>(dev, aq, bq, a, to_stream(stream));
}
