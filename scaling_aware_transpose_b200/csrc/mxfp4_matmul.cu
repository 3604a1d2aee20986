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
//   warp 0     TMA loads of the A and B codes; every fourth stage, bulk copies of the scale
//              tiles, which the quantizers store in the order the tensor core reads;
//   warp 1     four MMAs of 64 elements per stage and a commit that frees it;
//   warps 2-9  scales: shared memory -> registers -> tensor memory, each warp its quarter of
//              the lanes, two warps a quarter taking turns.  (tcgen05.cp from the MMA thread
//              took turns with the MMAs: 36 ns a 512-byte tile, and the pipe drained at each
//              change from one to the other: 141 us for what took 105 this way.)
//   warps 10-13  the epilogue: tensor memory -> registers -> BF16 -> global.
// What bounds it: at large sizes the tensor pipe and the 1000 W power cap (below, CTA pairs);
// at few rows the chain of a CTA's stages, about 0.3 us each, on top of 3 us of start, first
// copy and epilogue (1x4096x7168: 7.1 us, for 15.7 MB of weights: 2.4 us at the copy rate).
// Scale columns in tensor memory belong to the stage: they are rewritten only after the
// stage's MMAs have completed.
//
// Every wait is bounded; a role whose wait expires records FP8Q_ERR_TIMEOUT and leaves its
// loop, the others follow, outstanding copies and MMAs are waited for (again bounded) and
// the tensor memory is freed.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "abi_checks.h"
#include "bulk.cuh"
#include "cluster.cuh"
#include "launch.h"
#include "mxfp4.cuh"

namespace fp8q {
namespace {

constexpr int kBM = 128;
constexpr int kBK = 256;          // elements of k per stage
constexpr int kRowBytes = kBK / 2;
constexpr int kThreads = 448;
constexpr int kSfSteps = 4;       // stages per slot of scale tiles
constexpr int kSfSlots = 2;
constexpr int kTmemCols = 512;
constexpr int kPitch = 8;         // words of a staged row piece (16 columns)

template <int BN, int STAGES, int ACC>
struct Cfg {
  static constexpr int kAtoms = BN > 128 ? BN / 128 : 1;  // 128-row scale tiles per B tile
  static constexpr int kABytes = kBM * kRowBytes;
  static constexpr int kBBytes = BN * kRowBytes;
  // Codes first: A and B tiles stay on 1024-byte boundaries (the swizzle's period).
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kSfRun = kSfSteps * 2 * kSfTileBytes;  // one 128-row tile column of a slot
  static constexpr int kSlotBytes = (1 + kAtoms) * kSfRun;
  static constexpr int kSmem = 1024 + STAGES * kStageBytes + kSfSlots * kSlotBytes;
  static constexpr int kSfaCols = 8, kSfbCols = 8 * kAtoms;
  static constexpr int kSfCols = kSfaCols + kSfbCols;
  static constexpr int kAcc = ACC;  // accumulators in tensor memory
  static_assert(kAcc * BN + STAGES * kSfCols <= kTmemCols, "tensor memory");
  static_assert(kSmem <= 222 * 1024, "shared memory");  // 5 KB more are static
};

struct MatmulArgs {
  const uint8_t *a_sf, *b_sf;
  const int32_t* offsets;  // NULL: dense
  uint16_t* out;
  int64_t m, n;            // m: rows (dense) or the capacity (grouped)
  int k, groups;
  int a_rows;              // rows of A that a stage loads (the rest of its 128 are never stored)
  int* status;
};

// ------------------------------------------------------------------ PTX
// One lane of a converged warp, always the same.  The issuing roles run their loops with the
// whole warp and put only the asynchronous instructions under it: the compiler then keeps
// their operands in uniform registers (a loop run by one lane alone spent about 50 ns per
// MMA moving them there).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
// The same by one CTA of a pair: the barrier may lie in the other CTA.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_store4(uint32_t tmem, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tmem), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void tc_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                                 uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
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

// Shared-memory matrix descriptor (K-major, version 1): codes under the 128-byte swizzle,
// eight rows of 128 bytes apart by 1024.
__device__ __forceinline__ uint64_t desc_codes(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::mxf4: E2M1 operands, UE8M0 scales, M = 128 or 256, K = 64;
// the scale ids (bits 4-5 of B, 29-30 of A) pick the half of each 4-byte scale word.
__device__ __forceinline__ constexpr uint32_t idesc_mxf4(int m, int n, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27) |
         (sf_id << 29);
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

// Called by a whole warp; the same answer in every lane.
__device__ __forceinline__ bool wait_or_record(uint64_t* bar, uint32_t parity, int* status) {
  if (__all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, kWaitTimeoutNs))) return true;
  record_status(status, FP8Q_ERR_TIMEOUT);
  return false;
}

// One epilogue warp: 32 rows (row0 + lane) x BN columns of the accumulator at `tmem` to BF16
// rows of out below row_end and columns below n.  `read` is called once the accumulator has
// been read to the end: kPart columns are packed in registers at a time, all of a pair's, whose
// one accumulator the next tile waits for, and 64 of a CTA's alone (128 at a time spilled in the
// 256-column kernel: 1024x4096x4096 12.7 us, not 11.5).
//
// Where rows start on 16 bytes the words pass through shared memory, eight rows of 64 columns at
// a time (16-byte pieces, their order within a row exchanged by its number: no bank conflicts),
// so that a store instruction covers whole 128-byte runs, in 32-byte stores where rows start on
// 32 bytes.  The stores share the path between the SMs and L2 with the operands, which at large
// sizes take some 48 bytes a cycle of each SM: 8192x4096x7168 takes 86 us so, 89 with each lane
// storing its own row in 32-byte pieces, 96 in 16-byte pieces, 79 without stores.
template <int BN, int kPart, typename Read>
__device__ __forceinline__ void store_tile(const MatmulArgs& a, uint32_t tmem, int64_t row0, int64_t row_end, int64_t col,
                                           int lane, uint32_t* staging, Read read) {
  const bool aligned = (a.n & 7) == 0;
  const bool wide = (a.n & 15) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  const int left = (int)min((int64_t)BN, a.n - col);  // columns of this tile that exist
#pragma unroll 1
  for (int h = 0; h < BN; h += kPart) {
    uint32_t p[kPart / 2];
#pragma unroll
    for (int c = 0; c < kPart; c += 32) {
      uint32_t v[32];
      tc_load32(v, tmem + h + c);
      tc_wait_load();
#pragma unroll
      for (int i = 0; i < 16; ++i) p[c / 2 + i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
    if (h + kPart == BN) read();  // the next tile's MMAs may overwrite it
    if (aligned) {
      constexpr int kWide = kPart < 64 ? kPart : 64, kPieces = kWide / 8, kRowLanes = kWide / 16, kRows = 32 / kRowLanes;
      uint4* st = reinterpret_cast<uint4*>(staging);
      const int sr = lane / kRowLanes, sq = 2 * (lane % kRowLanes), turn = sr & (kPieces - 1);
#pragma unroll
      for (int c = 0; c < kPart; c += kWide) {
#pragma unroll 1
        for (int g = 0; g < 32; g += kRows) {
          if (lane / kRows * kRows == g) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
              st[(lane - g) * kPieces + (i ^ (lane & (kPieces - 1)))] =
                  make_uint4(p[c / 2 + 4 * i], p[c / 2 + 4 * i + 1], p[c / 2 + 4 * i + 2], p[c / 2 + 4 * i + 3]);
          }
          __syncwarp();
          const uint4 lo = st[sr * kPieces + (sq ^ turn)], hi = st[sr * kPieces + ((sq + 1) ^ turn)];
          const int64_t r = row0 + g + sr;
          const int x = h + c + 8 * sq;
          if (r < row_end && x < left) {
            uint16_t* to = a.out + r * a.n + col + x;
            if (wide) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(lo.x), "r"(lo.y),
                           "r"(lo.z), "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(to) = lo;
              if (x + 8 < left) *reinterpret_cast<uint4*>(to + 8) = hi;
            }
          }
          __syncwarp();
        }
      }
    } else {
      // Other rows: 16 columns at a time, so that half a warp stores 16 neighbouring elements of
      // a row, with all of a chunk's loads on their way before its stores (1003x2050x1408: 7.9 us,
      // 9.1 in rounds of four; each lane storing its own row element by element took 2.5 times
      // as long over the whole product).
      uint32_t* mine = staging + lane * kPitch;
      const uint16_t* all = reinterpret_cast<const uint16_t*>(staging);
      const int rows_here = (int)max((int64_t)0, min((int64_t)32, row_end - row0));
      uint16_t* base = a.out + row0 * a.n + col + h;
#pragma unroll
      for (int c = 0; c < kPart; c += 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) mine[i ^ (lane >> 2)] = p[c / 2 + i];
        __syncwarp();
        const int x = c + (lane & 15);
        uint16_t* to = base + (lane >> 4) * a.n + x;
        if (h + x < left) {
#pragma unroll 16
          for (int i = 0; i < 32; i += 2) {
            const int r = i + (lane >> 4);
            if (r < rows_here) *to = all[(r * kPitch + ((lane >> 1 & 7) ^ (r >> 2))) * 2 + (lane & 1)];
            to += 2 * a.n;
          }
        }
        __syncwarp();
      }
    }
  }
}

template <int BN, int STAGES, int ACC, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                        MatmulArgs a) {
  using C = Cfg<BN, STAGES, ACC>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[STAGES], empty[STAGES], scaled[STAGES], sf_full[kSfSlots], sf_empty[kSfSlots];
  __shared__ uint64_t acc_full[C::kAcc], acc_empty[C::kAcc], drain;
  __shared__ uint32_t tmem_sh;
  __shared__ __align__(16) uint32_t odd_rows[4][32 * kPitch];
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&scaled[s], 4);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_empty[s], 8);
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
  // Persistent: tiles blockIdx.x, + gridDim.x, ..., every step of k.  Split: the CTAs of a
  // cluster share one tile, each a contiguous run of the steps.
  const uint32_t split = SPLIT ? cluster_size() : 1u, rank = SPLIT ? cluster_rank() : 0u;
  const int64_t t0 = blockIdx.x / split, stride = gridDim.x / split;
  const int all_steps = (a.k + kBK - 1) / kBK;
  const int j0 = (int)((int64_t)all_steps * rank / split);
  const int steps = (int)((int64_t)all_steps * (rank + 1) / split) - j0;

  if (warp == 0) {
    asm volatile("fence.proxy.async.global;" ::: "memory");
    int s = 0, slot = 0;
    uint32_t phase = 0, slot_phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t t = t0; ok && t < tiles; t += stride) {
      Tile o;
      if (!locate(a, t, n_tiles, BN, o)) continue;
      const int64_t b_rows = a.offsets ? a.n * a.groups : a.n;
      const uint8_t* sfa = a.a_sf + (o.row >> 7) * k128 * kSfTileBytes;
      const uint8_t* sfb = a.b_sf + (o.b_row >> 7) * k128 * kSfTileBytes;
      int atoms = 1;  // scale tiles of B that exist under this tile
      if (C::kAtoms > 1) atoms = (int)min((int64_t)C::kAtoms, (b_rows - o.b_row + 127) >> 7);
      for (int j = 0; j < steps; ++j) {
        if (j % kSfSteps == 0) {
          ok = wait_or_record(&sf_empty[slot], slot_phase ^ 1u, a.status);
          if (!ok) break;
          const uint32_t bytes = min(2 * kSfSteps, k128 - 2 * (j0 + j)) * kSfTileBytes;
          const uint32_t sf = smem + STAGES * C::kStageBytes + slot * C::kSlotBytes;
          if (elect_one()) {
            mbar_expect_tx(&sf_full[slot], (1 + atoms) * bytes);
            bulk_load(sf, sfa + (int64_t)(j0 + j) * 2 * kSfTileBytes, bytes, &sf_full[slot]);
            for (int i = 0; i < atoms; ++i)
              bulk_load(sf + (1 + i) * C::kSfRun, sfb + ((int64_t)i * k128 + (int64_t)(j0 + j) * 2) * kSfTileBytes, bytes,
                        &sf_full[slot]);
          }
          __syncwarp();
          if (++slot == kSfSlots) {
            slot = 0;
            slot_phase ^= 1u;
          }
        }
        ok = wait_or_record(&empty[s], phase ^ 1u, a.status);
        if (!ok) break;
        const uint32_t base = smem + s * C::kStageBytes;
        if (elect_one()) {
          mbar_expect_tx(&full[s], a.a_rows * kRowBytes + C::kBBytes);
          tma_load_2d(base, &map_a, (j0 + j) * kRowBytes, (int)o.row, &full[s]);
          tma_load_2d(base + C::kABytes, &map_b, (j0 + j) * kRowBytes, (int)o.b_row, &full[s]);
        }
        __syncwarp();
        ++issued;
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    // Outstanding fills end before the CTA does: on the regular path each was consumed (its
    // stage was freed); after an expired wait its copies at least have landed.
    for (int i = 0; i < STAGES && issued > 0; ++i, --issued) {
      if (s == 0) {
        s = STAGES;
        phase ^= 1u;
      }
      --s;
      mbar_wait_bounded(ok ? &empty[s] : &full[s], phase, kWaitTimeoutNs);
    }
    for (int i = 0; i < kSfSlots; ++i) {  // (a slot never filled passes at once)
      if (slot == 0) {
        slot = kSfSlots;
        slot_phase ^= 1u;
      }
      --slot;
      mbar_wait_bounded(&sf_full[slot], slot_phase, kWaitTimeoutNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    int s = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int64_t t = t0; ok && t < tiles; t += stride) {
      Tile o;
      if (!locate(a, t, n_tiles, BN, o)) continue;
      ok = wait_or_record(&acc_empty[acc], acc_phase ^ 1u, a.status);
      if (!ok) break;
      const uint32_t d = tmem + acc * BN;
      for (int j = 0; j < steps; ++j) {
        ok = wait_or_record(&scaled[s], phase, a.status);  // the codes have landed, too
        if (!ok) break;
        tc_fence_after();
        const uint32_t tm_a = tmem + C::kAcc * BN + s * C::kSfCols;
        const uint32_t tm_b = tm_a + C::kSfaCols;
        const uint64_t da = desc_codes(smem + s * C::kStageBytes);
        const uint64_t db = desc_codes(smem + s * C::kStageBytes + C::kABytes);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < 4; ++h)  // 64 codes: 32 bytes, two scales of a row's four-byte word
            if (h < 2 || 2 * (j0 + j) + 1 < k128)
              tc_mma_mxf4(d, da + 2 * h, db + 2 * h, idesc_mxf4(kBM, BN, 2 * (h & 1)), tm_a + 4 * (h >> 1),
                          tm_b + 4 * (h >> 1) * C::kAtoms, (uint32_t)(j + h > 0));
          tc_commit(&empty[s]);
          if (j + 1 == steps) tc_commit(&acc_full[acc]);
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (++acc == C::kAcc) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok) {
      if (elect_one()) tc_commit(&drain);
      __syncwarp();
      mbar_wait_bounded(&drain, 0u, kWaitTimeoutNs);
    }
    __syncwarp();
  } else if (warp < 10) {
    const int quad = warp & 3;  // the tensor-memory lanes this warp may write
    int s = 0, slot = 0;
    uint32_t phase = 0, slot_phase = 0, turn = warp < 6 ? 0u : 1u;  // two warps a quarter take turns
    bool ok = true;
    for (int64_t t = t0; ok && t < tiles; t += stride) {
      Tile o;
      if (!locate(a, t, n_tiles, BN, o)) continue;
      for (int j = 0; j < steps; ++j) {
        const uint8_t* sf = smem_raw + (smem - smem_u32(smem_raw)) + STAGES * C::kStageBytes + slot * C::kSlotBytes +
                            (j % kSfSteps) * 2 * kSfTileBytes + lane * 16;
        if (j % kSfSteps == 0) ok = wait_or_record(&sf_full[slot], slot_phase, a.status);
        if (!ok) break;
        if (turn == 0) {
          uint4 v[2 * (1 + C::kAtoms)];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i <= C::kAtoms; ++i)
              v[c * (1 + C::kAtoms) + i] = *reinterpret_cast<const uint4*>(sf + i * C::kSfRun + c * kSfTileBytes);
          if (BN < 128) {
            // A B tile narrower than a scale tile starts inside it (32 rows per word): its first
            // word goes to the first column, whose address stays a multiple of four.
            const uint32_t first = (uint32_t)(o.b_row & 127) >> 5;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint4& w = v[2 * c + 1];
              if (first & 2) w = make_uint4(w.z, w.w, w.z, w.w);
              if (first & 1) w.x = w.y;  // (32 rows: one word)
            }
          }
          // A filled stage was free before: so are its scale columns.
          ok = wait_or_record(&full[s], phase, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tm = tmem + ((uint32_t)(quad * 32) << 16) + C::kAcc * BN + s * C::kSfCols;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tc_store4(tm + 4 * c, v[c * (1 + C::kAtoms)]);
#pragma unroll
            for (int i = 0; i < C::kAtoms; ++i)
              tc_store4(tm + C::kSfaCols + 4 * (c * C::kAtoms + i), v[c * (1 + C::kAtoms) + 1 + i]);
          }
          tc_wait_store();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&scaled[s]);
        }
        turn ^= 1u;
        const bool slot_done = (j + 1) % kSfSteps == 0 || j + 1 == steps;
        if (slot_done && lane == 0) mbar_arrive(&sf_empty[slot]);
        if (slot_done && ++slot == kSfSlots) {
          slot = 0;
          slot_phase ^= 1u;
        }
        if (++s == STAGES) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    const int quad = warp & 3;  // the tensor-memory lanes this warp may read
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int64_t t = t0; t < tiles; t += stride) {
      Tile o;
      if (!locate(a, t, n_tiles, BN, o)) continue;
      if (!wait_or_record(&acc_full[acc], acc_phase, a.status)) break;
      tc_fence_after();
      const int64_t r = o.row + quad * 32 + lane;
      if (SPLIT) {
        // This CTA's fp32 sums go to shared memory (the stages are all consumed), one padded
        // row per output row; they are added up below.
        float* part = reinterpret_cast<float*>(smem_raw + (smem - smem_u32(smem_raw))) + (quad * 32 + lane) * (BN + 4);
#pragma unroll 1
        for (int c = 0; c < BN; c += 32) {
          uint32_t v[32];
          tc_load32(v, tmem + ((uint32_t)(quad * 32) << 16) + acc * BN + c);
          tc_wait_load();
          if (r < rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(part + c + 4 * i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        break;
      }
      store_tile<BN, (BN < 64 ? BN : 64)>(a, tmem + ((uint32_t)(quad * 32) << 16) + acc * BN, o.row + quad * 32, rows, o.col, lane,
                     odd_rows[quad], [&] {
                       tc_fence_before();
                       __syncwarp();
                       if (lane == 0) mbar_arrive(&acc_empty[acc]);
                     });
      if (++acc == C::kAcc) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  tc_fence_before();
  if (SPLIT) {
    __syncwarp();
    cluster_sync();
    Tile o;
    if (t0 < tiles && locate(a, t0, n_tiles, BN, o)) {
      const int live = (int)min((int64_t)kBM, rows - o.row);
      const bool vec = (a.n & 3) == 0;
      for (int i = rank * kThreads + threadIdx.x; i < live * (BN / 4); i += split * kThreads) {
        const int r = i / (BN / 4), c = i % (BN / 4) * 4;
        if (o.col + c >= a.n) continue;
        float4 v = ld_cluster4(smem + (uint32_t)(r * (BN + 4) + c) * 4, 0);
        for (uint32_t q = 1; q < split; ++q) {  // in rank order
          const float4 w = ld_cluster4(smem + (uint32_t)(r * (BN + 4) + c) * 4, q);
          v.x += w.x;
          v.y += w.y;
          v.z += w.z;
          v.w += w.w;
        }
        uint16_t* dst = a.out + (o.row + r) * a.n + o.col + c;
        const uint32_t lo = pack_bf16(__float_as_uint(v.x), __float_as_uint(v.y));
        const uint32_t hi = pack_bf16(__float_as_uint(v.z), __float_as_uint(v.w));
        if (vec) {
          *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else {
          dst[0] = (uint16_t)lo;
          if (o.col + c + 1 < a.n) dst[1] = (uint16_t)(lo >> 16);
          if (o.col + c + 2 < a.n) dst[2] = (uint16_t)hi;
          if (o.col + c + 3 < a.n) dst[3] = (uint16_t)(hi >> 16);
        }
      }
    }
    cluster_sync();  // a peer may still be reading this CTA's sums
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

template <int BN, int STAGES, int ACC, bool SPLIT>
fp8q_status launch_matmul(const DeviceInfo& dev, const uint8_t* aq, const uint8_t* bq, const MatmulArgs& a, int split,
                          cudaStream_t stream) {
  using C = Cfg<BN, STAGES, ACC>;
  static_assert(!SPLIT || kBM * (BN + 4) * 4 <= STAGES * C::kStageBytes, "the sums fit the stages");
  CUtensorMap ma, mb;
  if (!code_map(&ma, aq, a.m, a.k, a.a_rows) || !code_map(&mb, bq, a.n * a.groups, a.k, BN)) return FP8Q_ERR_CUDA;
  auto kernel = mxfp4_matmul_kernel<BN, STAGES, ACC, SPLIT>;
  static std::atomic<uint64_t> prepared{0};  // devices (below 64) whose shared-memory limit was raised
  if (!(prepared.load(std::memory_order_relaxed) >> dev.device & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return FP8Q_ERR_CUDA;
    prepared.fetch_or(1ull << dev.device, std::memory_order_relaxed);
  }
  const int64_t tiles = (a.m + kBM - 1) / kBM * ((a.n + BN - 1) / BN);
  const unsigned grid = (unsigned)(SPLIT ? tiles * split : tiles < dev.num_sms ? tiles : dev.num_sms);
  return launch_clusters_after(kernel, grid, (unsigned)split, kThreads, (size_t)C::kSmem, stream, ma, mb, a) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

// ------------------------------------------------------------------ CTA pairs
// Large products: two CTAs of a cluster share one tile of 256 x 256.  Each loads its 128 rows
// of A and of B (half the B bytes of a CTA alone) and holds 128 rows of the accumulator; the
// first one's MMAs (cta_group::2, M = 256) read both.  A CTA alone at 128 x 256 moves 48 KB of
// codes into shared memory and 48 KB out per stage, more than the 128 bytes a cycle allow
// under the MMAs; a pair moves 32 KB each way.  8192x4096x7168: 86 us, 102 by CTAs alone; 8192^3:
// 190 us (5.8 PFLOP/s) for the first milliseconds and 210 us under the 1000 W cap, which takes
// the SM clock to 1.36 GHz.
// What the pair exchanges: the copies of both complete on the first CTA's `full`; the second
// one's scale warps and epilogue arrive on the first one's `scaled` and `acc_empty`; warp 18 of
// the first CTA passes `empty` and `acc_full`, which the MMAs' commits set, on to the second.
constexpr int kPairStages = 6;
constexpr int kPairThreads = 608;
constexpr int kPairMaxGroups = 256;
constexpr int kPairStageBytes = 2 * kBM * kRowBytes;
constexpr int kPairSlotBytes = 3 * kSfSteps * 2 * kSfTileBytes;
constexpr int kPairSmem = 1024 + kPairStages * kPairStageBytes + kSfSlots * kPairSlotBytes;
constexpr int kPairSfCols = 24, kPairN = 256;
static_assert(kPairN + kPairStages * kPairSfCols <= kTmemCols, "tensor memory");
static_assert(kPairSmem <= 217 * 1024, "shared memory");  // 10 KB more are static

// What crosses between the two CTAs through these barriers is the order of tensor-memory and
// asynchronous-copy operations, which tcgen05's fences and waits and the copies' completion
// settle; no ordinary memory is handed over.  So arrivals and waits keep the barriers' default
// (CTA) scope: at cluster scope each cost several hundred cycles (a stage 1050 ns, not 490).
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

struct PairTile {
  int64_t row, row_end, col, b_row;
};

__global__ void __launch_bounds__(kPairThreads, 1)
    mxfp4_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, MatmulArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kPairStages], empty[kPairStages], scaled[kPairStages], sf_full[kSfSlots], sf_empty[kSfSlots];
  __shared__ uint64_t acc_full, acc_empty, drain;
  __shared__ uint32_t tmem_sh;
  __shared__ __align__(16) uint32_t odd_rows[8][32 * kPitch];
  __shared__ int tiles_before[kPairMaxGroups + 1];  // of 256 rows, in the groups before g
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool first = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&scaled[s], 8);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_empty[s], 8);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&acc_empty, 16);
    mbar_init(&drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_sh)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and tensor memory exist
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  pdl_wait_for(a.a_sf, a.b_sf, a.offsets, a.out);
  pdl_trigger();

  const int64_t n_tiles = (a.n + kPairN - 1) / kPairN;
  int64_t m_tiles = (a.m + 2 * kBM - 1) / (2 * kBM);
  if (a.offsets != nullptr) {
    const bool report = blockIdx.x == 0 && threadIdx.x == 0;
    const int64_t rows = grouped_rows(a.offsets, a.groups, a.m, report ? a.status : nullptr);
    if (blockIdx.x == 0) validate_groups_cta(a.offsets, a.groups, a.status);
    if (warp == 0) {  // scan of the groups' tile counts; an inconsistent group has none
      int run = 0;
      for (int g0 = 0; g0 < a.groups; g0 += 32) {
        int c = 0;
        if (g0 + lane < a.groups) {
          const int64_t b = ld_g(a.offsets + g0 + lane), e = ld_g(a.offsets + g0 + lane + 1);
          if (b >= 0 && b <= e && e <= rows && ((b | e) & 127) == 0) c = (int)((e - b + 2 * kBM - 1) / (2 * kBM));
        }
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += v;
        }
        if (g0 + lane < a.groups) tiles_before[g0 + lane] = run + incl - c;
        run += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
      if (lane == 0) tiles_before[a.groups] = run;
    }
    __syncthreads();
    m_tiles = tiles_before[a.groups];
  }
  const int64_t tiles = m_tiles * n_tiles;
  const int64_t t0 = blockIdx.x >> 1, stride = gridDim.x >> 1;
  const int k128 = a.k / 128;
  const int steps = (a.k + kBK - 1) / kBK;
  auto locate_pair = [&](int64_t t) {
    PairTile o;
    const int64_t tm = t / n_tiles;
    o.col = t % n_tiles * kPairN;
    o.b_row = o.col;
    o.row = tm * 2 * kBM;
    o.row_end = a.m;
    if (a.offsets != nullptr) {
      int lo = 0, hi = a.groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles_before[mid] <= tm) lo = mid; else hi = mid;
      }
      o.row = ld_g(a.offsets + lo) + (tm - tiles_before[lo]) * 2 * kBM;
      o.row_end = ld_g(a.offsets + lo + 1);
      o.b_row += lo * a.n;
    }
    return o;
  };

  if (warp == 0) {
    asm volatile("fence.proxy.async.global;" ::: "memory");
    int s = 0, slot = 0;
    uint32_t phase = 0, slot_phase = 0;
    int64_t issued = 0;
    bool ok = true;
    const int64_t b_rows = a.offsets ? a.n * a.groups : a.n;
    for (int64_t t = t0; ok && t < tiles; t += stride) {
      const PairTile o = locate_pair(t);
      const int64_t row = o.row + rank * kBM;      // this CTA's rows of A and of B
      const int64_t b_row = o.b_row + rank * kBM;
      const uint8_t* sfa = a.a_sf + (row >> 7) * k128 * kSfTileBytes;
      const uint8_t* sfb = a.b_sf + (o.b_row >> 7) * k128 * kSfTileBytes;
      const int a_atoms = row < a.m ? 1 : 0;  // scale tiles that exist
      const int b_atoms = (int)min((int64_t)2, (b_rows - o.b_row + 127) >> 7);
      for (int j = 0; j < steps; ++j) {
        if (j % kSfSteps == 0) {
          ok = wait_or_record(&sf_empty[slot], slot_phase ^ 1u, a.status);
          if (!ok) break;
          const uint32_t bytes = min(2 * kSfSteps, k128 - 2 * j) * kSfTileBytes;
          const uint32_t sf = smem + kPairStages * kPairStageBytes + slot * kPairSlotBytes;
          constexpr uint32_t kRun = kSfSteps * 2 * kSfTileBytes;
          if (elect_one()) {
            mbar_expect_tx(&sf_full[slot], (a_atoms + b_atoms) * bytes);
            if (a_atoms) bulk_load(sf, sfa + (int64_t)j * 2 * kSfTileBytes, bytes, &sf_full[slot]);
            for (int i = 0; i < b_atoms; ++i)
              bulk_load(sf + (1 + i) * kRun, sfb + ((int64_t)i * k128 + (int64_t)j * 2) * kSfTileBytes, bytes,
                        &sf_full[slot]);
          }
          __syncwarp();
          if (++slot == kSfSlots) {
            slot = 0;
            slot_phase ^= 1u;
          }
        }
        ok = wait_or_record(&empty[s], phase ^ 1u, a.status);
        if (!ok) break;
        const uint32_t base = smem + s * kPairStageBytes;
        const uint32_t bar = peer_address(smem_u32(&full[s]), 0);
        if (elect_one()) {
          if (first) mbar_expect_tx(&full[s], 2 * kPairStageBytes);
          tma_load_2d_pair(base, &map_a, j * kRowBytes, (int)row, bar);
          tma_load_2d_pair(base + kBM * kRowBytes, &map_b, j * kRowBytes, (int)b_row, bar);
        }
        __syncwarp();
        ++issued;
        if (++s == kPairStages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    // Fills end before the CTA does: on the regular path each was consumed (its stage was
    // freed).  After an expired wait the first CTA's `full` says when both CTAs' copies have
    // landed; the second CTA then leaves with the cluster barrier below.
    for (int i = 0; i < kPairStages && issued > 0; ++i, --issued) {
      if (s == 0) {
        s = kPairStages;
        phase ^= 1u;
      }
      --s;
      if (ok) mbar_wait_bounded(&empty[s], phase, kWaitTimeoutNs);
      else if (first) mbar_wait_bounded(&full[s], phase, kWaitTimeoutNs);
    }
    for (int i = 0; i < kSfSlots; ++i) {  // (a slot never filled passes at once)
      if (slot == 0) {
        slot = kSfSlots;
        slot_phase ^= 1u;
      }
      --slot;
      mbar_wait_bounded(&sf_full[slot], slot_phase, kWaitTimeoutNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (first) {
      int s = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t t = t0; ok && t < tiles; t += stride) {
        ok = wait_or_record(&acc_empty, acc_phase ^ 1u, a.status);
        if (!ok) break;
        acc_phase ^= 1u;
        for (int j = 0; j < steps; ++j) {
          ok = wait_or_record(&scaled[s], phase, a.status);  // the codes have landed, too
          if (!ok) break;
          tc_fence_after();
          const uint32_t tm_a = tmem + kPairN + s * kPairSfCols, tm_b = tm_a + 8;
          const uint64_t da = desc_codes(smem + s * kPairStageBytes);
          const uint64_t db = desc_codes(smem + s * kPairStageBytes + kBM * kRowBytes);
          if (elect_one()) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (h < 2 || 2 * j + 1 < k128)
                tc_mma_mxf4_pair(tmem, da + 2 * h, db + 2 * h, idesc_mxf4(2 * kBM, kPairN, 2 * (h & 1)),
                                 tm_a + 4 * (h >> 1), tm_b + 8 * (h >> 1), (uint32_t)(j + h > 0));
            tc_commit_pair(&empty[s]);
            if (j + 1 == steps) tc_commit_pair(&acc_full);
          }
          __syncwarp();
          if (++s == kPairStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        if (elect_one()) tc_commit_pair(&drain);
        __syncwarp();
        mbar_wait_bounded(&drain, 0u, kWaitTimeoutNs);
      }
    }
    __syncwarp();
  } else if (warp < 10) {
    const int quad = warp & 3;  // the tensor-memory lanes this warp may write
    int s = 0, slot = 0;
    uint32_t phase = 0, slot_phase = 0, turn = warp < 6 ? 0u : 1u;  // two warps a quarter take turns
    bool ok = true;
    for (int64_t t = t0; ok && t < tiles; t += stride) {
      for (int j = 0; j < steps; ++j) {
        const uint8_t* sf = smem_raw + (smem - smem_u32(smem_raw)) + kPairStages * kPairStageBytes + slot * kPairSlotBytes +
                            (j % kSfSteps) * 2 * kSfTileBytes + lane * 16;
        if (j % kSfSteps == 0) ok = wait_or_record(&sf_full[slot], slot_phase, a.status);
        if (!ok) break;
        if (turn == 0) {
          uint4 v[6];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 3; ++i)
              v[c * 3 + i] = *reinterpret_cast<const uint4*>(sf + i * kSfSteps * 2 * kSfTileBytes + c * kSfTileBytes);
          // A stage filled (the first CTA sees that) or passed on as free: its scale columns are
          // free in both CTAs.
          ok = first ? wait_or_record(&full[s], phase, a.status) : wait_or_record(&empty[s], phase ^ 1u, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t tm = tmem + ((uint32_t)(quad * 32) << 16) + kPairN + s * kPairSfCols;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tc_store4(tm + 4 * c, v[c * 3]);
            tc_store4(tm + 8 + 8 * c, v[c * 3 + 1]);
            tc_store4(tm + 12 + 8 * c, v[c * 3 + 2]);
          }
          tc_wait_store();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(peer_address(smem_u32(&scaled[s]), 0));
        }
        turn ^= 1u;
        const bool slot_done = (j + 1) % kSfSteps == 0 || j + 1 == steps;
        if (slot_done && lane == 0) mbar_arrive(&sf_empty[slot]);
        if (slot_done && ++slot == kSfSlots) {
          slot = 0;
          slot_phase ^= 1u;
        }
        if (++s == kPairStages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp < 18) {
    const int quad = warp & 3, half = (warp - 10) >> 2;  // a quarter of the rows, half of the columns
    uint32_t acc_phase = 0;
    for (int64_t t = t0; t < tiles; t += stride) {
      const PairTile o = locate_pair(t);
      if (!wait_or_record(&acc_full, acc_phase, a.status)) break;
      acc_phase ^= 1u;
      tc_fence_after();
      const int64_t row0 = o.row + rank * kBM + quad * 32;
      store_tile<kPairN / 2, kPairN / 2>(a, tmem + ((uint32_t)(quad * 32) << 16) + half * (kPairN / 2), row0, o.row_end,
                             o.col + half * (kPairN / 2), lane, odd_rows[warp - 10], [&] {
                               tc_fence_before();
                               __syncwarp();
                               if (lane == 0) arrive_at(peer_address(smem_u32(&acc_empty), 0));
                             });
    }
    __syncwarp();
  } else if (first) {
    // Passes the commits on to the second CTA.
    int s = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int64_t t = t0; ok && t < tiles; t += stride) {
      for (int j = 0; ok && j < steps; ++j) {
        ok = wait_or_record(&empty[s], phase, a.status);
        if (ok && lane == 0) arrive_at(peer_address(smem_u32(&empty[s]), 1));
        __syncwarp();
        if (++s == kPairStages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      ok = wait_or_record(&acc_full, acc_phase, a.status);
      acc_phase ^= 1u;
      if (ok && lane == 0) arrive_at(peer_address(smem_u32(&acc_full), 1));
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of either CTA is in flight to the other
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
  }
}

fp8q_status launch_pair(const DeviceInfo& dev, const uint8_t* aq, const uint8_t* bq, MatmulArgs a, cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!code_map(&ma, aq, a.m, a.k, kBM) || !code_map(&mb, bq, a.n * a.groups, a.k, kBM)) return FP8Q_ERR_CUDA;
  static std::atomic<uint64_t> prepared{0};
  if (!(prepared.load(std::memory_order_relaxed) >> dev.device & 1)) {
    if (cudaFuncSetAttribute(mxfp4_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem) != cudaSuccess)
      return FP8Q_ERR_CUDA;
    prepared.fetch_or(1ull << dev.device, std::memory_order_relaxed);
  }
  const int64_t tiles = ((a.m + 2 * kBM - 1) / (2 * kBM) + (a.offsets ? a.groups : 0)) * ((a.n + kPairN - 1) / kPairN);
  const int64_t pairs = dev.num_sms / 2;
  return launch_clusters_after(mxfp4_pair_kernel, (unsigned)(2 * (tiles < pairs ? tiles : pairs)), 2u, kPairThreads,
                               (size_t)kPairSmem, stream, ma, mb, a) == cudaSuccess
             ? FP8Q_OK
             : FP8Q_ERR_CUDA;
}

// Which kernel: a tile width for CTAs alone, and how many of them share a tile's k; or pairs.
// Modelled time in ns; each CTA runs `steps` stages for each of its tiles.  Measured (an SM at
// a time, then all of them):
//   a stage of a CTA alone takes 290 / 300 / 345 / 500 ns at 32 / 64 / 128 / 256 columns (the
//   wait, four MMAs of at least 50 ns, and with every SM busy the shared-memory traffic), so
//   the widest tile is the fastest per output as long as its tiles fill the SMs;
//   a tile's epilogue that no other tile's MMAs cover takes about 4 ns a column;
//   sharing k saves stages and costs the exchange of the sums: 1.2 us and 0.12 ns for each of
//   the tile's stored elements (1x4096x7168: 11.3 us unshared at 64 columns, 7.0 us with 4
//   CTAs at 128; 256x4096x4096: 7.9 us unshared at 64, 9.1 us with 2 at 128).  It is taken
//   within one wave only, where the clusters are resident together;
//   rows of out that do not start on 16 bytes take longer to store: 0.11 ns for each element of
//   a tile, by a pair 0.7 us (1003x2050x1408: 7.7 us at 128, 8.9 by pairs; 1500x2050x2048: 12.6 at
//   128, 10.2 by pairs);
//   a pair's stage takes 330 ns for twice the rows, its start 3.1 us more than a CTA's alone,
//   a change of tiles 0.7 us (8192x4096x7168: 86 us against 102 us at 256; 2048x4096x4096: 18.2
//   against 21.8; 1024x4096x4096: 11.9 both; 512x4096x4096: 11.2 against 9.3 at 128).
// With groups only the capacity m is known here.  A permute's capacity exceeds its pairs by at
// least 127 a group, so m - 127 * groups pairs are assumed, spread at random: a group without a
// pair has no tile, one with few has one, one with many ends half a tile late on average (one
// token to 8 of 32 experts, 2048x7168: 17.1 us at 128 by the 8 tiles expected, 20.5 at 256 by the
// 32 of the capacity; 512 tokens to 2 of 8, 4096x4096: 22 us by pairs, 26 at 256).
struct Variant {
  int bn, split;  // bn 0: pairs
};
Variant choose(int64_t m, int64_t n, int64_t k, bool grouped, int groups, int sms) {
  constexpr int kBn[4] = {256, 128, 64, 32};
  constexpr double kStage[4] = {500, 345, 300, 290};
  const int64_t steps = (k + kBK - 1) / kBK;
  Variant best = {256, 1};
  double least = 1e30;
  const double pairs = grouped ? (double)m - 127.0 * groups : 0.0;
  const double hit = grouped ? (pairs > 0 ? groups * (1.0 - std::exp(-pairs / groups)) : groups) : 0.0;
  auto row_tiles = [&](int rows) {  // of `rows` rows
    const int64_t all = (m + rows - 1) / rows + (grouped && rows > kBM ? groups / 2 : 0);
    if (pairs <= 0) return all;
    return std::min(all, (int64_t)std::ceil(std::max(hit, pairs / rows + hit / 2)));
  };
  for (int i = 0; i < 4; ++i) {
    const int64_t n_tiles = (n + kBn[i] - 1) / kBn[i], tiles = row_tiles(kBM) * n_tiles;
    const int64_t most = (m + kBM - 1) / kBM * n_tiles;  // a shared k takes CTAs for each of these
    for (int s = 1; s <= 4; s *= 2) {
      if (s > 1 && (most * s > sms || s > steps || kBn[i] == 32)) break;
      const double waves = (double)((tiles * s + sms - 1) / sms);
      double t = waves * (double)((steps + s - 1) / s) * kStage[i] + 4.0 * kBn[i] * (i == 0 ? waves : 1.0);
      const double stored = (double)(m < kBM ? m : kBM) * kBn[i];  // of a tile
      if (s > 1) t += 1200 + 0.12 * stored;
      else if (n % 8) t += waves * 0.11 * stored;
      if (t < least) {
        least = t;
        best = {kBn[i], s};
      }
    }
  }
  if (!grouped || groups <= kPairMaxGroups) {
    const int64_t tiles = row_tiles(2 * kBM) * ((n + kPairN - 1) / kPairN);
    const double waves = (double)((tiles + sms / 2 - 1) / (sms / 2));
    if (3100 + waves * ((double)steps * 330 + (n % 8 ? 1400 : 700)) < least) best = {0, 1};
  }
  return best;
}

}  // namespace
}  // namespace fp8q

using namespace fp8q;

extern "C" fp8q_status fp8q_debug_mxfp4_variant(int64_t m, int64_t n, int64_t k, int32_t num_groups, int32_t sms,
                                                int32_t* columns, int32_t* split) {
  if (m < 1 || n < 1 || k < 128 || k % 128 || num_groups < 0 || sms < 2) return FP8Q_ERR_ARG;
  if (!columns || !split) return FP8Q_ERR_NULL;
  const Variant v = choose(m, n, k, num_groups > 0, num_groups > 0 ? num_groups : 1, sms);
  *columns = v.bn;
  *split = v.split;
  return FP8Q_OK;
}

// A tile's sum over the largest k takes about 30 ms, far below the bound on the waits.
constexpr int64_t kMaxK = 1 << 24;

extern "C" fp8q_status fp8q_matmul_mxfp4(const uint8_t* aq, const uint8_t* asf, int64_t m, const uint8_t* bq,
                                         const uint8_t* bsf, int64_t n, int64_t k, const int32_t* group_offsets,
                                         int32_t num_groups, void* out, fp8q_stream_t stream) {
  if (m < 0 || n < 0 || k < 0 || k % 128 || m > kMaxInt32 || n > kMaxInt32 || k > kMaxK) return FP8Q_ERR_SHAPE;
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
  const int a_rows = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  const MatmulArgs a = {asf, bsf, group_offsets, static_cast<uint16_t*>(out), m, n, (int)k, num_groups, a_rows, dev.status};
  cudaStream_t st = to_stream(stream);
  const Variant v = choose(m, n, k, group_offsets != nullptr, num_groups, dev.num_sms);
  switch (v.bn * (v.split > 1 ? -1 : 1)) {
    case 0: return launch_pair(dev, aq, bq, a, st);
    case 32: return launch_matmul<32, 9, 2, false>(dev, aq, bq, a, 1, st);
    case 64: return launch_matmul<64, 8, 2, false>(dev, aq, bq, a, 1, st);
    case 128: return launch_matmul<128, 6, 2, false>(dev, aq, bq, a, 1, st);
    case 256: return launch_matmul<256, 4, 1, false>(dev, aq, bq, a, 1, st);
    case -64: return launch_matmul<64, 8, 2, true>(dev, aq, bq, a, v.split, st);
    case -128: return launch_matmul<128, 6, 2, true>(dev, aq, bq, a, v.split, st);
    default: return launch_matmul<256, 4, 1, true>(dev, aq, bq, a, v.split, st);
  }
}
