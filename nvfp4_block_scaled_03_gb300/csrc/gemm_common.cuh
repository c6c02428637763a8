// gemm_common.cuh -- what the block-scaled GEMM kernels share: the bounded
// mbarrier waits with their error word, shared-memory descriptors, the
// tensor-store epilogue box, the tensor maps and the once-per-kernel launch
// set-up.  Each translation unit that includes it has its own error word and
// injection switches.
#pragma once

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace nvfp4 {

static __device__ unsigned int g_gemm_error;
// Failure injection for tests of the bounded waits (nvfp4_debug_inject):
// while bit 0 of g_gemm_stall is set the producers of every GEMM kernel issue
// no loads; while bit 1 is set the MMA threads give up before their first
// wait, the producers' loads in flight.  The pipeline waits give up after
// g_gemm_wait_ns.
static __device__ unsigned int g_gemm_stall;
static __device__ unsigned long long g_gemm_wait_ns = 2000000000ull;

namespace {

constexpr uint64_t kWaitTimeoutNs = 2000000000ull;
constexpr int kBKBytes = 128;       // K bytes per stage (256 FP4 elements)
constexpr uint32_t kTmemCols = 512;

// K-major operand descriptor for a stage row width of BKB bytes (128-byte or
// 64-byte swizzle; 8-row swizzle atoms stacked 8*BKB bytes apart).
template <int BKB>
NVFP4_DEV uint64_t smem_desc_kmajor(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)((8 * BKB) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(BKB == 128 ? 2 : 4) << 61;  // SWIZZLE_128B or SWIZZLE_64B
  return d;
}


// Drain wait used after an abort: bounded, ignores the abort flag.
NVFP4_DEV void wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
      atomicCAS(&g_gemm_error, 0u, 0xDEu);
      return;
    }
  }
}

// Bounded wait of the single-SM kernel: on expiry it raises the CTA's abort
// flag and records `code` in the error word.
NVFP4_DEV bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                            unsigned int code) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  const uint64_t limit = *reinterpret_cast<volatile unsigned long long*>(&g_gemm_wait_ns);
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit) {
      *abort_flag = 1;
      atomicCAS(&g_gemm_error, 0u, code);
      return false;
    }
  }
}

NVFP4_DEV uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Bounded wait for the pair: a timeout also raises the peer CTA's abort flag.
NVFP4_DEV bool wait_bounded_pair(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                 uint32_t peer_abort_addr, unsigned int code) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  const uint64_t limit = *reinterpret_cast<volatile unsigned long long*>(&g_gemm_wait_ns);
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit) {
      *abort_flag = 1;
      st_cluster_u32(peer_abort_addr, 1u);
      atomicCAS(&g_gemm_error, 0u, code);
      return false;
    }
  }
}

// The injection switches, which thread 0 of a CTA puts into shared memory before
// the roles start.
enum : uint32_t { kStall = 1, kQuit = 2 };
NVFP4_DEV uint32_t injected() {
  return *reinterpret_cast<volatile unsigned int*>(&g_gemm_stall) & 3u;
}
// Injected quit: the caller gives up as if its first wait had run out.
NVFP4_DEV bool quits(uint32_t injected, volatile int* abort_flag) {
  if (!(injected & kQuit)) return false;
  *abort_flag = 1;
  atomicCAS(&g_gemm_error, 0u, 0x52u);
  return true;
}
NVFP4_DEV bool quits_pair(uint32_t injected, volatile int* abort_flag, uint32_t peer_abort_addr) {
  if (!quits(injected, abort_flag)) return false;
  st_cluster_u32(peer_abort_addr, 1u);
  return true;
}

// After an abort, once every role has stopped: until the last copy into each
// of S stages has landed.  Fill f of `fills` went to stage f % S.
template <int S>
NVFP4_DEV void drain_stages(uint32_t bars, uint32_t fills) {
#pragma unroll 1
  for (uint32_t s = 0; s < (uint32_t)S && s < fills; ++s)
    wait_drain(bars + 8u * s, ((fills - 1 - s) / S) & 1u);
}
// The same for the full barriers of a pair, on which the leader counts the
// copies of both CTAs (`bytes` a fill from each).  Their producers may have
// stopped at different fills: of those that only the peer issued the arrival
// is missing, of those that it did not issue its bytes.
template <int S>
NVFP4_DEV void drain_pair_stages(uint32_t bars, uint32_t mine, uint32_t peers, uint32_t bytes) {
#pragma unroll 1
  for (uint32_t f = mine; f < peers; ++f) mbar_arrive_expect_tx(bars + 8u * (f % S), bytes);
#pragma unroll 1
  for (uint32_t f = peers; f < mine; ++f) mbar_complete_tx(bars + 8u * (f % S), bytes);
  drain_stages<S>(bars, max(mine, peers));
}

// The last barriers of a pair kernel, behind which it frees its tensor memory.  If
// it has given up, its copies and MMAs in flight finish first: every role of
// every CTA in the cluster has stopped by then.  L lays out the shared memory:
// at offMisc + 4 the abort flag, + 8 the stages that this CTA's producer filled,
// + 12 a byte for each of warps 1 to 3 (behind the injection switches) that says
// whether it issued MMAs or scale copies; from offBar on S full, empty,
// scales-ready and scales-landed barriers, two of the accumulator, the drains'.
// `bytes`: what a fill by one CTA puts on the leader's full barrier.  SCALES: its
// scales land on a barrier of its own.  (The addresses are computed anew: kept
// through the kernel they cost the epilogue registers.)
template <class L, int S, int CLUSTER, bool SCALES>
NVFP4_DEV void pair_leave(uint32_t bytes) {
  extern __shared__ uint8_t smem_raw[];
  uint32_t base = smem_u32(smem_raw);
  asm volatile("" : "+r"(base));
  base = (base + 1023u) & ~1023u;
  const uint32_t misc = base + L::offMisc, bars = base + L::offBar;
  __syncthreads();
  // a flag raised in one pair of a larger cluster holds for all of it
  if (CLUSTER > 2 && ld_shared_u32(misc + 4) && threadIdx.x < CLUSTER)
    st_cluster_u32(mapa_shared(misc + 4, threadIdx.x), 1u);
  cluster_sync();
  if (!ld_shared_u32(misc + 4)) return;
  const uint32_t crank = cluster_ctarank(), warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    const uint32_t fills = ld_shared_u32(misc + 8);
    if ((crank & 1u) == 0)
      drain_pair_stages<S>(bars, fills, ld_cluster_u32(mapa_shared(misc + 8, crank ^ 1u)), bytes);
    if (SCALES) drain_stages<S>(bars + 8u * 3 * S, fills);
  } else if ((threadIdx.x & 31) == 0 && warp <= 3 &&
             (ld_shared_u32(misc + 12) >> (8 * warp) & 0xFFu)) {
    const uint32_t bar = bars + 8u * (4 * S + 2 + warp - 1);
    tc_commit_pair(bar, (uint16_t)(1u << crank));
    wait_drain(bar, 0);
  }
  __syncthreads();
  cluster_sync();
}

// Pulls the part of D that a row of a later tile's epilogue reads (128-byte
// lines from col0 on, `bytes` of them) into L2 while the tile's MMAs run.
NVFP4_DEV void prefetch_l2_row(const void* p, int bytes) {
  const char* c = static_cast<const char*>(p);
  for (int o = 0; o < bytes; o += 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(c + o)));
}

// Epilogue helper: one warp's 32 rows x 32 bf16 columns (lane = row, 16
// packed pairs) into its staging box, then one tensor store at (x, y).  The
// box is rewritten only after the previous store has read it; the 16-byte
// pieces are rotated so a warp's writes hit distinct banks.
NVFP4_DEV void store_box_bf16(uint8_t* box, int lane, const uint32_t (&pk)[16],
                              const CUtensorMap* tmD, int32_t x, int32_t y) {
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
#pragma unroll
  for (int pc = 0; pc < 4; ++pc) {
    const int piece = (pc + (lane >> 1)) & 3;
    uint4 v;
    switch (piece) {
      case 0: v = make_uint4(pk[0], pk[1], pk[2], pk[3]); break;
      case 1: v = make_uint4(pk[4], pk[5], pk[6], pk[7]); break;
      case 2: v = make_uint4(pk[8], pk[9], pk[10], pk[11]); break;
      default: v = make_uint4(pk[12], pk[13], pk[14], pk[15]); break;
    }
    *reinterpret_cast<uint4*>(box + lane * 64 + piece * 16) = v;
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(tmD, smem_u32(box), x, y);
    bulk_commit_group();
  }
}

// ---- host side -----------------------------------------------------------------
inline EncodeTiledFn encode_fn() { return tensor_map_encoder(); }

// 2-D map over a K-major code matrix [rows, kbytes] with a box of box_bytes
// (128: 128-byte swizzle, 64: 64-byte swizzle) x box_rows.
inline bool make_code_map(CUtensorMap* map, const void* base, int64_t rows, int64_t kbytes,
                   int box_rows, int box_bytes = kBKBytes) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kbytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kbytes};
  const cuuint32_t box[2] = {(cuuint32_t)box_bytes, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D map over a scale tensor viewed as rows of 128 bytes (4 rows per atom),
// box of 16 rows (the 4 atoms of one stage).
inline bool make_sf_map(CUtensorMap* map, const void* base, size_t bytes, int box_rows = 16) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {128, (cuuint64_t)(bytes / 128)};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D map over a bf16 output [rows, cols] with 32 x 32 boxes (no swizzle);
// tensor stores skip the part of a box outside the matrix.
inline bool make_out_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(cols * 2)};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Per-device, once-per-kernel launch set-up of a GEMM kernel, under a lock:
// its dynamic shared memory attribute, for a kernel that splits registers
// with setmaxnreg the check that the compiled count covers the split
// (setmaxnreg.inc waits until the registers it asks for are free in the
// block's launch allotment, so a split above it would wait forever), and
// for a kernel on clusters how many are resident at once (cluster placement
// can leave SMs of a GPC over).  Returns the resident clusters (1 for a
// single-SM kernel, `cluster` 1), 0 when the set-up failed.
struct GemmLaunchState {
  std::mutex mu;
  int resident[64] = {};  // per device: 0 not yet set up, -1 refused for good
};

template <typename K>
int gemm_setup(GemmLaunchState& ls, K kern, uint32_t smem, int threads, int split_regs,
               int cluster, int sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(ls.mu);
  if (ls.resident[dev] == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess)
      return 0;
    if (split_regs > 0) {
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return 0;
      if (fa.numRegs * threads < split_regs) {
        ls.resident[dev] = -1;  // the compiled kernel can never run
        return 0;
      }
    }
    int n = 1;
    if (cluster > 1) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(cluster * (sms / cluster));
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = cluster;
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      const bool known = cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0;
      if (!known && cluster > 2) {  // no room for such clusters: the caller has another way
        cudaGetLastError();
        ls.resident[dev] = -1;
        return 0;
      }
      n = known ? std::min(n, sms / cluster) : sms / cluster;
    }
    ls.resident[dev] = n;
  }
  return ls.resident[dev] > 0 ? ls.resident[dev] : 0;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace nvfp4
