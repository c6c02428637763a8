// group_gemm.cu -- NVFP4 products grouped by expert, with ragged groups whose
// sizes only the device knows:
//   rows   D[r, :] = alpha A[r, :] . B_e^T   for the rows r of group e
//          (FPROP; DGRAD through the weights' transposed codes),
//   wgrad  D_e = alpha A[:, rows of e] . B[:, rows of e]^T
//          (the contraction runs over the group's rows).
// Group e owns rows offsets[e] .. offsets[e] + sizes[e] - 1; the offsets are
// multiples of 128, so a group starts on a scale atom of a row operand and on
// a whole number of scale atoms (64 elements) of a contraction.  Each CTA reads
// sizes and offsets once into a table in shared memory and walks its output
// tiles, group after group; no host round trip, one launch for all groups.
//
// Kernel (one CTA per SM, persistent): warp 0 the TMA producer, warp 1 the
// thread that copies scales to tensor memory and issues the MMAs
// (tcgen05.mma kind::mxf4nvf4, K = 64), warps 2..9 the epilogue, as in
// gemm.cu's single-SM kernel, whose waits, abort and drain rules hold here too.
// What differs: a tile's operand rows, contraction window and length come from
// the table; a contraction ends at the group's last whole atom of 64 (rows past
// a group's size hold zeros there); output rows past a group's size are
// written as zeros whatever A holds there, and so are the rows behind the
// last group; an empty group's weight gradient is zero.
#include "gemm_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kThreads = 320;  // producer, MMA, 8 epilogue warps
constexpr int kBM = 128;
constexpr int kAtom = 64;      // contraction elements per scale atom
constexpr int kMaxGroups = 512;

struct GroupArgs {
  const uint8_t* sfa;
  const uint8_t* sfb;
  const float* sdec_a;
  const float* sdec_b;
  void* D;
  const void* C;
  const int32_t* sizes;
  const int32_t* offsets;
  int groups;
  int rows;          // rows: rows of A and D; wgrad: the contraction's extent
  int M, N, K;       // wgrad: D_e is [M, N]; rows: N and the contraction K
  int kga, kgb;      // scale atoms per 128-row block of A, of B
  int nrb_b;         // 128-row blocks of B's scale tensor
  int num_m_blk;     // wgrad: tiles along M
  int num_n_blk;
  int b_row_step;    // rows: B rows from one group to the next (0 with the transposed view)
  int b_atom_step;   // rows: B scale atoms from one group to the next (transposed view)
};

enum { kRows = 0, kWgrad = 1 };

// Sizes, offsets and (rows) the running number of row blocks, in shared memory.
struct GroupTable {
  int size[kMaxGroups], off[kMaxGroups], first[kMaxGroups + 1];
};

// A group that does not lie in [0, rows), or starts inside a block of 128,
// counts as empty.
template <int KIND, int BM>
NVFP4_DEV void fill_table(GroupTable* t, const GroupArgs& a) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    int run = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 32) {
      const int g = g0 + lane;
      int size = 0, off = 0;
      if (g < a.groups) {
        size = a.sizes[g];
        off = a.offsets[g];
        if (size < 0 || off < 0 || off % 128 || off > a.rows || size > a.rows - off) size = off = 0;
      }
      const int blocks = (size + BM - 1) / BM;
      int s = blocks;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
      }
      if (g < a.groups) {
        t->size[g] = size;
        t->off[g] = off;
        t->first[g] = run + s - blocks;
      }
      run += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane == 0) t->first[a.groups] = run;
  }
}

template <int KIND>
NVFP4_DEV int num_tiles(const GroupTable* t, const GroupArgs& a) {
  return KIND == kRows ? t->first[a.groups] * a.num_n_blk
                       : a.groups * a.num_m_blk * a.num_n_blk;
}

// One output tile: rows of A and B, where the contraction starts in each (in
// scale atoms) and how many atoms it has, and where the tile lies in D.
struct Tile {
  int a_row, b_row, a_atom, b_atom, atoms;
  int64_t d_row;
  int d_col;
  int live;  // rows of the tile that belong to the group
};

// Tiles come in rising order, so the group is found by stepping on from the
// last one.  Within a group the row blocks run fastest: neighbouring CTAs
// share a tile of weights.
template <int KIND, int BM, int BN>
NVFP4_DEV Tile tile_at(int tile, int& g, const GroupTable* t, const GroupArgs& a) {
  Tile r;
  if (KIND == kRows) {
    while (tile >= t->first[g + 1] * a.num_n_blk) ++g;
    const int mb = t->first[g + 1] - t->first[g];
    const int local = tile - t->first[g] * a.num_n_blk;
    const int m = local % mb, n = local / mb;
    r.a_row = t->off[g] + m * BM;
    r.b_row = g * a.b_row_step + n * BN;
    r.a_atom = 0;
    r.b_atom = g * a.b_atom_step;
    r.atoms = a.K / kAtom;
    r.d_row = r.a_row;
    r.d_col = n * BN;
    r.live = t->size[g] - m * BM;
  } else {
    const int per = a.num_m_blk * a.num_n_blk;
    g = tile / per;
    const int local = tile - g * per;
    const int m = local % a.num_m_blk, n = local / a.num_m_blk;
    r.a_row = m * BM;
    r.b_row = n * BN;
    r.a_atom = r.b_atom = t->off[g] / kAtom;
    r.atoms = (t->size[g] + kAtom - 1) / kAtom;
    r.d_row = (int64_t)g * a.M + r.a_row;
    r.d_col = n * BN;
    r.live = BM;
  }
  return r;
}

// Thirty-two columns of one row of D from FP32 accumulators.  A row that is
// not live is written as zero (as C alone where C is added).
template <int DMODE>
NVFP4_DEV void store_cols(const GroupArgs& a, int64_t row, int col0, const uint32_t (&r)[32],
                          float alpha, bool live) {
  if (DMODE == NVFP4_D_F32_ACCUM) {
    float* D = static_cast<float*>(a.D) + row * a.N + col0;
#pragma unroll
    for (int g0 = 0; g0 < 8; g0 += 4) {
      float4 d[4];
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (col0 + (g0 + g) * 4 < a.N) d[g] = *reinterpret_cast<const float4*>(D + (g0 + g) * 4);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (col0 + (g0 + g) * 4 >= a.N) break;
        const uint32_t* v = r + (g0 + g) * 4;
        d[g].x = fmaf(alpha, __uint_as_float(v[0]), d[g].x);
        d[g].y = fmaf(alpha, __uint_as_float(v[1]), d[g].y);
        d[g].z = fmaf(alpha, __uint_as_float(v[2]), d[g].z);
        d[g].w = fmaf(alpha, __uint_as_float(v[3]), d[g].w);
        *reinterpret_cast<float4*>(D + (g0 + g) * 4) = d[g];
      }
    }
    return;
  }
  __nv_bfloat16* D = static_cast<__nv_bfloat16*>(a.D) + row * a.N + col0;
  const __nv_bfloat16* Cp = static_cast<const __nv_bfloat16*>(a.C) + row * a.N + col0;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (col0 + g * 8 >= a.N) break;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = live ? __fmul_rn(__uint_as_float(r[g * 8 + e]), alpha) : 0.0f;
    if (DMODE == NVFP4_D_BF16_ADD_C && live) {
      const uint4 c = *reinterpret_cast<const uint4*>(Cp + g * 8);
      const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = __fadd_rn(f[2 * e], __uint_as_float(cw[e] << 16));
        f[2 * e + 1] = __fadd_rn(f[2 * e + 1], __uint_as_float(cw[e] & 0xFFFF0000u));
      }
    }
    uint4 o;
    o.x = pack_bf16x2(f[0], f[1]);
    o.y = pack_bf16x2(f[2], f[3]);
    o.z = pack_bf16x2(f[4], f[5]);
    o.w = pack_bf16x2(f[6], f[7]);
    *reinterpret_cast<uint4*>(D + g * 8) = o;
  }
}

// The rows of D behind the last group become zero (thread `i` of `n`).
NVFP4_DEV void clear_tail(const GroupArgs& a, int64_t i, int64_t n) {
  int64_t first = a.offsets[a.groups];
  first = first < 0 ? 0 : first > a.rows ? a.rows : first;
  uint4* D = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.D) + first * a.N);
  const int64_t count = (a.rows - first) * (a.N / 8);
  for (; i < count; i += n) D[i] = make_uint4(0u, 0u, 0u, 0u);
}

template <int BN, int STAGES>
struct GroupSmem {
  static constexpr int kAt = 4;  // scale atoms per stage (256 elements of K)
  static constexpr uint32_t kA = kBM * kBKBytes, kB = BN * kBKBytes;
  static constexpr uint32_t kSFA = kAt * 512, kSFB = (BN / 128) * kAt * 512;
  static constexpr uint32_t offA = 0, offB = offA + STAGES * kA;
  static constexpr uint32_t offSFA = offB + STAGES * kB, offSFB = offSFA + STAGES * kSFA;
  static constexpr uint32_t offBar = offSFB + STAGES * kSFB;
  static constexpr uint32_t kNumBars = 2 * STAGES + 3;  // full, empty, acc full, acc empty, drain
  static constexpr uint32_t offMisc = offBar + kNumBars * 8;
  static constexpr uint32_t offTable = offMisc + 16;
  static constexpr uint32_t kBytes = offTable + sizeof(GroupTable);
  static constexpr uint32_t kAlloc = kBytes + 1024;  // room to align the base to 1024
  static constexpr uint32_t kSfCol0 = BN;
  static constexpr uint32_t kSfColsPerStage = 16 + BN / 8;
  static_assert(kSfCol0 + STAGES * kSfColsPerStage <= kTmemCols, "tensor memory overflow");
  static_assert(kAlloc <= 232448, "shared memory overflow");
};

template <int KIND, int BN, int STAGES, int DMODE>
__global__ void __launch_bounds__(kThreads, 1)
    group_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB, const GroupArgs args) {
  using L = GroupSmem<BN, STAGES>;
  constexpr int kAt = L::kAt;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::offBar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t acc_full = bar0 + 8u * (2 * STAGES);
  const uint32_t acc_empty = acc_full + 8;
  const uint32_t drain_bar = acc_full + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::offMisc + 4);
  GroupTable* table = reinterpret_cast<GroupTable*>(smem + L::offTable);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 8);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  fill_table<KIND, kBM>(table, args);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles = num_tiles<KIND>(table, args);

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      uint32_t s = 0, ph = 0;
      int g = 0;
      int armed[STAGES];
      for (int i = 0; i < STAGES; ++i) armed[i] = -1;
      // injected stall: no loads, so the MMA thread's first wait runs out
      bool ok = *reinterpret_cast<volatile unsigned int*>(&g_gemm_stall) == 0u;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const Tile t = tile_at<KIND, kBM, BN>(tile, g, table, args);
        const int num_kb = (t.atoms + kAt - 1) / kAt;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!wait_bounded(empty_bar(s), ph ^ 1u, abort_flag, 0x10u)) {
            ok = false;
            break;
          }
          const int natoms = min(kAt, t.atoms - kb * kAt);
          const int a_at = t.a_atom + kb * kAt, b_at = t.b_atom + kb * kAt;
          const int rb_b = t.b_row >> 7;
          const int nb = min(BN / 128, args.nrb_b - rb_b);
          mbar_arrive_expect_tx(full_bar(s),
                                L::kA + L::kB + (uint32_t)natoms * 512u * (1u + (uint32_t)nb));
          armed[s] = (int)ph;
          tma_load_2d(sbase + L::offA + s * L::kA, &tmA, full_bar(s), a_at * (kAtom / 2), t.a_row);
          tma_load_2d(sbase + L::offB + s * L::kB, &tmB, full_bar(s), b_at * (kAtom / 2), t.b_row);
          bulk_load(sbase + L::offSFA + s * L::kSFA,
                    args.sfa + ((int64_t)(t.a_row >> 7) * args.kga + a_at) * 512, natoms * 512u,
                    full_bar(s));
          for (int j = 0; j < nb; ++j)
            bulk_load(sbase + L::offSFB + s * L::kSFB + j * (kAt * 512),
                      args.sfb + ((int64_t)(rb_b + j) * args.kgb + b_at) * 512, natoms * 512u,
                      full_bar(s));
          if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
      }
      if (!ok) {  // let the copies already issued land before the CTA exits
        for (int i = 0; i < STAGES; ++i)
          if (armed[i] >= 0) wait_drain(full_bar(i), (uint32_t)armed[i]);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------------- MMA
      constexpr uint32_t idesc = idesc_nvf4(kBM, BN);
      uint32_t s = 0, ph = 0, acc_ph = 0;
      int g = 0;
      bool ok = true, issued = false;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const Tile t = tile_at<KIND, kBM, BN>(tile, g, table, args);
        if (t.atoms == 0) continue;
        if (!wait_bounded(acc_empty, acc_ph ^ 1u, abort_flag, 0x20u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int num_kb = (t.atoms + kAt - 1) / kAt;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!wait_bounded(full_bar(s), ph, abort_flag, 0x21u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int natoms = min(kAt, t.atoms - kb * kAt);
          const uint32_t sfa_t = tmem + L::kSfCol0 + s * L::kSfColsPerStage;
          const uint32_t sfb_t = sfa_t + 16;
          const uint32_t sa = sbase + L::offSFA + s * L::kSFA;
          const uint32_t sb = sbase + L::offSFB + s * L::kSFB;
          const uint32_t a0 = sbase + L::offA + s * L::kA;
          const uint32_t b0 = sbase + L::offB + s * L::kB;
          for (int j = 0; j < natoms; ++j) {
            tc_cp_32x128b_warpx4(sfa_t + 4 * j, smem_desc_sf(sa + j * 512));
#pragma unroll
            for (int b = 0; b < BN / 128; ++b)
              tc_cp_32x128b_warpx4(sfb_t + j * (BN / 32) + 4 * b,
                                   smem_desc_sf(sb + b * (kAt * 512) + j * 512));
            tc_mma_nvf4(tmem, smem_desc_sw128(a0 + 32 * j), smem_desc_sw128(b0 + 32 * j), idesc,
                        sfa_t + 4 * j, sfb_t + j * (BN / 32), (kb | j) != 0 ? 1u : 0u);
          }
          issued = true;
          tc_commit(empty_bar(s));
          if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        tc_commit(acc_full);
        acc_ph ^= 1u;
      }
      if (!ok && issued) {  // MMAs in flight must finish before tensor memory is freed
        tc_commit(drain_bar);
        wait_drain(drain_bar, 0);
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    constexpr int kCols = BN / 2, kChunks = kCols / 32;
    const int q = warp & 3, h = (warp - 2) >> 2;
    const float alpha = __fmul_rn(__ldg(args.sdec_a), __ldg(args.sdec_b));
    uint32_t acc_ph = 0;
    int g = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const Tile t = tile_at<KIND, kBM, BN>(tile, g, table, args);
      const int64_t row = t.d_row + q * 32 + lane;
      const bool live = q * 32 + lane < t.live;
      uint32_t r[kChunks][32];
      if (t.atoms > 0) {
        if (!wait_bounded(acc_full, acc_ph, abort_flag, 0x30u)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * kCols + c * 32), r[c]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
        acc_ph ^= 1u;
      } else if (DMODE == NVFP4_D_F32_ACCUM) {
        continue;  // nothing to add
      } else {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) r[c][e] = 0u;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int col0 = t.d_col + h * kCols + c * 32;
        if (col0 < args.N) store_cols<DMODE>(args, row, col0, r[c], alpha, live);
      }
    }
    if (KIND == kRows && ok)
      clear_tail(args, (int64_t)blockIdx.x * 256 + threadIdx.x - 64, (int64_t)gridDim.x * 256);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int KIND, int BN, int STAGES, int DMODE>
nvfp4_status launch_group(const CUtensorMap& ma, const CUtensorMap& mb, const GroupArgs& a,
                          int sms, cudaStream_t stream) {
  using L = GroupSmem<BN, STAGES>;
  auto kern = group_gemm_kernel<KIND, BN, STAGES, DMODE>;
  static GemmLaunchState ls;
  if (gemm_setup(ls, kern, L::kAlloc, kThreads, 0, false, sms) <= 0) return NVFP4_ERR_CUDA;
  return cuda_status(launch_pdl(kern, sms, kThreads, L::kAlloc, stream, ma, mb, a));
}

nvfp4_status check_groups(const nvfp4_tensor* A, const nvfp4_tensor* B, const int32_t* sizes,
                          const int32_t* offsets, int32_t groups, const void* D) {
  if (!A || !B || !sizes || !offsets || !D) return NVFP4_ERR_INVALID_ARG;
  if (!A->codes || !A->scales || !A->s_dec || !B->s_dec) return NVFP4_ERR_INVALID_ARG;
  if (groups < 1 || groups > kMaxGroups) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

nvfp4_status group_set_injection(unsigned int stall, unsigned long long wait_ns) {
  if (cudaMemcpyToSymbol(g_gemm_stall, &stall, sizeof(stall)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_gemm_wait_ns, &wait_ns, sizeof(wait_ns)) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return NVFP4_OK;
}

nvfp4_status group_read_error(unsigned int* code) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemm_error, sizeof(v)) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (v && cudaMemcpyToSymbol(g_gemm_error, &zero, sizeof(zero)) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  *code = v;
  return NVFP4_OK;
}

nvfp4_status group_gemm_impl(const nvfp4_tensor* A, const nvfp4_tensor* B, int32_t b_view,
                             const int32_t* sizes, const int32_t* offsets, int32_t groups,
                             void* D, int32_t d_mode, const void* C, int64_t rows, int64_t N,
                             int64_t K, cudaStream_t stream) {
  nvfp4_status st = check_groups(A, B, sizes, offsets, groups, D);
  if (st != NVFP4_OK) return st;
  if (b_view < 0 || b_view > 1) return NVFP4_ERR_INVALID_ARG;
  if (d_mode != NVFP4_D_BF16 && d_mode != NVFP4_D_BF16_ADD_C) return NVFP4_ERR_INVALID_ARG;
  if ((d_mode == NVFP4_D_BF16_ADD_C) != (C != nullptr)) return NVFP4_ERR_INVALID_ARG;
  const void* b_codes = b_view ? B->codes_t : B->codes;
  const void* b_sf = b_view ? B->scales_t : B->scales;
  if (!b_codes || !b_sf) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || rows % 128 || N <= 0 || N % 128 || K <= 0 || K % 64) return NVFP4_ERR_SHAPE;
  if (rows > INT32_MAX - 256 || groups * N > INT32_MAX || groups * K > INT32_MAX)
    return NVFP4_ERR_SHAPE;
  if (A->rows != rows || A->cols != K) return NVFP4_ERR_SHAPE;
  if (b_view ? (B->rows != groups * K || B->cols != N) : (B->rows != groups * N || B->cols != K))
    return NVFP4_ERR_SHAPE;
  if (!aligned16(A->codes) || !aligned16(A->scales) || !aligned16(b_codes) || !aligned16(b_sf) ||
      !aligned16(D) || !aligned16(C) || !aligned4(sizes) || !aligned4(offsets))
    return NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  GroupArgs a = {};
  a.sfa = static_cast<const uint8_t*>(A->scales);
  a.sfb = static_cast<const uint8_t*>(b_sf);
  a.sdec_a = A->s_dec;
  a.sdec_b = B->s_dec;
  a.D = D;
  a.C = C;
  a.sizes = sizes;
  a.offsets = offsets;
  a.groups = groups;
  a.rows = (int)rows;
  a.N = (int)N;
  a.K = (int)K;
  const int64_t b_rows = b_view ? N : groups * N, b_cols = b_view ? groups * K : K;
  a.kga = (int)(K / kAtom);
  a.kgb = (int)(b_cols / kAtom);
  a.nrb_b = (int)(b_rows / 128);
  a.b_row_step = b_view ? 0 : (int)N;
  a.b_atom_step = b_view ? (int)(K / kAtom) : 0;
  a.num_n_blk = (int)((N + 255) / 256);
  CUtensorMap ma, mb;
  if (!make_code_map(&ma, A->codes, rows, K / 2, kBM) ||
      !make_code_map(&mb, b_codes, b_rows, b_cols / 2, 256))
    return NVFP4_ERR_CUDA;
  return d_mode == NVFP4_D_BF16
             ? launch_group<kRows, 256, 4, NVFP4_D_BF16>(ma, mb, a, dev.sm_count, stream)
             : launch_group<kRows, 256, 4, NVFP4_D_BF16_ADD_C>(ma, mb, a, dev.sm_count, stream);
}

nvfp4_status group_wgrad_impl(const nvfp4_tensor* A, const nvfp4_tensor* B, const int32_t* sizes,
                              const int32_t* offsets, int32_t groups, void* D, int32_t d_mode,
                              int64_t M, int64_t N, int64_t rows, cudaStream_t stream) {
  nvfp4_status st = check_groups(A, B, sizes, offsets, groups, D);
  if (st != NVFP4_OK) return st;
  if (!B->codes || !B->scales) return NVFP4_ERR_INVALID_ARG;
  if (d_mode != NVFP4_D_BF16 && d_mode != NVFP4_D_F32_ACCUM) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || rows % 128 || M <= 0 || M % 128 || N <= 0 || N % 128) return NVFP4_ERR_SHAPE;
  if (rows > INT32_MAX - 256 || M > INT32_MAX - 256 || N > INT32_MAX - 256) return NVFP4_ERR_SHAPE;
  if ((M / 128) * (N / 128) * groups > INT32_MAX - 1024) return NVFP4_ERR_SHAPE;
  if (A->rows != M || A->cols != rows || B->rows != N || B->cols != rows) return NVFP4_ERR_SHAPE;
  if (!aligned16(A->codes) || !aligned16(A->scales) || !aligned16(B->codes) ||
      !aligned16(B->scales) || !aligned16(D) || !aligned4(sizes) || !aligned4(offsets))
    return NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  GroupArgs a = {};
  a.sfa = static_cast<const uint8_t*>(A->scales);
  a.sfb = static_cast<const uint8_t*>(B->scales);
  a.sdec_a = A->s_dec;
  a.sdec_b = B->s_dec;
  a.D = D;
  a.sizes = sizes;
  a.offsets = offsets;
  a.groups = groups;
  a.rows = (int)rows;
  a.M = (int)M;
  a.N = (int)N;
  a.kga = a.kgb = (int)(rows / kAtom);
  a.nrb_b = (int)(N / 128);
  a.num_m_blk = (int)(M / kBM);
  a.num_n_blk = (int)((N + 255) / 256);
  CUtensorMap ma, mb;
  if (!make_code_map(&ma, A->codes, M, rows / 2, kBM) ||
      !make_code_map(&mb, B->codes, N, rows / 2, 256))
    return NVFP4_ERR_CUDA;
  return d_mode == NVFP4_D_BF16
             ? launch_group<kWgrad, 256, 4, NVFP4_D_BF16>(ma, mb, a, dev.sm_count, stream)
             : launch_group<kWgrad, 256, 4, NVFP4_D_F32_ACCUM>(ma, mb, a, dev.sm_count, stream);
}

}  // namespace nvfp4
