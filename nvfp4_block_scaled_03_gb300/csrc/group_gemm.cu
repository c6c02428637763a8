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
// The kernels follow gemm.cu's (persistent CTAs; a TMA producer, MMA, scale and
// epilogue warps around a ring of stages; tcgen05.mma kind::mxf4nvf4, K = 64) and
// its rules on waits, aborts and drains.  What differs: a tile's operand rows,
// contraction window and length come from the table; a contraction ends at the
// group's last whole atom of 64 (rows past a group's size hold zeros there);
// output rows past a group's size are written as zeros whatever A holds there,
// and so are the rows behind the last group; an empty group's weight gradient
// is zero.
#include "gemm_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kBM = 256;       // rows of a CTA pair's tile
constexpr int kAtom = 64;      // contraction elements per scale atom
constexpr int kMaxGroups = 512;

struct GroupArgs {
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
      const int blocks = (size + kBM - 1) / kBM;
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
template <int KIND, int BN>
NVFP4_DEV Tile tile_at(int tile, int& g, const GroupTable* t, const GroupArgs& a) {
  Tile r;
  if (KIND == kRows) {
    while (tile >= t->first[g + 1] * a.num_n_blk) ++g;
    const int mb = t->first[g + 1] - t->first[g];
    const int local = tile - t->first[g] * a.num_n_blk;
    const int m = local % mb, n = local / mb;
    r.a_row = t->off[g] + m * kBM;
    r.b_row = g * a.b_row_step + n * BN;
    r.a_atom = 0;
    r.b_atom = g * a.b_atom_step;
    r.atoms = a.K / kAtom;
    r.d_row = r.a_row;
    r.d_col = n * BN;
    r.live = t->size[g] - m * kBM;
  } else {
    const int per = a.num_m_blk * a.num_n_blk;
    g = tile / per;
    const int local = tile - g * per;
    const int m = local % a.num_m_blk, n = local / a.num_m_blk;
    r.a_row = m * kBM;
    r.b_row = n * BN;
    r.a_atom = r.b_atom = t->off[g] / kAtom;
    r.atoms = (t->size[g] + kAtom - 1) / kAtom;
    r.d_row = (int64_t)g * a.M + r.a_row;
    r.d_col = n * BN;
    r.live = a.M - r.a_row;
  }
  return r;
}

// The rows of D behind the last group become zero (thread `i` of `n`).
NVFP4_DEV void clear_tail(const GroupArgs& a, int64_t i, int64_t n) {
  int64_t first = a.offsets[a.groups];
  first = first < 0 ? 0 : first > a.rows ? a.rows : first;
  uint4* D = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.D) + first * a.N);
  const int64_t count = (a.rows - first) * (a.N / 8);
  for (; i < count; i += n) D[i] = make_uint4(0u, 0u, 0u, 0u);
}

// =============================================================================
// CTA-pair kernel: tiles of 256 x BN (BN = 256 or 384) on a cluster of two SMs
// (tcgen05 cta_group::2).  As gemm.cu's pair kernels: CTA r loads rows [128 r,
// 128 r + 128) of A's 256 and its half of B's rows, four scale warps of each CTA
// store the stage's scales into tensor memory, the leader issues the MMAs (a
// second MMA warp takes the last 128 columns of a 384-wide tile), and 8 epilogue
// warps of each CTA drain its 128 rows.  Of a 256-row tile whose group ends in its first half, and of
// the last tile of an M that is an odd multiple of 128, the second CTA stores
// nothing.
//
// With SK > 1 a cluster holds SK pairs, which share a tile: pair i takes the
// i-th part of the contraction, then the others hand their FP32 sums of the
// rows that are the group's to pair 0 through its shared memory (the ring is
// idle by then), which adds them in order and stores.  For a few tiles with
// long contractions, which would leave most SMs idle.
//
// Outputs leave through shared-memory boxes of 32 rows x 32 columns and tensor
// stores; the FP32 fold as tensor reductions (one FP32 add in L2 for each
// element, subnormals flushed there), so D is never read into the SM.
//
// What bounds it, and measured: long contractions the stages' 48 KB into each SM
// and the scales' stores (16384 rows, 8 groups, 4096 x 14336: 320 us alone, 6.0
// PF/s; 281 without scales; the dense kernel takes 304), few rows the weights'
// bytes (2 rows of the same, 73 MB: 19.5 us, 11 at the copy rate).  Weight
// gradients have a few stages a tile: 64 x [1024, 2048] bf16 over 32000 rows take
// 70 us (324 MB, 4.6 TB/s), 57 without stores, 63 without MMAs; the fold of 16384
// rows into 8 x [4096, 2048] takes 123 (593 MB, 4.8 TB/s), 66 without its
// reductions.  256 x 128 tiles with two accumulators took 88 and 151 there; more
// boxes a warp or 128-byte box rows changed nothing.
// =============================================================================
template <int BN, int DMODE, int SK>
struct PairGroup {
  static constexpr bool kF32 = DMODE == NVFP4_D_F32_ACCUM;
  static constexpr bool kAddC = DMODE == NVFP4_D_BF16_ADD_C && SK == 1 && BN == 256;
  static constexpr int kAt = 4, kRowBlocks = BN / 128;
  static constexpr int kStages = BN == 384 || kF32 || kAddC ? 4 : 5;
  static constexpr int kBoxes = kAddC ? 4 : 1;  // of an epilogue warp
  static constexpr int kMmaWarps = BN == 384 ? 2 : 1;
  static constexpr uint32_t kA = 128 * kBKBytes, kB = (BN / 2) * kBKBytes;
  static constexpr uint32_t kSFA = kAt * 512, kSFB = kRowBlocks * kAt * 512;
  static constexpr uint32_t kBox = 32 * (kF32 ? 128 : 64);
  static constexpr uint32_t offA = 0, offB = offA + kStages * kA;
  static constexpr uint32_t offStore = offB + kStages * kB;
  static constexpr uint32_t offSFA = offStore + 8 * kBoxes * kBox;
  static constexpr uint32_t offSFB = offSFA + kStages * kSFA;
  static constexpr uint32_t offBar = offSFB + kStages * kSFB;
  // full, empty, scales-ready, scales-landed per stage; acc full, acc empty;
  // a drain barrier per MMA warp; a barrier per epilogue warp for its part of C
  static constexpr uint32_t kNumBars = 4 * kStages + 2 + kMmaWarps + (kAddC ? 8 : 0);
  static constexpr uint32_t offMisc = offBar + kNumBars * 8;
  static constexpr uint32_t offTable = offMisc + 16;
  static constexpr uint32_t kBytes = offTable + sizeof(GroupTable);
  static constexpr uint32_t kAlloc = kBytes + 1024;
  // tensor memory: the accumulator, then scale slots of [B rows 256..: 4 per
  // atom] [A: 4 per atom] [B rows 0..255: 8 per atom] columns
  static constexpr uint32_t kSfCol0 = BN;
  static constexpr uint32_t kColA = BN == 384 ? 16 : 0, kColB01 = kColA + 16;
  static constexpr uint32_t kSlotCols = kColB01 + 32;
  static constexpr int kSlots = BN == 384 ? 2 : kStages;
  static constexpr int kThreads = 512;
  static constexpr int kRegsIssue = 88, kRegsEpilogue = 168;
  static constexpr int kSplitRegs = 2 * 128 * kRegsIssue + 2 * 128 * kRegsEpilogue;
  static_assert(kSfCol0 + kSlots * kSlotCols <= kTmemCols, "tensor memory overflow");
  static_assert(kAlloc <= 232448, "shared memory overflow");
  static_assert(kSplitRegs <= kThreads * 128, "register split exceeds the launch's");
  static_assert(offStore % 1024 == 0, "store boxes start on their swizzle's period");
  static_assert(BN == 256 || (BN == 384 && !kF32), "tile");
  // a part's sums in the ring of pair 0: rows padded by 16 bytes, so that the
  // 16-byte pieces of 8 rows hit distinct banks
  [[maybe_unused]] static constexpr uint32_t kPartRow = BN * 4 + 16;
  [[maybe_unused]] static constexpr uint32_t kRing = kStages * (kA + kB);
};

// Tensor reduction (add) of a shared-memory box into global memory.
NVFP4_DEV void tma_reduce_add_2d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], "
      "[%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y)
      : "memory");
}

// Asks L2 for a box of D ahead of its reduction.
NVFP4_DEV void tma_prefetch_2d(const CUtensorMap* map, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

// One warp's 32 rows x 32 columns (lane = row) into its box and out.  The 16-byte
// pieces of a row are permuted as the map's swizzle says (64- or 128-byte), so
// a warp's writes hit distinct banks; the box is rewritten once the store
// before has read it (FREE: that has been waited for).
template <bool FREE>
NVFP4_DEV void store_box(uint8_t* box, int lane, const uint32_t (&pk)[16], const CUtensorMap* map,
                         int32_t x, int32_t y) {
  if (!FREE) {
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }
#pragma unroll
  for (int p = 0; p < 4; ++p)
    *reinterpret_cast<uint4*>(box + lane * 64 + ((p ^ ((lane >> 1) & 3)) * 16)) =
        make_uint4(pk[4 * p], pk[4 * p + 1], pk[4 * p + 2], pk[4 * p + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, smem_u32(box), x, y);
    bulk_commit_group();
  }
}
NVFP4_DEV void reduce_box(uint8_t* box, int lane, const float (&v)[32], const CUtensorMap* map,
                          int32_t x, int32_t y) {
  if (lane == 0) bulk_wait_group_read<0>();
  __syncwarp();
#pragma unroll
  for (int p = 0; p < 8; ++p)
    *reinterpret_cast<float4*>(box + lane * 128 + ((p ^ (lane & 7)) * 16)) =
        make_float4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_reduce_add_2d(map, smem_u32(box), x, y);
    bulk_commit_group();
  }
}

// 16 bytes into another CTA of the cluster.
NVFP4_DEV void st_cluster_f4(uint32_t cluster_addr, const float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

template <int KIND, int BN, int DMODE, int SK>
__global__ void __cluster_dims__(2 * SK, 1, 1) __launch_bounds__(PairGroup<BN, DMODE, SK>::kThreads, 1)
    group_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmB2,
                      const __grid_constant__ CUtensorMap tmSFA,
                      const __grid_constant__ CUtensorMap tmSFB,
                      const __grid_constant__ CUtensorMap tmD,
                      const __grid_constant__ CUtensorMap tmC, const GroupArgs args) {
  using L = PairGroup<BN, DMODE, SK>;
  constexpr int S = L::kStages, kAt = L::kAt;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::offBar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto sf_bar = [&](int s) { return bar0 + 8u * (2 * S + s); };
  auto scf_bar = [&](int s) { return bar0 + 8u * (3 * S + s); };
  const uint32_t acc_full = bar0 + 8u * (4 * S);
  const uint32_t acc_empty = acc_full + 8;
  const uint32_t drain_bar = acc_full + 16;
  [[maybe_unused]] const uint32_t c_bar = drain_bar + 8u * L::kMmaWarps;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::offMisc + 4);
  GroupTable* table = reinterpret_cast<GroupTable*>(smem + L::offTable);
  // this CTA in its pair, and the pair's first CTA in the cluster
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, first = crank & ~1u;
  const bool leader = rank == 0;
  const uint16_t both = (uint16_t)(3u << first);
  const uint32_t peer_abort = mapa_shared(smem_u32(smem + L::offMisc + 4), crank ^ 1u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / (2 * SK), num_units = gridDim.x / (2 * SK);
  // what the roles leave in flight (pair_leave): stages that this CTA's producer
  // filled, and of the MMA warps whether they issued any
  const uint32_t fills = sbase + L::offMisc + 8, inject = fills + 4;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), L::kMmaWarps);  // one commit per MMA warp
      mbar_init(sf_bar(s), 8);                // four scale warps in each CTA
      mbar_init(scf_bar(s), 1);
    }
    mbar_init(acc_full, L::kMmaWarps);
    mbar_init(acc_empty, 16);  // 8 epilogue warps in each CTA
    for (int d = 0; d < L::kMmaWarps; ++d) mbar_init(drain_bar + 8u * d, 1);
    if (L::kAddC)
      for (int w = 0; w < 8; ++w) mbar_init(c_bar + 8u * w, 1);
    *abort_flag = 0;
    st_shared_u32(inject, injected());
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  griddep_wait();
  fill_table(table, args);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles = num_tiles<KIND>(table, args);
  // the pairs that share this cluster's tile (its only one then) and this
  // pair's part of the contraction; otherwise pair 0 works alone
  int parts = 1, part = 0;
  if constexpr (SK > 1) {
    part = (int)(crank >> 1);
    if (unit < tiles && tiles <= num_units) {
      int g = 0;
      const Tile t = tile_at<KIND, BN>(unit, g, table, args);
      const int rows = (min(t.live, 128) + 31) / 32 * 32;
      parts = SK;
      while (parts > 1 && ((parts - 1) * rows * L::kPartRow > L::kRing ||
                           (t.atoms + kAt - 1) / kAt < 2 * parts))
        parts /= 2;
    }
  }
  const int tile0 = part < parts ? unit : tiles;
  auto k_begin = [&](int num_kb) { return SK == 1 ? 0 : num_kb * part / parts; };
  auto k_end = [&](int num_kb) { return SK == 1 ? num_kb : num_kb * (part + 1) / parts; };

  if (warp < 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kRegsIssue));
  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      if (BN == 384) prefetch_tmap(&tmB2);
      prefetch_tmap(&tmSFA);
      prefetch_tmap(&tmSFB);
      uint32_t s = 0, ph = 0, count = 0;
      int g = 0;
      // injected stall: no loads, so every consumer's first wait runs out
      bool ok = !(ld_shared_u32(inject) & kStall);
      for (int tile = tile0; ok && tile < tiles; tile += num_units) {
        const Tile t = tile_at<KIND, BN>(tile, g, table, args);
        const int num_kb = (t.atoms + kAt - 1) / kAt;
        const int a_row = t.a_row + (int)rank * 128;
        const int sfa_row = (a_row >> 7) * args.kga + t.a_atom;
        const int sfb_row = (t.b_row >> 7) * args.kgb + t.b_atom;
        for (int kb = k_begin(num_kb); kb < k_end(num_kb); ++kb) {
          if (!wait_bounded_pair(empty_bar(s), ph ^ 1u, abort_flag, peer_abort, 0x11u)) {
            ok = false;
            break;
          }
          ++count;
          const uint32_t fb = mapa_shared(full_bar(s), first);
          const int a_x = (t.a_atom + kb * kAt) * (kAtom / 2);
          const int b_x = (t.b_atom + kb * kAt) * (kAtom / 2);
          if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * (L::kA + L::kB));
          tma_load_2d_pair(sbase + L::offA + s * L::kA, &tmA, fb, a_x, a_row);
          tma_load_2d_pair(sbase + L::offB + s * L::kB, &tmB, fb, b_x, t.b_row + (int)rank * 128);
          if (BN == 384)
            tma_load_2d_pair(sbase + L::offB + s * L::kB + 128 * kBKBytes, &tmB2, fb, b_x,
                             t.b_row + 256 + (int)rank * 64);
          // this CTA's scale atoms on its own barrier (past the tensor: zeros)
          mbar_arrive_expect_tx(scf_bar(s), L::kSFA + L::kSFB);
          tma_load_2d(sbase + L::offSFA + s * L::kSFA, &tmSFA, scf_bar(s), 0,
                      (sfa_row + kb * kAt) * 4);
#pragma unroll
          for (int i = 0; i < L::kRowBlocks; ++i)
            tma_load_2d(sbase + L::offSFB + s * L::kSFB + i * kAt * 512, &tmSFB, scf_bar(s), 0,
                        (sfb_row + i * args.kgb + kb * kAt) * 4);
          if (++s == S) { s = 0; ph ^= 1u; }
        }
      }
      st_shared_u32(fills, count);
    }
  } else if (warp <= L::kMmaWarps) {
    if (lane == 0 && leader) {
      // ---------------------------------------------------------------- MMA
      const bool second = warp == 2;
      const uint32_t idesc = second ? idesc_nvf4(256, 128) : idesc_nvf4(256, 256);
      const uint32_t d_tmem = tmem + (second ? 256u : 0u);
      const uint32_t b_off = second ? 128u * kBKBytes : 0u;
      const uint32_t sfb_col = second ? 0u : L::kColB01;
      const uint32_t sfb_step = second ? 4u : 8u;  // columns per atom
      uint32_t s = 0, ph = 0, acc_ph = 0, it = 0;
      int g = 0;
      bool ok = !quits_pair(ld_shared_u32(inject), abort_flag, peer_abort);
      for (int tile = tile0; ok && tile < tiles; tile += num_units) {
        const Tile t = tile_at<KIND, BN>(tile, g, table, args);
        if (t.atoms == 0) continue;
        const int num_kb = (t.atoms + kAt - 1) / kAt;
        if (!wait_bounded_pair(acc_empty, acc_ph ^ 1u, abort_flag, peer_abort, 0x22u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = k_begin(num_kb); kb < k_end(num_kb); ++kb, ++it) {
          if (!wait_bounded_pair(full_bar(s), ph, abort_flag, peer_abort, 0x24u) ||
              !wait_bounded_pair(sf_bar(s), ph, abort_flag, peer_abort, 0x23u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int nmma = min(kAt, t.atoms - kb * kAt);
          const uint32_t slot = tmem + L::kSfCol0 + (it % L::kSlots) * L::kSlotCols;
          const uint32_t a0 = sbase + L::offA + s * L::kA;
          const uint32_t b0 = sbase + L::offB + s * L::kB + b_off;
          for (int j = 0; j < nmma; ++j)
            tc_mma_pair_nvf4(d_tmem, smem_desc_sw128(a0 + 32 * j), smem_desc_sw128(b0 + 32 * j),
                             idesc, slot + L::kColA + 4 * j, slot + sfb_col + sfb_step * j,
                             kb != k_begin(num_kb) || j != 0 ? 1u : 0u);
          st_shared_u8(inject + warp, 1u);
          tc_commit_pair(empty_bar(s), both);
          if (++s == S) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(acc_full, both);
        acc_ph ^= 1u;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scale warps
    // Warp q stores the stage's atoms into its 32-lane quarter: lane i gets
    // line i of an atom (the scale words of rows i, i + 32, i + 64, i + 96) in
    // 4 columns.  A slot is rewritten once the MMAs that read it completed.
    const int q = warp & 3;
    const uint32_t sf_leader = mapa_shared(sf_bar(0), first);
    uint32_t s = 0, ph = 0, it = 0;
    int g = 0;
    bool ok = true;
    for (int tile = tile0; ok && tile < tiles; tile += num_units) {
      const int num_kb = (tile_at<KIND, BN>(tile, g, table, args).atoms + kAt - 1) / kAt;
      for (int kb = k_begin(num_kb); kb < k_end(num_kb); ++kb, ++it) {
        if (!wait_bounded_pair(scf_bar(s), ph, abort_flag, peer_abort, 0x26u)) {
          ok = false;
          break;
        }
        if (L::kSlots < S && it >= (uint32_t)L::kSlots) {
          const uint32_t prev = it - L::kSlots;
          if (!wait_bounded_pair(empty_bar(prev % S), (prev / S) & 1u, abort_flag, peer_abort,
                                 0x25u)) {
            ok = false;
            break;
          }
        }
        const uint8_t* sa = smem + L::offSFA + s * L::kSFA + lane * 16;
        const uint8_t* sb = smem + L::offSFB + s * L::kSFB + lane * 16;
        uint32_t v[L::kSlotCols];
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
          const uint4 a = *reinterpret_cast<const uint4*>(sa + j * 512);
          const uint4 b0 = *reinterpret_cast<const uint4*>(sb + j * 512);
          const uint4 b1 = *reinterpret_cast<const uint4*>(sb + (kAt + j) * 512);
          const uint32_t w[12] = {a.x,  a.y,  a.z,  a.w,  b0.x, b0.y,
                                  b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[L::kColA + 4 * j + e] = w[e];
            v[L::kColB01 + 8 * j + e] = w[4 + e];
            v[L::kColB01 + 8 * j + 4 + e] = w[8 + e];
          }
          if (BN == 384) {
            const uint4 b2 = *reinterpret_cast<const uint4*>(sb + (2 * kAt + j) * 512);
            v[4 * j] = b2.x;
            v[4 * j + 1] = b2.y;
            v[4 * j + 2] = b2.z;
            v[4 * j + 3] = b2.w;
          }
        }
        const uint32_t taddr =
            tmem + ((uint32_t)(32 * q) << 16) + L::kSfCol0 + (it % L::kSlots) * L::kSlotCols;
#pragma unroll
        for (int c = 0; c < (int)L::kSlotCols; c += 16) tmem_st16(taddr + c, v + c);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(sf_leader + 8u * s);
        if (++s == S) { s = 0; ph ^= 1u; }
      }
    }
  }
  if (SK > 1 && parts > 1) {  // the two barriers of the epilogue's exchange
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  } else {
    // -------------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kRegsEpilogue));
    constexpr int kCols = BN / 2, kChunks = kCols / 32;
    const int ew = warp - 8;
    const int q = warp & 3, h = ew >> 2;
    const uint32_t acc_empty_leader = mapa_shared(acc_empty, first);
    const float alpha = __fmul_rn(__ldg(args.sdec_a), __ldg(args.sdec_b));
    uint8_t* box = smem + L::offStore + ew * (L::kBoxes * L::kBox);
    if (lane == 0) prefetch_tmap(&tmD);
    // 32 columns of a row: times alpha, plus C (from `c_box`, this lane's row of a
    // box, or from memory), rounded; zero outside the group
    auto finish = [&](float (&f)[32], int64_t row, int col, bool live, const uint8_t* c_box,
                      uint32_t (&pk)[16]) {
#pragma unroll
      for (int e = 0; e < 32; ++e) f[e] = __fmul_rn(f[e], alpha);
      if (DMODE == NVFP4_D_BF16_ADD_C && live && col < args.N) {
        const uint4* cp = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(args.C) + row * args.N + col);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint4 u = L::kAddC ? *reinterpret_cast<const uint4*>(
                                         c_box + ((p ^ ((lane >> 1) & 3)) * 16))
                                   : cp[p];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[8 * p + 2 * e] = __fadd_rn(f[8 * p + 2 * e], __uint_as_float(w[e] << 16));
            f[8 * p + 2 * e + 1] =
                __fadd_rn(f[8 * p + 2 * e + 1], __uint_as_float(w[e] & 0xFFFF0000u));
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) pk[e] = live ? pack_bf16x2(f[2 * e], f[2 * e + 1]) : 0u;
    };
    uint32_t acc_ph = 0;
    int g = 0;
    bool ok = true;
    // What a later tile adds to.  The fold wants its boxes of D in L2 by then: a
    // tile ahead takes 4000 rows into 128 x [1024, 1024] from 209 to 184 us and
    // 16384 rows into 8 x [4096, 2048] from 125 to 123.
    [[maybe_unused]] auto ahead = [&](int tile) {
      int gn = g;
      const Tile t = tile_at<KIND, BN>(tile, gn, table, args);
      const int x0 = t.d_col + h * kCols;
      if (lane == 0 && t.atoms > 0 && t.live > (int)rank * 128)
        for (int c = 0; c < kChunks; ++c)
          if (x0 + c * 32 < args.N)
            tma_prefetch_2d(&tmD, x0 + c * 32, (int32_t)(t.d_row + (int)rank * 128 + q * 32));
    };
    if (L::kF32 && tile0 < tiles) ahead(tile0);
    // C lands in the warp's boxes while the tile's MMAs run; the sums leave from
    // the same places (65536 rows, 64 groups, 1024 x 2048: 127 us; 219 with C read
    // by each lane's loads, 89 without C).  N is a multiple of 128, so a warp's
    // kCols columns lie in N or behind it as a whole.
    static_assert(!L::kAddC || (kCols == 128 && kChunks == L::kBoxes), "boxes");
    [[maybe_unused]] bool c_due = false;
    [[maybe_unused]] uint32_t c_ph = 0;
    auto fetch = [&](int tile) {
      int gn = g;
      const Tile t = tile_at<KIND, BN>(tile, gn, table, args);
      const int x0 = t.d_col + h * kCols;
      c_due = t.live > (int)rank * 128 && x0 < args.N;
      if (c_due && lane == 0) {
        bulk_wait_group_read<0>();
        mbar_arrive_expect_tx(c_bar + 8u * ew, L::kBoxes * L::kBox);
        for (int c = 0; c < kChunks; ++c)
          tma_load_2d(smem_u32(box + c * L::kBox), &tmC, c_bar + 8u * ew, x0 + c * 32,
                      (int32_t)(t.d_row + (int)rank * 128 + q * 32));
      }
      __syncwarp();
    };
    if (L::kAddC && tile0 < tiles) fetch(tile0);
    for (int tile = tile0; tile < tiles; tile += num_units) {
      const Tile t = tile_at<KIND, BN>(tile, g, table, args);
      if (L::kF32 && tile + num_units < tiles) ahead(tile + num_units);
      const int r0 = (int)rank * 128 + q * 32;  // this warp's first row of the tile
      const bool mine = t.live > (int)rank * 128;
      const bool live = r0 + lane < t.live;
      const int32_t y = (int32_t)(t.d_row + r0);
      const int x0 = t.d_col + h * kCols;
      if constexpr (L::kF32) {
        if (t.atoms == 0) continue;  // nothing to add
        if (!wait_bounded_pair(acc_full, acc_ph, abort_flag, peer_abort, 0x33u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * kCols + c * 32), r[c]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_leader);
        acc_ph ^= 1u;
        if (!mine) continue;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __fmul_rn(__uint_as_float(r[c][e]), alpha);
          if (x0 + c * 32 < args.N) reduce_box(box, lane, v, &tmD, x0 + c * 32, y);
        }
      } else if (SK > 1 && parts > 1) {
        // every pair's MMAs are done behind the first barrier, and pair 0's ring
        // with them; the sums have arrived behind the second.  A warp that gave up
        // meets the others at both and reads nothing: its MMAs may still run.
        if (!wait_bounded_pair(acc_full, acc_ph, abort_flag, peer_abort, 0x33u)) ok = false;
        tc_fence_after();
        __syncwarp();
        cluster_sync();
        const int rows = (min(max(t.live - (int)rank * 128, 0), 128) + 31) / 32 * 32;
        const uint32_t line = (uint32_t)(q * 32 + lane) * L::kPartRow + (uint32_t)(h * kCols) * 4;
        const uint32_t tm = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * kCols);
        if (ok && part > 0 && q * 32 < rows) {
          const uint32_t to =
              mapa_shared(sbase + (uint32_t)((part - 1) * rows) * L::kPartRow + line, rank);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t r[32];
            tmem_ld32(tm + (uint32_t)(c * 32), r);
            tmem_ld_wait();
#pragma unroll
            for (int p = 0; p < 8; ++p)
              st_cluster_f4(to + (uint32_t)(c * 128 + p * 16),
                            make_float4(__uint_as_float(r[4 * p]), __uint_as_float(r[4 * p + 1]),
                                        __uint_as_float(r[4 * p + 2]),
                                        __uint_as_float(r[4 * p + 3])));
          }
        }
        cluster_sync();
        if (ok && part == 0 && mine) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t r[32];
            tmem_ld32(tm + (uint32_t)(c * 32), r);
            tmem_ld_wait();
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(r[e]);
            if (q * 32 < rows)
              for (int i = 0; i < parts - 1; ++i) {
                const float4* v = reinterpret_cast<const float4*>(
                    smem + (uint32_t)(i * rows) * L::kPartRow + line + (uint32_t)(c * 128));
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                  const float4 u = v[p];
                  f[4 * p] += u.x;
                  f[4 * p + 1] += u.y;
                  f[4 * p + 2] += u.z;
                  f[4 * p + 3] += u.w;
                }
              }
            uint32_t pk[16];
            finish(f, t.d_row + r0 + lane, x0 + c * 32, live, nullptr, pk);
            if (x0 + c * 32 < args.N) store_box<false>(box, lane, pk, &tmD, x0 + c * 32, y);
          }
        }
        break;  // the cluster's only tile
      } else {
        uint32_t pk[kChunks][16];
        if (t.atoms > 0) {
          if (!wait_bounded_pair(acc_full, acc_ph, abort_flag, peer_abort, 0x33u)) {
            ok = false;
            break;
          }
          if (L::kAddC && c_due) {
            if (!wait_bounded_pair(c_bar + 8u * ew, c_ph, abort_flag, peer_abort, 0x44u)) {
              ok = false;
              break;
            }
            c_due = false;
            c_ph ^= 1u;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t r[32];
            tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * kCols + c * 32), r);
            tmem_ld_wait();
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(r[e]);
            finish(f, t.d_row + r0 + lane, x0 + c * 32, live,
                   box + (L::kAddC ? c : 0) * L::kBox + lane * 64, pk[c]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty_leader);
          acc_ph ^= 1u;
        } else {
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[c][e] = 0u;
        }
        if (mine)
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (x0 + c * 32 < args.N)
              store_box<L::kAddC>(box + (L::kAddC ? c : 0) * L::kBox, lane, pk[c], &tmD,
                                  x0 + c * 32, y);
        if (L::kAddC && tile + num_units < tiles) fetch(tile + num_units);
      }
    }
    if (L::kAddC && c_due) wait_drain(c_bar + 8u * ew, c_ph);  // given up: its loads have landed
    if (SK > 1 && part >= parts && parts > 1) {  // a pair without a part of the tile
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
    if (KIND == kRows && ok)
      clear_tail(args, (int64_t)blockIdx.x * 256 + threadIdx.x - 256, (int64_t)gridDim.x * 256);
    if (lane == 0) bulk_wait_group<0>();  // stores done before exit
  }

  tc_fence_before();
  pair_leave<L, S, 2 * SK, true>(L::kA + L::kB);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(ld_shared_u32(sbase + L::offMisc), kTmemCols);
  }
}

// 2-D map over an output [rows, cols] with boxes of 32 x 32, swizzled over a
// box row's 64 (bf16) or 128 (FP32) bytes.
bool make_box_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, bool f32) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(cols * (f32 ? 4 : 2))};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Where the operands of a product lie, for the maps.
struct Operands {
  const void *a_codes, *a_sf, *b_codes, *b_sf;
  int64_t a_rows, a_cols, b_rows, b_cols, d_rows;
};

// Clusters of a kernel that are resident at once; 0 when its set-up failed.
template <int KIND, int BN, int DMODE, int SK>
int group_units(int sms) {
  using L = PairGroup<BN, DMODE, SK>;
  static GemmLaunchState ls;
  return gemm_setup(ls, group_pair_kernel<KIND, BN, DMODE, SK>, L::kAlloc, L::kThreads,
                    L::kSplitRegs, 2 * SK, sms);
}

template <int KIND, int BN, int DMODE, int SK>
nvfp4_status launch_group_pair(const Operands& o, GroupArgs a, int sms, cudaStream_t stream) {
  using L = PairGroup<BN, DMODE, SK>;
  auto kern = group_pair_kernel<KIND, BN, DMODE, SK>;
  const int units = group_units<KIND, BN, DMODE, SK>(sms);
  if (units <= 0) return NVFP4_ERR_CUDA;
  a.num_m_blk = (a.M + 255) / 256;
  a.num_n_blk = (a.N + BN - 1) / BN;
  CUtensorMap ma, mb, mb2 = {}, msa, msb, md, mc = {};  // mb2, mc: where the kernel reads them
  if (!make_code_map(&ma, o.a_codes, o.a_rows, o.a_cols / 2, 128) ||
      !make_code_map(&mb, o.b_codes, o.b_rows, o.b_cols / 2, 128) ||
      (BN == 384 && !make_code_map(&mb2, o.b_codes, o.b_rows, o.b_cols / 2, 64)) ||
      !make_sf_map(&msa, o.a_sf, swizzled_scale_bytes(o.a_rows, o.a_cols)) ||
      !make_sf_map(&msb, o.b_sf, swizzled_scale_bytes(o.b_rows, o.b_cols)) ||
      !make_box_map(&md, a.D, o.d_rows, a.N, L::kF32) ||
      (L::kAddC && !make_box_map(&mc, a.C, o.d_rows, a.N, false)))
    return NVFP4_ERR_CUDA;
  return cuda_status(launch_pdl(kern, 2 * SK * units, L::kThreads, L::kAlloc, stream, ma, mb, mb2, msa,
                                msb, md, mc, a));
}

// The width of a product's tiles: the one whose rounds of tiles over the pairs
// cost less.  The host knows the rows and the number of groups, not the sizes;
// with the padding to 128 taken off, that gives about `m_blocks` blocks of 256
// rows.  A 384-wide tile costs 1.2 256-wide ones where the tensor cores set the
// pace (as in gemm.cu), 1.5, its bytes, where groups have too few rows for
// that.  Measured (us, 256 and 384 wide): 16384 rows, 8 groups, 4096 x 14336:
// 381, 321; 2 rows, 2 of 8 groups, the same weights: 23.0, 20.2; 2 rows,
// 14336 x 4096: 30.5, 36.0; 6216 rows, 64 groups, 2048 x 1024: 29.6, 28.9.
int32_t rows_tile(int64_t rows, int64_t groups, int64_t n, int pairs) {
  const int64_t used = std::min(groups, rows / 128);
  const int64_t per = std::max<int64_t>(1, rows / used - 64);
  const int64_t m_blocks = used * ((per + 255) / 256);
  const int64_t r256 = (m_blocks * ((n + 255) / 256) + pairs - 1) / pairs;
  const int64_t r384 = (m_blocks * ((n + 383) / 384) + pairs - 1) / pairs;
  return 10 * r256 <= (per >= 256 ? 12 : 15) * r384 ? NVFP4_TILE_PAIR_256X256
                                                    : NVFP4_TILE_PAIR_256X384;
}

// A contraction from here on is shared by pairs where tiles are few.  Measured
// (us, one pair a tile and shared): 2 rows x 14336 x 4096: 29.6, 22.0; 1 row x
// 8192 x 1024: 18.5, 14.1; 2 rows x 4096 x 2048: 12.3, 11.9; 8 rows x 2048 x
// 1024: 11.1, 13.6.
constexpr int kSharedK = 4096;

template <int KIND, int DMODE>
nvfp4_status launch_tile(int32_t tile, const Operands& o, const GroupArgs& a, int sms,
                         cudaStream_t stream) {
  if constexpr (KIND == kRows) {
    if (tile == NVFP4_TILE_AUTO) {
      // the most tiles there can be, each with a cluster of its own
      const int64_t tiles = (int64_t)a.rows / 128 * ((a.N + 255) / 256);
      if (a.K >= kSharedK && tiles <= group_units<KIND, 256, DMODE, 4>(sms))
        return launch_group_pair<KIND, 256, DMODE, 4>(o, a, sms, stream);
      if (a.K >= kSharedK && tiles <= group_units<KIND, 256, DMODE, 2>(sms))
        return launch_group_pair<KIND, 256, DMODE, 2>(o, a, sms, stream);
      // with C the narrow tiles, whose boxes have room for it.  Measured (us, 256
      // and 384 wide): 8192 rows, 8 groups, 14336 x 4096: 217, 215; 16384 rows, 8
      // groups, 2048 x 4096: 94, 120; 65536 rows, 64 groups, 1024 x 2048: 127, 219.
      tile = DMODE == NVFP4_D_BF16_ADD_C ? NVFP4_TILE_PAIR_256X256
                                         : rows_tile(a.rows, a.groups, a.N, sms / 2);
    }
  }
  if constexpr (DMODE != NVFP4_D_F32_ACCUM)
    if (tile == NVFP4_TILE_PAIR_256X384)
      return launch_group_pair<KIND, 384, DMODE, 1>(o, a, sms, stream);
  return launch_group_pair<KIND, 256, DMODE, 1>(o, a, sms, stream);
}

bool known_tile(int32_t tile, int32_t d_mode) {
  return tile == NVFP4_TILE_AUTO || tile == NVFP4_TILE_PAIR_256X256 ||
         (tile == NVFP4_TILE_PAIR_256X384 && d_mode != NVFP4_D_F32_ACCUM);
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
                             int64_t K, int32_t tile, cudaStream_t stream) {
  nvfp4_status st = check_groups(A, B, sizes, offsets, groups, D);
  if (st != NVFP4_OK) return st;
  if (b_view < 0 || b_view > 1) return NVFP4_ERR_INVALID_ARG;
  if (d_mode != NVFP4_D_BF16 && d_mode != NVFP4_D_BF16_ADD_C) return NVFP4_ERR_INVALID_ARG;
  if ((d_mode == NVFP4_D_BF16_ADD_C) != (C != nullptr) || !known_tile(tile, d_mode))
    return NVFP4_ERR_INVALID_ARG;
  const void* b_codes = b_view ? B->codes_t : B->codes;
  const void* b_sf = b_view ? B->scales_t : B->scales;
  if (!b_codes || !b_sf) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || rows % 128 || N <= 0 || N % 128 || K <= 0 || K % 64) return NVFP4_ERR_SHAPE;
  if (rows > INT32_MAX - 256 || groups * N > INT32_MAX - 512 || groups * K > INT32_MAX)
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
  a.b_row_step = b_view ? 0 : (int)N;
  a.b_atom_step = b_view ? (int)(K / kAtom) : 0;
  const Operands o = {A->codes, A->scales, b_codes, b_sf, rows, K, b_rows, b_cols, rows};
  return d_mode == NVFP4_D_BF16
             ? launch_tile<kRows, NVFP4_D_BF16>(tile, o, a, dev.sm_count, stream)
             : launch_tile<kRows, NVFP4_D_BF16_ADD_C>(tile, o, a, dev.sm_count, stream);
}

nvfp4_status group_wgrad_impl(const nvfp4_tensor* A, const nvfp4_tensor* B, const int32_t* sizes,
                              const int32_t* offsets, int32_t groups, void* D, int32_t d_mode,
                              int64_t M, int64_t N, int64_t rows, int32_t tile,
                              cudaStream_t stream) {
  nvfp4_status st = check_groups(A, B, sizes, offsets, groups, D);
  if (st != NVFP4_OK) return st;
  if (!B->codes || !B->scales) return NVFP4_ERR_INVALID_ARG;
  if (d_mode != NVFP4_D_BF16 && d_mode != NVFP4_D_F32_ACCUM) return NVFP4_ERR_INVALID_ARG;
  if (!known_tile(tile, d_mode)) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || rows % 128 || M <= 0 || M % 128 || N <= 0 || N % 128) return NVFP4_ERR_SHAPE;
  if (rows > INT32_MAX - 256 || M > INT32_MAX - 256 || N > INT32_MAX - 256) return NVFP4_ERR_SHAPE;
  if ((M / 128) * (N / 128) * groups > INT32_MAX - 1024 || M * groups > INT32_MAX)
    return NVFP4_ERR_SHAPE;
  if (A->rows != M || A->cols != rows || B->rows != N || B->cols != rows) return NVFP4_ERR_SHAPE;
  if (!aligned16(A->codes) || !aligned16(A->scales) || !aligned16(B->codes) ||
      !aligned16(B->scales) || !aligned16(D) || !aligned4(sizes) || !aligned4(offsets))
    return NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  GroupArgs a = {};
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
  const Operands o = {A->codes, A->scales, B->codes, B->scales, M, rows, N, rows, groups * M};
  // weight gradients are bound by D: both widths take the same time (64 x [1024,
  // 2048] over 32000 rows: 74 us), and the narrow one wastes less of odd widths
  if (tile == NVFP4_TILE_AUTO) tile = NVFP4_TILE_PAIR_256X256;
  return d_mode == NVFP4_D_BF16
             ? launch_tile<kWgrad, NVFP4_D_BF16>(tile, o, a, dev.sm_count, stream)
             : launch_tile<kWgrad, NVFP4_D_F32_ACCUM>(tile, o, a, dev.sm_count, stream);
}

}  // namespace nvfp4
