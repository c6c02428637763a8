// muon.cu -- orthogonalised momentum: the update of a weight matrix (or of a
// stack of them, an expert each) that an optimiser of the Muon kind takes.
//
//   momentum  V <- mu V + G,  U = G + mu V (nesterov) or V
//   start     X = U / max(||U||_F, eps)
//   step      A = X X^T,  B = b A + c A A,  X <- a X + B X      (Newton-Schulz)
//
// An odd polynomial of X's singular values, which the steps bring near 1; the
// products run on the side of the fewer rows or columns (m of them, n on the
// other side): X X^T for a wide matrix, X^T X and X <- a X + X B for a tall
// one.  Nothing is transposed in memory: an operand whose contraction does not
// lie along its rows is read as an MN-major operand.
//
// Precision.  The products take f16 operands, at the rate of bf16 and with 3
// bits more, scaled by 2^12: every entry of X, A and B is bounded by a spectral
// norm (below 1.3 for X, 2.9 for B with the usual coefficients), so 16, where
// f16 ends, is out of reach, and what is 2^-26 still has all its bits.  Where
// a rounding to f16 would be multiplied by the later steps (by up to 3.4 each,
// for small singular values) it is not made: X is carried as the sum of two
// f16 numbers (22 bits), of which the products see the first and the term a X
// both; A's and B's diagonals, which hold most of them once X is near
// orthogonal, are kept in FP32 outside of the f16 matrices, and their terms are
// added where a product is finished:
//   A = D + E:       A A = E E + (d_i + d_j) E_ij + diag(d_i^2)
//   B = D' + F:      a X + B X = (a + d'_i) X + F X
// The result is 1e-4 to 1.3e-3 off that of 64 bits in the 2-norm, for full and
// for deficient rank (a rank of 8 in 512 rows: 6e-4; with X in f16 alone 4e-2,
// in bf16 3e-1); rounding it to bf16 costs 1.7e-3.
//
// What bounds it, and measured.  Large matrices: the tensor cores under the power cap
// (14336 x 4096, 3.95 TFLOP: 2615 to 2985 us by card and by how long the cap has held, the
// last at a median of 1511 MHz in a loop of seconds, 1.32 to 1.5 PF/s; cuBLAS holds 1.72 in
// such a loop): X X^T 145 us (2 rounds of tiles where 1.8 would do), E E 50, an update 285,
// momentum and start 185 at 7.2 TB/s.  Stacks of smaller ones: what an SM takes in of
// operands and of X's halves (64 x [1024, 2048]: 2510 to 2855 us, the last at a median of
// 1616 MHz in a loop of seconds; an update's tensor cores 52 % busy, DRAM 4.5 TB/s), 450 of
// it momentum and start.  One matrix of 1024 x 1024: 137 us, 15 products of 8: 3.4 us for 16
// stages at what an SM takes in (24 KB each), 2.5 for the meeting and the stores before it,
// 1.5 for the epilogue.
#include <cmath>

#include "muon_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kBK = 64;     // contraction elements of a stage, 128 bytes

// A warp goes on only together: its lanes may give up at a wait one by one.
NVFP4_DEV bool all_waited(bool ok) { return __all_sync(0xFFFFFFFFu, ok); }

// One lane of a converged warp, the same every time.  A role's warp runs its loop
// together and has this lane issue what one thread issues: its operands are uniform
// then, and a stage costs its producer and its MMA thread 150 cycles, 500 with the
// whole loop in one lane's branch.
NVFP4_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// An MN-major operand lies in boxes of 64 (along M or N) x 64 (along K).
constexpr uint32_t kBoxMN = 64 * kBK * 2;

// One product over a stack of matrices, and what becomes of it.  With r a result of
// the tensor cores, x what the chunk brings in (nothing, E, or X's two halves) and d
// the diagonal's entries of its row and column, all of them are
//   v = (p + q (d_i + d_j)) x + s r
// and on a symmetric product's diagonal  p d_i + q d_i^2 + t r, which goes to dout:
//   E, D of X X^T       p = q = 0, s = 2^-12, t = 2^-24
//   F, D' from E E      p = b, q = c, s = c 2^-12, t = c 2^-24
//   X' = (a + d') X + F X   p = a, q = 1, s = 2^-12, d' of the rows or the columns
// (One formula, and one code for all of them: where a launch goes through every kind
// of product, code of their own for each, 20 KB a kind, came anew from memory at each.)
struct NsArgs {
  int m, n, k;             // its rows, columns and contraction
  int tiles_m, tiles_n;
  int tiles_per, tiles;    // of a matrix; of all, each as often as it has splits
  int splits;              // parts of the contraction, each a CTA's
  int last;                // >= 0: matrices from this one down to the first
  int a_mn, b_mn;          // operands whose contraction does not lie along their rows
  int symmetric;
  int loads;               // boxes that a chunk brings in
  int by_row, by_col;      // whose diagonal entries count
  int final;               // the result is stored as bf16, not as f16 (and lo)
  float p, q, s, t;
  const float* din;
  float* dout;
  int64_t dstride;         // from one matrix's diagonal to the next's
  float4* part;            // splits: [tile][split][chunk][8][32 lanes], 4 columns each
  unsigned int* tickets;   // [tile][chunk], zero before and after
  __nv_bfloat16* out;      // final
  int out_boxes;           // final: rows are whole multiples of 16 bytes
};
struct NsMaps {
  const CUtensorMap *a, *b, *in0, *in1, *out0, *out1;
};

NVFP4_DEV void tc_mma_f16(bool pair, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                          uint32_t idesc, uint32_t accumulate) {
  if (pair)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

NVFP4_DEV void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster,
                                int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}
NVFP4_DEV void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                           int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
NVFP4_DEV void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y,
                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Between what the generic proxy sees and what tensor copies read or wrote.
NVFP4_DEV void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// A 32 x 32 box of 16-bit values in shared memory, rows of 64 bytes with the
// 64-byte swizzle: 16-byte piece p of row r.
NVFP4_DEV uint32_t box_piece(int r, int p) {
  return (uint32_t)(r * 64 + ((p ^ ((r >> 1) & 3)) * 16));
}
NVFP4_DEV void box_put(uint8_t* box, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
    *reinterpret_cast<uint4*>(box + box_piece(lane, p)) =
        make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
}
NVFP4_DEV void box_get(const uint8_t* box, int lane, uint32_t (&w)[16]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint4 u = *reinterpret_cast<const uint4*>(box + box_piece(lane, p));
    w[4 * p] = u.x;
    w[4 * p + 1] = u.y;
    w[4 * p + 2] = u.z;
    w[4 * p + 3] = u.w;
  }
}
// to = from^T, one warp, 8 x 8 at a time.
NVFP4_DEV void box_transpose(uint32_t from, uint32_t to, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r0, r1, r2, r3;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(from + box_piece(8 * i + (lane & 7), lane >> 3))
                 : "memory");
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     to + box_piece(8 * (lane >> 3) + (lane & 7), i)),
                 "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
  }
}

// =============================================================================
// The products.  Tiles of 128 rows x BN columns of a CTA, or of 256 x BN of a CTA
// pair (tcgen05 cta_group::2: CTA r loads rows [128 r, 128 r + 128) of A and its half
// of B's), contraction 64 a stage (kind::f16, K = 16 an instruction).  A TMA
// producer, an MMA thread and 8 epilogue warps in each CTA, which walks its tiles;
// two accumulators in tensor memory, so a tile's epilogue runs under the next one's
// MMAs.  An epilogue warp takes 32 rows x 32 columns at a time through a slot of two
// boxes: what the chunk needs (E, or X's two halves) comes in ahead by tensor loads,
// the results go out of the same boxes by tensor stores.  Of a symmetric product the
// tiles that reach the diagonal or lie below it are computed, their boxes below the
// diagonal stored twice, the second time transposed (ldmatrix and stmatrix).  Rows,
// columns and contraction behind a matrix's end are filled with zeros by the loads and
// left out by the stores.
// Of a contraction in `splits` parts every CTA writes its sums of a tile to memory;
// whichever warp comes last to a chunk adds all of them, in their order, and finishes it.
// =============================================================================
template <bool PAIR, int BN, int STAGES, int SLOTS>
struct NsLayout {
  static constexpr bool kPair = PAIR;
  static constexpr int kBN = BN, kBM = PAIR ? 256 : 128, kStages = STAGES, kSlots = SLOTS;
  static constexpr int kRowsB = PAIR ? BN / 2 : BN;  // of B that a CTA loads
  static constexpr uint32_t kA = 128 * kBK * 2, kB = kRowsB * kBK * 2;
  static constexpr uint32_t kBox = 32 * 64, kSlot = 2 * kBox;
  static constexpr uint32_t offA = 0, offB = offA + kStages * kA;
  static constexpr uint32_t offSlots = offB + kStages * kB;
  static constexpr uint32_t offBar = offSlots + 8 * kSlots * kSlot;
  // full, empty per stage, accumulator full and empty, and the drains' barrier
  // where pair_leave looks for it; then one per epilogue warp and slot
  static constexpr uint32_t kAccBar = 2 * kStages, kDrainBar = 4 * kStages + 2;
  static constexpr uint32_t kSlotBar = kDrainBar + 3;
  // between the products of one launch: the warps are done, and may go on
  static constexpr uint32_t kDoneBar = kSlotBar + 8 * kSlots, kGoBar = kDoneBar + 1;
  static constexpr uint32_t offMisc = offBar + (kGoBar + 1 + (kGoBar + 1) % 2) * 8;
  static constexpr uint32_t kAlloc = offMisc + 16 + 1024;
  static constexpr int kThreads = 384;
  static constexpr int kChunks = BN / 64;  // of an epilogue warp
  static_assert(kAlloc <= 232448, "shared memory overflow");
  static_assert(offSlots % 1024 == 0 && kAccBar + 4 <= kDrainBar, "layout");
  static_assert(2 * BN <= (int)kTmemCols, "tensor memory overflow");
};

// A CTA's place and what its roles share.
template <class L>
struct Ns {
  uint8_t* smem;
  uint32_t base, bar0, tmem;
  volatile int* abort_flag;
  uint32_t peer_abort, rank;
  int warp, lane, unit, units;

  NVFP4_DEV uint32_t full_bar(uint32_t s) const { return bar0 + 8u * s; }
  NVFP4_DEV uint32_t empty_bar(uint32_t s) const { return bar0 + 8u * (L::kStages + s); }
  NVFP4_DEV uint32_t acc_full(uint32_t b) const { return bar0 + 8u * (L::kAccBar + b); }
  NVFP4_DEV uint32_t acc_empty(uint32_t b) const { return bar0 + 8u * (L::kAccBar + 2 + b); }
  NVFP4_DEV uint32_t fills() const { return base + L::offMisc + 8; }
  NVFP4_DEV uint32_t inject() const { return base + L::offMisc + 12; }
  NVFP4_DEV bool wait(uint32_t bar, uint32_t parity, unsigned int code) const {
    return L::kPair ? wait_bounded_pair(bar, parity, abort_flag, peer_abort, code)
                    : wait_bounded(bar, parity, abort_flag, code);
  }
  NVFP4_DEV void commit(uint32_t bar) const {
    if (L::kPair)
      tc_commit_pair(bar, (uint16_t)3);
    else
      tc_commit(bar);
  }
};

// Barriers, tensor memory; ends with all of the cluster's CTAs set up.
template <class L>
NVFP4_DEV Ns<L> ns_enter() {
  extern __shared__ uint8_t smem_raw[];
  Ns<L> c;
  c.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~uintptr_t(1023));
  c.base = smem_u32(c.smem);
  c.bar0 = c.base + L::offBar;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(c.smem + L::offMisc);
  c.abort_flag = reinterpret_cast<volatile int*>(c.smem + L::offMisc + 4);
  c.rank = L::kPair ? cluster_ctarank() : 0;
  c.peer_abort = L::kPair ? mapa_shared(c.base + L::offMisc + 4, c.rank ^ 1u) : 0;
  c.warp = threadIdx.x >> 5;
  c.lane = threadIdx.x & 31;
  c.unit = L::kPair ? blockIdx.x / 2 : blockIdx.x;
  c.units = L::kPair ? gridDim.x / 2 : gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(c.full_bar(s), 1);
      mbar_init(c.empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(c.acc_full(b), 1);
      mbar_init(c.acc_empty(b), L::kPair ? 16 : 8);  // 8 epilogue warps in each CTA
    }
    mbar_init(c.bar0 + 8u * L::kDrainBar, 1);
    mbar_init(c.bar0 + 8u * (L::kDrainBar + 1), 1);
    for (int w = 0; w < 8 * L::kSlots; ++w) mbar_init(c.bar0 + 8u * (L::kSlotBar + w), 1);
    mbar_init(c.bar0 + 8u * L::kDoneBar, 8);
    mbar_init(c.bar0 + 8u * L::kGoBar, 1);
    *c.abort_flag = 0;
    st_shared_u32(c.fills(), 0);
    st_shared_u32(c.inject(), injected());
    fence_mbar_init();
  }
  if (c.warp == 1) {
    if (L::kPair) {
      tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (L::kPair) cluster_sync();
  tc_fence_after();
  c.tmem = *tmem_slot;
  return c;
}

// The end: what a CTA that has given up left in flight finishes before its memory goes.
template <class L>
NVFP4_DEV void ns_leave(const Ns<L>& c) {
  tc_fence_before();
  __syncthreads();
  // the MMAs, by the lane that issued them
  if (*c.abort_flag && c.warp == 1 && (ld_shared_u32(c.inject()) >> 8 & 0xFFu) && elect_one()) {
    const uint32_t bar = c.bar0 + 8u * (L::kDrainBar + 1);
    if (L::kPair)
      tc_commit_pair(bar, (uint16_t)(1u << c.rank));
    else
      tc_commit(bar);
    wait_drain(bar, 0);
  }
  if (L::kPair) {
    pair_leave<L, L::kStages, 2, false>(L::kA + L::kB);
  } else {
    if (*c.abort_flag && threadIdx.x == 0)
      drain_stages<L::kStages>(c.bar0, ld_shared_u32(c.fills()));
    __syncthreads();
  }
  if (c.warp == 1) {
    tc_fence_after();
    if (L::kPair)
      tmem_dealloc_pair(ld_shared_u32(c.base + L::offMisc), kTmemCols);
    else
      tmem_dealloc(ld_shared_u32(c.base + L::offMisc), kTmemCols);
  }
}

// Tile t of a matrix.  A symmetric product's: row by row, those that begin left of the
// row's end.  Else with the matrix's smaller side running fastest: tiles at work
// together then read X, the operand that L2 may not hold, once (14336 x 4096: an
// update 375 us the other way round, 330 this).
template <class L>
NVFP4_DEV void tile_of(int t, const NsArgs& a, int& tm, int& tn) {
  if (a.symmetric) {
    constexpr int kPer = L::kBM / L::kBN;  // more tiles in each row; the last may be short
    tm = (int)((sqrtf(8.0f / kPer * (float)t + 1.0f) - 1.0f) * 0.5f);
    while (kPer * ((tm + 1) * (tm + 2) / 2) <= t) ++tm;
    while (kPer * (tm * (tm + 1) / 2) > t) --tm;
    tn = t - kPer * (tm * (tm + 1) / 2);
  } else {
    const int fast = min(a.tiles_m, a.tiles_n), slow = t / fast;
    tm = a.tiles_m > a.tiles_n ? slow : t - slow * fast;
    tn = a.tiles_m > a.tiles_n ? t - slow * fast : slow;
  }
}

struct Pipe {
  uint32_t s = 0, ph = 0;  // stage, and its phase
  uint32_t it = 0;         // tiles done (which accumulator), producer: stages filled
};

// The producer's warp.  `begin` waits for what the product reads, once the first tile
// is known; false: given up.
template <class L, class B>
NVFP4_DEV bool ns_produce(const Ns<L>& c, const NsArgs& a, const NsMaps& maps, Pipe& p, B begin) {
  const int num_kb = (a.k + kBK - 1) / kBK;
  int tile = c.unit, z = 0, tm = 0, tn = 0;
  int kb0 = 0, kb1 = num_kb;
  auto find = [&]() {
    if (tile >= a.tiles) return;
    int t = tile;
    if (a.splits > 1) {
      t = tile / a.splits;
      const int part = tile - t * a.splits;
      kb0 = num_kb * part / a.splits;
      kb1 = num_kb * (part + 1) / a.splits;
    }
    z = t / a.tiles_per;
    tile_of<L>(t - z * a.tiles_per, a, tm, tn);
    if (a.last >= 0) z = a.last - z;
  };
  find();
  if (!begin()) return false;
  for (; tile < a.tiles; tile += c.units, find()) {
    const int a0 = tm * L::kBM + (int)c.rank * 128;
    const int b0 = tn * L::kBN + (int)c.rank * L::kRowsB;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!all_waited(c.wait(c.empty_bar(p.s), p.ph ^ 1u, 0x71u))) return false;
      ++p.it;
      if (elect_one()) {
        const uint32_t sa = c.base + L::offA + p.s * L::kA, sb = c.base + L::offB + p.s * L::kB;
        const int k = kb * kBK;
        if (L::kPair) {
          const uint32_t fb = mapa_shared(c.full_bar(p.s), 0);
          if (c.rank == 0) mbar_arrive_expect_tx(c.full_bar(p.s), 2 * (L::kA + L::kB));
          if (a.a_mn)
            for (int i = 0; i < 2; ++i)
              tma_load_3d_pair(sa + i * kBoxMN, maps.a, fb, a0 + 64 * i, k, z);
          else
            tma_load_3d_pair(sa, maps.a, fb, k, a0, z);
          if (a.b_mn)
            for (int i = 0; i < L::kRowsB / 64; ++i)
              tma_load_3d_pair(sb + i * kBoxMN, maps.b, fb, b0 + 64 * i, k, z);
          else
            tma_load_3d_pair(sb, maps.b, fb, k, b0, z);
        } else {
          const uint32_t fb = c.full_bar(p.s);
          mbar_arrive_expect_tx(fb, L::kA + L::kB);
          if (a.a_mn)
            for (int i = 0; i < 2; ++i)
              tma_load_3d(sa + i * kBoxMN, maps.a, fb, a0 + 64 * i, k, z);
          else
            tma_load_3d(sa, maps.a, fb, k, a0, z);
          if (a.b_mn)
            for (int i = 0; i < L::kRowsB / 64; ++i)
              tma_load_3d(sb + i * kBoxMN, maps.b, fb, b0 + 64 * i, k, z);
          else
            tma_load_3d(sb, maps.b, fb, k, b0, z);
        }
      }
      __syncwarp();
      if (++p.s == L::kStages) {
        p.s = 0;
        p.ph ^= 1u;
      }
    }
  }
  return true;
}

// The MMA warp (of a pair: the first CTA's).
template <class L>
NVFP4_DEV bool ns_multiply(const Ns<L>& c, const NsArgs& a, Pipe& p) {
  const int num_kb = (a.k + kBK - 1) / kBK;
  const uint32_t idesc = idesc_f16(L::kBM, L::kBN, a.a_mn, a.b_mn);
  // a step of 16 lies 32 bytes on in K-major operands, 16 rows in others
  const uint64_t as = a.a_mn ? 2048 >> 4 : 32 >> 4, bs = a.b_mn ? 2048 >> 4 : 32 >> 4;
  for (int tile = c.unit; tile < a.tiles; tile += c.units, ++p.it) {
    const uint32_t b = p.it & 1u;
    if (!all_waited(c.wait(c.acc_empty(b), ((p.it >> 1) & 1u) ^ 1u, 0x72u))) return false;
    tc_fence_after();
    int kb0 = 0, kb1 = num_kb;
    if (a.splits > 1) {
      const int part = tile % a.splits;
      kb0 = num_kb * part / a.splits;
      kb1 = num_kb * (part + 1) / a.splits;
    }
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!all_waited(c.wait(c.full_bar(p.s), p.ph, 0x74u))) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sa = c.base + L::offA + p.s * L::kA, sb = c.base + L::offB + p.s * L::kB;
        const int left = a.k - kb * kBK;
        const uint64_t ad = a.a_mn ? smem_desc_mn(sa, kBoxMN) : smem_desc_sw128(sa);
        const uint64_t bd = a.b_mn ? smem_desc_mn(sb, kBoxMN) : smem_desc_sw128(sb);
#pragma unroll
        for (int j = 0; j < kBK / 16; ++j) {
          if (16 * j >= left) break;
          tc_mma_f16(L::kPair, c.tmem + b * L::kBN, ad + j * as, bd + j * bs, idesc,
                     kb != kb0 || j ? 1u : 0u);
        }
        if (kb == kb0) st_shared_u8(c.inject() + 1, 1u);
        c.commit(c.empty_bar(p.s));
        if (kb == kb1 - 1) c.commit(c.acc_full(b));
      }
      __syncwarp();
      if (++p.s == L::kStages) {
        p.s = 0;
        p.ph ^= 1u;
      }
    }
  }
  return true;
}

// Leaves a warp's 32 x 32 sums of a split tile in memory; the last of the parts to come
// gets the sum of all.
NVFP4_DEV bool last_part(const NsArgs& a, int item, int chunk, int chunks, int lane,
                         uint32_t (&r)[32]) {
  const int tile = item / a.splits, part = item - tile * a.splits;
  float4* first = a.part + ((int64_t)tile * a.splits * chunks + chunk) * 256 + lane;
  const int64_t step = (int64_t)chunks * 256;  // to the next part
#pragma unroll
  for (int x = 0; x < 8; ++x)
    __stcg(first + part * step + 32 * x,
           make_float4(__uint_as_float(r[4 * x]), __uint_as_float(r[4 * x + 1]),
                       __uint_as_float(r[4 * x + 2]), __uint_as_float(r[4 * x + 3])));
  __threadfence();
  __syncwarp();
  unsigned int* ticket = a.tickets + tile * chunks + chunk;
  unsigned int before = 0;
  if (lane == 0) before = atomicAdd(ticket, 1u);
  before = __shfl_sync(0xFFFFFFFFu, before, 0);
  if (before != (unsigned int)a.splits - 1u) return false;
  __threadfence();
  float4 t[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) t[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
  for (int k = 0; k < a.splits; ++k)
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float4 u = __ldcg(first + k * step + 32 * x);
      t[x].x += u.x;
      t[x].y += u.y;
      t[x].z += u.z;
      t[x].w += u.w;
    }
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    r[4 * x] = __float_as_uint(t[x].x);
    r[4 * x + 1] = __float_as_uint(t[x].y);
    r[4 * x + 2] = __float_as_uint(t[x].z);
    r[4 * x + 3] = __float_as_uint(t[x].w);
  }
  if (lane == 0) *ticket = 0;  // for the next step's
  return true;
}

// An epilogue warp's position: its next tile's accumulator, chunks sent for and done.
struct Chunks {
  uint32_t it = 0, loaded = 0, used = 0;
};

template <class L, class B>
NVFP4_DEV bool ns_finish(const Ns<L>& c, const NsArgs& a, const NsMaps& maps, Chunks& p, B begin) {
  const int ew = c.warp - 4, q = c.warp & 3, h = ew >> 2, lane = c.lane;
  uint8_t* slots = c.smem + L::offSlots + ew * (L::kSlots * L::kSlot);
  const uint32_t slot_bar = c.bar0 + 8u * (L::kSlotBar + ew * L::kSlots);
  // where this warp's chunks of a tile lie, and how many there are
  auto place = [&](int tile, int& x, int& y, int& z) {
    if (a.splits > 1) tile /= a.splits;
    z = tile / a.tiles_per;
    int tm, tn;
    tile_of<L>(tile - z * a.tiles_per, a, tm, tn);
    if (a.last >= 0) z = a.last - z;
    y = tm * L::kBM + (int)c.rank * 128 + q * 32;
    x = tn * L::kBN + h * (L::kBN / 2);
    if (y >= a.m || x >= a.n) return 0;
    const int end = a.symmetric ? min(a.n, y + 32) : a.n;  // up to the diagonal
    return max(0, min(L::kChunks, (end - x + 31) / 32));
  };
  // the loads run up to kSlots - 1 chunks ahead, over the tiles
  int ltile = a.loads ? c.unit : a.tiles, lc = 0, lcount = 0, lx = 0, ly = 0, lz = 0;
  int x0 = 0, y = 0, z = 0, count = 0;
  if (c.unit < a.tiles) count = place(c.unit, x0, y, z);
  if (a.loads) lx = x0, ly = y, lz = z, lcount = count;
  auto load_next = [&]() {
    while (ltile < a.tiles && lc >= lcount) {
      ltile += c.units;
      lc = 0;
      if (ltile < a.tiles) lcount = place(ltile, lx, ly, lz);
    }
    if (ltile >= a.tiles) return;
    if (lane == 0) {
      const uint32_t s = p.loaded % L::kSlots, bar = slot_bar + 8u * s;
      const uint32_t to = smem_u32(slots + s * L::kSlot);
      mbar_arrive_expect_tx(bar, a.loads * L::kBox);
      tma_load_3d(to, maps.in0, bar, lx + lc * 32, ly, lz);
      if (a.loads > 1) tma_load_3d(to + L::kBox, maps.in1, bar, lx + lc * 32, ly, lz);
    }
    ++p.loaded;
    ++lc;
  };
  if (!begin()) return false;
#pragma unroll 1
  for (int i = 0; i < L::kSlots - 1; ++i) load_next();
  uint32_t stores = 0;  // chunks without loads
#pragma unroll 1
  for (int tile = c.unit; tile < a.tiles; tile += c.units, ++p.it) {
    const uint32_t b = p.it & 1u;
    if (tile != c.unit) count = place(tile, x0, y, z);
    const float* din = a.din + (int64_t)z * a.dstride;
    const int row = y + lane;
    // the diagonal's entries: this row's, and of the chunk's columns the lane's
    const float di = a.by_row && row < a.m ? __ldcg(din + row) : 0.0f;
    float dj = a.by_col && count > 0 ? __ldcg(din + x0 + lane) : 0.0f;
    if (!all_waited(c.wait(c.acc_full(b), (p.it >> 1) & 1u, 0x73u))) return false;
    tc_fence_after();
#pragma unroll 1
    for (int ch = 0; ch < count; ++ch) {
      const uint32_t s = (p.used + stores) % L::kSlots;
      uint8_t* box = slots + s * L::kSlot;
      const int x = x0 + ch * 32;
      // the slot that the next load takes is free once its stores have read it
      if (lane == 0) {
        if (a.loads)
          bulk_wait_group_read<0>();
        else
          bulk_wait_group_read<L::kSlots - 1>();
      }
      __syncwarp();
      load_next();
      uint32_t r[32];
      tmem_ld32(c.tmem + ((uint32_t)(q * 32) << 16) + b * L::kBN +
                    (uint32_t)(h * (L::kBN / 2) + ch * 32),
                r);
      if (a.splits > 1) {
        tmem_ld_wait();
        if (!last_part(a, tile, ew * L::kChunks + ch, 8 * L::kChunks, lane, r)) continue;
      }
      uint32_t in0[16] = {}, in1[16] = {};
      if (a.loads) {
        if (!all_waited(c.wait(slot_bar + 8u * s, (p.used / L::kSlots) & 1u, 0x75u))) return false;
        box_get(box, lane, in0);
        if (a.loads > 1) box_get(box + L::kBox, lane, in1);
        ++p.used;
      } else {
        ++stores;
      }
      tmem_ld_wait();
      const float base = fmaf(a.q, di, a.p);
      float v[32];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 x0f = unpack_f16x2(in0[e]), x1f = unpack_f16x2(in1[e]);
        const float f0 = fmaf(a.q, __shfl_sync(0xFFFFFFFFu, dj, 2 * e), base);
        const float f1 = fmaf(a.q, __shfl_sync(0xFFFFFFFFu, dj, 2 * e + 1), base);
        v[2 * e] = fmaf(f0, x0f.x + x1f.x, __uint_as_float(r[2 * e]) * a.s);
        v[2 * e + 1] = fmaf(f1, x0f.y + x1f.y, __uint_as_float(r[2 * e + 1]) * a.s);
      }
      if (a.by_col && ch + 1 < count) dj = __ldcg(din + x + 32 + lane);
      if (a.symmetric && x == y) {
        float d = 0.0f;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          d = e == lane ? __uint_as_float(r[e]) : d;
          v[e] = e == lane ? 0.0f : v[e];
        }
        if (row < a.m)
          a.dout[(int64_t)z * a.dstride + row] = fmaf(base, di, a.t * d);
      }
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        w[e] = a.final ? pack_bf16x2(v[2 * e] * kUnscale, v[2 * e + 1] * kUnscale)
                       : pack_f16x2(v[2 * e], v[2 * e + 1]);
      __syncwarp();
      box_put(box, lane, w);
      const bool mirror = a.symmetric && x < y, both = a.loads > 1 && !a.final;
      if (both) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 hi = unpack_f16x2(w[e]);
          w[e] = pack_f16x2(v[2 * e] - hi.x, v[2 * e + 1] - hi.y);
        }
        box_put(box + L::kBox, lane, w);
      }
      __syncwarp();
      if (mirror) {
        box_transpose(smem_u32(box), smem_u32(box + L::kBox), lane);
        __syncwarp();
      }
      if (a.final && !a.out_boxes) {
        // rows of the result that do not start on 16 bytes: a row at a time
        const int rows = min(32, a.m - y);
        for (int i = 0; i < rows; ++i) {
          const uint16_t u = *reinterpret_cast<const uint16_t*>(box + box_piece(i, lane >> 3) +
                                                                (lane & 7) * 2);
          if (x + lane < a.n)
            reinterpret_cast<uint16_t*>(a.out)[((int64_t)z * a.m + y + i) * a.n + x + lane] = u;
        }
        __syncwarp();
      } else {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(maps.out0, smem_u32(box), x, y, z);
          if (mirror) tma_store_3d(maps.out0, smem_u32(box + L::kBox), y, x, z);
          if (both) tma_store_3d(maps.out1, smem_u32(box + L::kBox), x, y, z);
          bulk_commit_group();
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (L::kPair)
        mbar_arrive_cluster_relaxed(mapa_shared(c.acc_empty(b), 0));
      else
        mbar_arrive(c.acc_empty(b));
    }
  }
  return true;
}

// The coefficients of a step's product k (0: X X^T, 1: E E, 2: the update).
__host__ __device__ inline void set_coefs(NsArgs& n, int k, const float* abc, bool last) {
  n.p = k == 0 ? 0.0f : k == 1 ? abc[1] : abc[0];
  n.q = k == 0 ? 0.0f : k == 1 ? abc[2] : 1.0f;
  n.s = k == 1 ? abc[2] * kUnscale : kUnscale;
  n.t = n.s * kUnscale;
  n.final = k == 2 && last;
}

// The chunks that a warp that has given up sent for land before the block ends.
template <class L>
NVFP4_DEV void drain_chunks(const Ns<L>& c, Chunks& p) {
  const uint32_t slot_bar = c.bar0 + 8u * (L::kSlotBar + (c.warp - 4) * L::kSlots);
  for (; (int32_t)(p.loaded - p.used) > 0; ++p.used)
    wait_drain(slot_bar + 8u * (p.used % L::kSlots), (p.used / L::kSlots) & 1u);
}

// ---- a launch for each product: large matrices ---------------------------------------
// Five stages and two slots: an update of 14336 x 4096 takes 285 us, with four and three
// 313.
using PairLayout = NsLayout<true, 256, 5, 2>;

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairLayout::kThreads, 1)
    ns_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmIn0,
                   const __grid_constant__ CUtensorMap tmIn1,
                   const __grid_constant__ CUtensorMap tmOut0,
                   const __grid_constant__ CUtensorMap tmOut1, const NsArgs args) {
  using L = PairLayout;
  const Ns<L> c = ns_enter<L>();
  const NsMaps maps = {&tmA, &tmB, &tmIn0, &tmIn1, &tmOut0, &tmOut1};
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  griddep_wait();
  if (c.warp == 0) {
    Pipe p;
    if (!(ld_shared_u32(c.inject()) & kStall)) ns_produce(c, args, maps, p, [] { return true; });
    if (c.lane == 0) st_shared_u32(c.fills(), p.it);
  } else if (c.warp == 1) {
    Pipe p;
    if (c.rank == 0 && all_waited(!quits_pair(ld_shared_u32(c.inject()), c.abort_flag, c.peer_abort)))
      ns_multiply(c, args, p);
  } else if (c.warp >= 4) {
    Chunks p;
    if (!ns_finish(c, args, maps, p, [] { return true; })) drain_chunks(c, p);
    if (c.lane == 0) bulk_wait_group<0>();
  }
  ns_leave(c);
}

// ---- momentum and start ----------------------------------------------------------
// Two passes over the gradient and the momentum, bound by memory: the first
// writes V and sums U's squares (one partial sum a CTA, a matrix's are added in a
// fixed order), the second computes U again from V and G, scales it and writes
// its two halves.
constexpr int kEwThreads = 256, kEwUnroll = 4;

constexpr size_t kBarBytes = 16384;  // two counters, then the tickets
constexpr int kTicketWord = 64;
constexpr int kMaxParts = 1024;
constexpr int kWholeTiles = 2;

struct MomentumArgs {
  void* grad;
  float* momentum;
  __half *hi, *lo;
  float* partial;   // [batch][parts]
  int parts;        // CTAs of a matrix
  int64_t size;     // elements of a matrix
  int cols, ld;     // of a row, and in hi and lo
  int64_t padded;   // elements of a matrix of hi and lo
  float mu, eps;
  int nesterov, zero;
};

NVFP4_DEV float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) s += red[w];
  return s;
}

NVFP4_DEV float4 fma4(float m, const float4 v, const float4 g) {
  return make_float4(fmaf(m, v.x, g.x), fmaf(m, v.y, g.y), fmaf(m, v.z, g.z), fmaf(m, v.w, g.w));
}

// Matrix `mat` lies at elements [first, last) of the stack; its quads are the aligned
// fours that hold them, of which the ends may belong to other matrices in part.
struct Quads {
  int64_t first, last, q0, count;
};
NVFP4_DEV Quads quads_of(const MomentumArgs& a, int mat) {
  const int64_t first = (int64_t)mat * a.size, last = first + a.size;
  return {first, last, first / 4, (last + 3) / 4 - first / 4};
}
NVFP4_DEV bool whole_quad(const Quads& q, int64_t at) {
  return 4 * at >= q.first && 4 * at + 4 <= q.last;
}
NVFP4_DEV float* parts_of(float4& v) { return reinterpret_cast<float*>(&v); }

// A quad of the gradient and of the momentum; zeros outside the matrix.
template <bool WIDE>
NVFP4_DEV void load_quad(const MomentumArgs& a, const Quads& q, int64_t at, bool grad, float4& g,
                         float4& v) {
  if (whole_quad(q, at)) {
    if (grad) g = grad4_at<WIDE>(a.grad, 4 * at);
    v = *reinterpret_cast<const float4*>(a.momentum + 4 * at);
    return;
  }
  g = v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t i = 4 * at + e;
    if (i < q.first || i >= q.last) continue;
    if (grad) parts_of(g)[e] = grad_at<WIDE>(a.grad, i);
    parts_of(v)[e] = a.momentum[i];
  }
}

// Part `part` of matrix `mat`.
template <bool WIDE>
NVFP4_DEV void momentum_part(const MomentumArgs& a, int mat, int part, float* red) {
  const Quads q = quads_of(a, mat);
  const int64_t stride = (int64_t)a.parts * blockDim.x;
  float sum = 0.0f;
  for (int64_t i = (int64_t)part * blockDim.x + threadIdx.x; i < q.count; i += kEwUnroll * stride) {
    float4 g[kEwUnroll], v[kEwUnroll];
#pragma unroll
    for (int u = 0; u < kEwUnroll; ++u)
      if (i + u * stride < q.count) load_quad<WIDE>(a, q, q.q0 + i + u * stride, true, g[u], v[u]);
#pragma unroll
    for (int u = 0; u < kEwUnroll; ++u) {
      if (i + u * stride >= q.count) continue;
      const int64_t at = q.q0 + i + u * stride;
      v[u] = fma4(a.mu, v[u], g[u]);
      if (whole_quad(q, at)) {
        *reinterpret_cast<float4*>(a.momentum + 4 * at) = v[u];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * at + e >= q.first && 4 * at + e < q.last) a.momentum[4 * at + e] = parts_of(v[u])[e];
      }
      if (a.nesterov) v[u] = fma4(a.mu, v[u], g[u]);
      sum += (v[u].x * v[u].x + v[u].y * v[u].y) + (v[u].z * v[u].z + v[u].w * v[u].w);
    }
  }
  const float s = block_sum(sum, red);
  if (threadIdx.x == 0) a.partial[(int64_t)mat * a.parts + part] = s;
}

// From the matrix's end to its beginning: the first pass left the end in L2.
// FLAT: rows of a multiple of 8 elements, so hi and lo are laid out as the matrix.
template <bool WIDE, bool FLAT>
NVFP4_DEV void start_part(const MomentumArgs& a, int mat, int part, float* red) {
  float sum = 0.0f;
  for (int p = threadIdx.x; p < a.parts; p += blockDim.x)
    sum += __ldcg(a.partial + (int64_t)mat * a.parts + p);
  const float scale = start_scale(block_sum(sum, red), a.eps);
  const Quads q = quads_of(a, mat);
  const int64_t to = (int64_t)mat * a.padded, stride = (int64_t)a.parts * blockDim.x;
  for (int64_t i = (int64_t)part * blockDim.x + threadIdx.x; i < q.count; i += kEwUnroll * stride) {
    float4 g[kEwUnroll], v[kEwUnroll];
#pragma unroll
    for (int u = 0; u < kEwUnroll; ++u)
      if (i + u * stride < q.count)
        load_quad<WIDE>(a, q, q.q0 + q.count - 1 - i - u * stride, a.nesterov, g[u], v[u]);
#pragma unroll
    for (int u = 0; u < kEwUnroll; ++u) {
      if (i + u * stride >= q.count) continue;
      const int64_t at = q.q0 + q.count - 1 - i - u * stride;
      if (a.nesterov) v[u] = fma4(a.mu, v[u], g[u]);
      float* x = parts_of(v[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= scale;
      const uint32_t h[2] = {pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3])};
      const float2 h0 = unpack_f16x2(h[0]), h1 = unpack_f16x2(h[1]);
      const uint32_t l[2] = {pack_f16x2(x[0] - h0.x, x[1] - h0.y),
                             pack_f16x2(x[2] - h1.x, x[3] - h1.y)};
      const bool whole = FLAT || whole_quad(q, at);
      if (FLAT) {
        const int64_t e = to + 4 * at - q.first;
        *reinterpret_cast<uint2*>(a.hi + e) = make_uint2(h[0], h[1]);
        *reinterpret_cast<uint2*>(a.lo + e) = make_uint2(l[0], l[1]);
      } else {
        // elements before the matrix's first (of a quad shared with the one before) are
        // skipped; the first that counts gives row and column
        const int skip = (int)max((int64_t)0, q.first - 4 * at);
        const uint32_t k = (uint32_t)(4 * at + skip - q.first);
        uint32_t row = k / (uint32_t)a.cols, col = k - row * (uint32_t)a.cols;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e < skip || 4 * at + e >= q.last) continue;
          const int64_t place = to + (int64_t)row * a.ld + col;
          reinterpret_cast<uint16_t*>(a.hi)[place] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
          reinterpret_cast<uint16_t*>(a.lo)[place] = (uint16_t)(l[e >> 1] >> (16 * (e & 1)));
          if (++col == (uint32_t)a.cols) {
            col = 0;
            ++row;
          }
        }
      }
      if (a.zero) {
        if (whole) {
          if (WIDE)
            *reinterpret_cast<float4*>(static_cast<float*>(a.grad) + 4 * at) =
                make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.grad) + 4 * at) =
                make_uint2(0u, 0u);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (4 * at + e >= q.first && 4 * at + e < q.last) {
              if (WIDE)
                static_cast<float*>(a.grad)[4 * at + e] = 0.0f;
              else
                static_cast<uint16_t*>(a.grad)[4 * at + e] = 0;
            }
        }
      }
    }
  }
}

template <bool WIDE>
__global__ void __launch_bounds__(kEwThreads) momentum_kernel(const MomentumArgs a) {
  __shared__ float red[kEwThreads / 32];
  griddep_wait();
  momentum_part<WIDE>(a, blockIdx.y, blockIdx.x, red);
}
template <bool WIDE, bool FLAT>
__global__ void __launch_bounds__(kEwThreads) start_kernel(const MomentumArgs a) {
  __shared__ float red[kEwThreads / 32];
  griddep_wait();
  start_part<WIDE, FLAT>(a, gridDim.y - 1 - blockIdx.y, blockIdx.x, red);
}

// ---- one launch for all of it: matrices of some hundred rows or columns -----------
// The CTAs, one an SM, go through momentum, start and the products of every step
// together; between two products they meet at a counter: a CTA's epilogue warps tell
// its producer that their stores have been written, which counts up for all of them,
// waits for the other CTAs and lets them go on.  (Counted by every warp, 1216 additions
// to one word took longer than the products.)  A launch each costs 12 us a product here,
// most of it ends and beginnings.
struct WholeArgs {
  MomentumArgs e;
  NsArgs gram, poly, update;  // without coefficients
  unsigned int* bars;  // two counters, zero at the start
  int batch, steps, flat;
  float coefs[3 * NVFP4_MUON_MAX_STEPS];
};
struct WholeMaps {
  CUtensorMap gram_a[2], gram_b[2], poly_a, poly_b, upd_a[2], upd_b[2];
  CUtensorMap x[2], lo, e, f, out;
};

// One thread waits until a counter has come to `target`, or gives up.
NVFP4_DEV bool count_wait(const unsigned int* bar, unsigned int target, volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  const uint64_t limit = *reinterpret_cast<volatile unsigned long long*>(&g_gemm_wait_ns);
  while (true) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
    if ((int)(v - target) >= 0) break;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit) {
      *abort_flag = 1;
      atomicCAS(&g_gemm_error, 0u, 0x76u);
      return false;
    }
  }
  fence_proxy_async();
  return true;
}
NVFP4_DEV void count_up(unsigned int* bar) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(bar) : "memory");
}

// All CTAs' threads meet (before the roles part); false when the wait ran out.
template <class L>
NVFP4_DEV bool whole_barrier(const Ns<L>& c, const WholeArgs& a, unsigned int target) {
  fence_proxy_async();
  __syncthreads();
  if (threadIdx.x == 0) {
    count_up(a.bars);
    count_wait(a.bars, target, c.abort_flag);
  }
  __syncthreads();
  return *c.abort_flag == 0;
}

template <int BN>
using WholeLayout = NsLayout<false, BN, BN == 64 ? 6 : 4, BN == 64 ? 2 : 3>;

template <int BN, bool WIDE>
__global__ void __launch_bounds__(WholeLayout<BN>::kThreads, 1)
    whole_kernel(const __grid_constant__ WholeMaps maps, const __grid_constant__ WholeArgs a) {
  using L = WholeLayout<BN>;
  __shared__ float red[L::kThreads / 32];
  const Ns<L> c = ns_enter<L>();
  if (threadIdx.x < sizeof(WholeMaps) / sizeof(CUtensorMap))
    prefetch_tmap(reinterpret_cast<const CUtensorMap*>(&maps) + threadIdx.x);
  const int items = a.batch * a.e.parts;
  for (int w = blockIdx.x; w < items; w += gridDim.x) {
    const int mat = w / a.e.parts, part = w - mat * a.e.parts;
    momentum_part<WIDE>(a.e, mat, part, red);
  }
  bool ok = whole_barrier(c, a, gridDim.x);
  if (ok) {
    for (int w = blockIdx.x; w < items; w += gridDim.x) {
      const int mat = w / a.e.parts, part = w - mat * a.e.parts;
      if (a.flat)
        start_part<WIDE, true>(a.e, mat, part, red);
      else
        start_part<WIDE, false>(a.e, mat, part, red);
    }
    ok = whole_barrier(c, a, 2 * gridDim.x);
  }
  unsigned int* bar = a.bars + 32;
  const uint32_t done_bar = c.bar0 + 8u * L::kDoneBar, go_bar = c.bar0 + 8u * L::kGoBar;
  if (!ok) {
  } else if (c.warp == 0) {
    Pipe p;
    unsigned int products = 0;  // behind
    // the product before is done, in all CTAs
    auto meet = [&]() {
      bool k = c.wait(done_bar, products & 1u, 0x77u);
      ++products;
      if (c.lane == 0 && k) {
        count_up(bar);
        k = count_wait(bar, products * gridDim.x, c.abort_flag);
        if (k) mbar_arrive(go_bar);
      }
      k = all_waited(k);
      fence_proxy_async();
      return k;
    };
    fence_proxy_async();
    ok = !(ld_shared_u32(c.inject()) & kStall);
    for (int step = 0; ok && step < a.steps; ++step) {
      const int x = step & 1;
      const NsMaps g = {&maps.gram_a[x], &maps.gram_b[x]}, q = {&maps.poly_a, &maps.poly_b},
                   u = {&maps.upd_a[x], &maps.upd_b[x]};
#pragma unroll 1
      for (int k = 0; ok && k < 3; ++k)
        ok = ns_produce(c, k == 0 ? a.gram : k == 1 ? a.poly : a.update,
                        k == 0 ? g : k == 1 ? q : u, p,
                        [&] { return step + k == 0 || meet(); });
    }
    if (c.lane == 0) st_shared_u32(c.fills(), p.it);
  } else if (c.warp == 1) {
    Pipe p;
    ok = all_waited(!quits(ld_shared_u32(c.inject()), c.abort_flag));
#pragma unroll 1
    for (int i = 0; ok && i < 3 * a.steps; ++i)
      ok = ns_multiply(c, i % 3 == 0 ? a.gram : i % 3 == 1 ? a.poly : a.update, p);
  } else if (c.warp >= 4) {
    Chunks p;
    uint32_t products = 0;
    // a product's end for this warp: its stores have been written, and it says so
    auto next = [&]() {
      __syncwarp();
      if (c.lane == 0) {
        bulk_wait_group<0>();
        fence_proxy_async();
        mbar_arrive(done_bar);
      }
    };
    auto meet = [&]() {
      const bool k = all_waited(c.wait(go_bar, products & 1u, 0x78u));
      ++products;
      fence_proxy_async();
      return k;
    };
    fence_proxy_async();
#pragma unroll 1
    for (int i = 0; ok && i < 3 * a.steps; ++i) {
      const int step = i / 3, k = i - 3 * step, x = step & 1;
      const bool last = step == a.steps - 1;
      NsArgs n = k == 0 ? a.gram : k == 1 ? a.poly : a.update;
      set_coefs(n, k, a.coefs + 3 * step, last);
      NsMaps t = {};
      t.in0 = k == 1 ? &maps.e : &maps.x[x];
      t.in1 = t.out1 = &maps.lo;
      t.out0 = k == 0 ? &maps.e : k == 1 ? &maps.f : last ? &maps.out : &maps.x[x ^ 1];
      ok = ns_finish(c, n, t, p, [&] { return i == 0 || meet(); });
      if (ok && i < 3 * a.steps - 1) next();
    }
    if (!ok) drain_chunks(c, p);
    if (c.lane == 0) bulk_wait_group<0>();
  }
  ns_leave(c);
}

// ---- host side -----------------------------------------------------------------
// 3-D map over 16-bit matrices [batch][rows][cols] with leading dimension ld.
bool make_map(CUtensorMap* map, const void* base, int64_t batch, int64_t rows, int64_t cols,
              int64_t ld, int box_cols, int box_rows, bool bf16 = false) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * 2), (cuuint64_t)(rows * ld * 2)};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             box_cols == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How a product's tiles lie.
void set_tiles(NsArgs& a, int64_t batch, int bm, int bn) {
  a.tiles_m = (a.m + bm - 1) / bm;
  a.tiles_n = (a.n + bn - 1) / bn;
  const int per = bm / bn;  // a row's tiles up to the diagonal rise by these; past the
  a.tiles_per = a.symmetric  // matrix's end there may be some, which have no chunks
                    ? per * (a.tiles_m * (a.tiles_m + 1) / 2)
                    : a.tiles_m * a.tiles_n;
  a.splits = 1;
  a.tiles = (int)(a.tiles_per * batch);
}

nvfp4_status launch_ns(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& in0,
                       const CUtensorMap& in1, const CUtensorMap& out0, const CUtensorMap& out1,
                       NsArgs a, int64_t batch, int sms, cudaStream_t stream) {
  using L = PairLayout;
  static GemmLaunchState ls;
  auto kern = ns_pair_kernel;
  const int units = gemm_setup(ls, kern, L::kAlloc, L::kThreads, 0, 2, sms);
  if (units <= 0) return NVFP4_ERR_CUDA;
  set_tiles(a, batch, L::kBM, L::kBN);
  return cuda_status(launch_pdl(kern, 2 * std::min(units, a.tiles), L::kThreads, L::kAlloc, stream,
                                ma, mb, in0, in1, out0, out1, a));
}

template <int BN, bool WIDE>
nvfp4_status launch_whole(const WholeMaps& maps, WholeArgs& a, int sms, cudaStream_t stream) {
  using L = WholeLayout<BN>;
  static GemmLaunchState ls;
  auto kern = whole_kernel<BN, WIDE>;
  if (gemm_setup(ls, kern, L::kAlloc, L::kThreads, 0, 1, sms) <= 0) return NVFP4_ERR_CUDA;
  set_tiles(a.gram, a.batch, L::kBM, BN);
  set_tiles(a.poly, a.batch, L::kBM, BN);
  set_tiles(a.update, a.batch, L::kBM, BN);
  // Long contractions of few tiles are shared by the CTAs that have none, 1024 a part at
  // least (us, whole and in parts, all steps: 256 x 8192 268, 172; 1024 x 1024 in two
  // 137, 146).
  const int parts = std::min({16, sms / a.gram.tiles, a.gram.k / 1024});
  if (parts > 1) {
    a.gram.splits = parts;
    a.gram.tiles *= parts;
  }
  if (cudaMemsetAsync(a.bars, 0, kBarBytes, stream) != cudaSuccess) return NVFP4_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  // no more CTAs than have a tile, or a share of the momentum
  const int64_t share = (a.e.size * a.batch + 8191) / 8192;
  const int ctas = (int)std::min<int64_t>(
      sms, std::max<int64_t>({share, a.gram.tiles, a.poly.tiles, a.update.tiles}));
  a.e.parts = (int)std::min<int64_t>(kMaxParts, std::max<int64_t>(1, ctas / a.batch));
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;  // the CTAs wait on one another
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, maps, a));
}

// Where the parts of a workspace lie.
struct Layout {
  int64_t m, n;          // the matrix's smaller and larger side
  int64_t ldx, ldm, dstride;
  size_t x_bytes, g_bytes, d_bytes;
  size_t total;
  bool panel;
};
constexpr int64_t kMaxSide = 1 << 20;

// Whether one launch does it all: as long as an update has no more than two rounds of
// 128 x 128 tiles, or X X^T in tiles of 256 x 256 would leave three quarters of the SMs
// idle through a long contraction, which the one launch splits.  Measured (us, one launch
// and a launch each): 200 x 328 90, 140; 1024 x 1024 141, 195; 2048 x 2048 285, 277; 2 x
// [2048, 2048] 489, 355; 2048 x 4096 438, 379; by tiles of X X^T: 3, 512 x 16384 300, 541;
// 9, 3 x [348, 14268] 409, 652; 10, 1024 x 8192 331, 401; 16, 16 x [256, 8192] 600, 622; 20,
// 2 x [1024, 4096] 327, 321; 32, 32 x [256, 8192] 1113, 994.
bool takes_whole(const Layout& l, int64_t batch, int sms) {
  const int64_t t = (l.m + 255) / 256;
  return ((l.m + 127) / 128) * ((l.n + 127) / 128) * batch <= kWholeTiles * sms ||
         t * (t + 1) / 2 * batch * 8 <= sms;
}
// Its tiles' width: 64 while every CTA has one of an update (us, 64 and 128 wide: 1024 x
// 1024 142, 168; 3 x [777, 1290] 242, 211; 2048 x 2048 432, 293).
int whole_width(const Layout& l, int64_t batch, int sms) {
  return ((l.m + 127) / 128) * ((l.n + 63) / 64) * batch <= sms ? 64 : 128;
}

nvfp4_status muon_layout(int64_t batch, int64_t rows, int64_t cols, Layout* l) {
  if (batch <= 0 || rows <= 0 || cols <= 0 || batch > 65535 || rows > kMaxSide || cols > kMaxSide)
    return NVFP4_ERR_SHAPE;
  if (rows * cols > INT32_MAX || std::min(rows, cols) > 32768) return NVFP4_ERR_SHAPE;
  l->m = std::min(rows, cols);
  l->n = std::max(rows, cols);
  l->ldx = (cols + 7) / 8 * 8;
  l->ldm = (l->m + 7) / 8 * 8;
  l->dstride = (l->m + 31) / 32 * 32;
  const int64_t tm = (l->m + 255) / 256, tn = (l->n + 255) / 256;
  if (tm * tn * batch > INT32_MAX / 2) return NVFP4_ERR_SHAPE;
  l->x_bytes = up1k((size_t)batch * rows * l->ldx * 2);
  l->g_bytes = up1k((size_t)batch * l->m * l->ldm * 2);
  l->d_bytes = up1k((size_t)batch * l->dstride * 4);
  l->panel = muon_panel_fits(rows, cols);
  l->total = l->panel ? muon_panel_workspace(rows, cols)
                      : 3 * l->x_bytes + 2 * l->g_bytes + 2 * l->d_bytes +
                            up1k((size_t)batch * kMaxParts * 4) + kBarBytes +
                            (takes_whole(*l, batch, kMaxSms) ? (size_t)kMaxSms * 128 * 128 * 4 : 0);
  return NVFP4_OK;
}

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

}  // namespace

nvfp4_status muon_set_injection(unsigned int stall, unsigned long long wait_ns) {
  if (cudaMemcpyToSymbol(g_gemm_stall, &stall, sizeof(stall)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_gemm_wait_ns, &wait_ns, sizeof(wait_ns)) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return muon_panel_set_injection(stall, wait_ns);
}

nvfp4_status muon_read_error(unsigned int* code) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemm_error, sizeof(v)) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (v && cudaMemcpyToSymbol(g_gemm_error, &zero, sizeof(zero)) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  unsigned int panel = 0;
  const nvfp4_status st = muon_panel_read_error(&panel);
  *code = v ? v : panel;
  return st;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_muon_sizes(int64_t batch, int64_t rows, int64_t cols,
                                         size_t* workspace_bytes) {
  Layout l;
  const nvfp4_status st = muon_layout(batch, rows, cols, &l);
  if (st != NVFP4_OK) return st;
  if (workspace_bytes) *workspace_bytes = l.total;
  return NVFP4_OK;
}

extern "C" nvfp4_status nvfp4_muon_update(const nvfp4_muon_params* p, void* grad, float* momentum,
                                          void* update, uint32_t flags, void* workspace,
                                          size_t workspace_bytes, nvfp4_stream stream) {
  if (!p || !grad || !momentum || !update || !p->coefs || (flags & ~(uint32_t)NVFP4_ZERO_GRAD))
    return NVFP4_ERR_INVALID_ARG;
  if (p->grad_dtype != NVFP4_IN_BF16 && p->grad_dtype != NVFP4_IN_FP32)
    return NVFP4_ERR_INVALID_ARG;
  if (p->nesterov < 0 || p->nesterov > 1 || p->steps < 1 || p->steps > NVFP4_MUON_MAX_STEPS ||
      !std::isfinite(p->mu) || !(p->eps > 0.0f) || !std::isfinite(p->eps))
    return NVFP4_ERR_INVALID_ARG;
  for (int i = 0; i < 3 * p->steps; ++i)
    if (!std::isfinite(p->coefs[i])) return NVFP4_ERR_INVALID_ARG;
  Layout l;
  nvfp4_status st = muon_layout(p->batch, p->rows, p->cols, &l);
  if (st != NVFP4_OK) return st;
  const bool wide = p->grad_dtype == NVFP4_IN_FP32;
  const size_t count = (size_t)(p->batch * p->rows * p->cols);
  if (overlap(grad, count * (wide ? 4 : 2), momentum, count * 4) ||
      overlap(grad, count * (wide ? 4 : 2), update, count * 2) ||
      overlap(momentum, count * 4, update, count * 2))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned16(grad) || !aligned16(momentum) || !aligned16(update)) return NVFP4_ERR_ALIGN;
  if (!workspace || !aligned16(workspace) || workspace_bytes < l.total) return NVFP4_ERR_WORKSPACE;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (l.panel)
    return muon_panel({p, grad, momentum, static_cast<__nv_bfloat16*>(update), wide,
                       (flags & NVFP4_ZERO_GRAD) != 0, workspace, dev.sm_count, s});

  uint8_t* w = static_cast<uint8_t*>(workspace);
  void* hi[2] = {w, w + l.x_bytes};
  void* lo = w + 2 * l.x_bytes;
  void* E = w + 3 * l.x_bytes;
  void* F = w + 3 * l.x_bytes + l.g_bytes;
  float* d = reinterpret_cast<float*>(w + 3 * l.x_bytes + 2 * l.g_bytes);
  float* db = reinterpret_cast<float*>(w + 3 * l.x_bytes + 2 * l.g_bytes + l.d_bytes);

  MomentumArgs e = {};
  e.grad = grad;
  e.momentum = momentum;
  e.hi = static_cast<__half*>(hi[0]);
  e.lo = static_cast<__half*>(lo);
  e.partial = reinterpret_cast<float*>(w + 3 * l.x_bytes + 2 * l.g_bytes + 2 * l.d_bytes);
  e.size = p->rows * p->cols;
  e.cols = (int)p->cols;
  e.ld = (int)l.ldx;
  e.padded = p->rows * l.ldx;
  e.mu = p->mu;
  e.eps = p->eps;
  e.nesterov = p->nesterov;
  e.zero = (flags & NVFP4_ZERO_GRAD) != 0;
  const bool tall = p->rows > p->cols, whole = takes_whole(l, p->batch, dev.sm_count);
  const int bn = whole ? whole_width(l, p->batch, dev.sm_count) : 256;
  const int b_rows = whole ? bn : 128;  // rows of B that a CTA loads at a time
  const bool flat = p->cols % 8 == 0;
  WholeMaps t;
  bool ok = true;
  const int64_t mm = l.m;
  for (int i = 0; i < 2; ++i) {
    auto x = [&](CUtensorMap* map, int box_cols, int box_rows) {
      ok = ok && make_map(map, hi[i], p->batch, p->rows, p->cols, l.ldx, box_cols, box_rows);
    };
    x(&t.gram_a[i], 64, tall ? 64 : 128);
    x(&t.gram_b[i], 64, tall ? 64 : b_rows);
    x(&t.x[i], 32, 32);
    if (tall) {
      x(&t.upd_a[i], 64, 128);
      ok = ok && make_map(&t.upd_b[i], F, p->batch, mm, mm, l.ldm, 64, b_rows);
    } else {
      ok = ok && make_map(&t.upd_a[i], F, p->batch, mm, mm, l.ldm, 64, 128);
      x(&t.upd_b[i], 64, 64);
    }
  }
  ok = ok && make_map(&t.poly_a, E, p->batch, mm, mm, l.ldm, 64, 128) &&
       make_map(&t.poly_b, E, p->batch, mm, mm, l.ldm, 64, b_rows) &&
       make_map(&t.e, E, p->batch, mm, mm, l.ldm, 32, 32) &&
       make_map(&t.f, F, p->batch, mm, mm, l.ldm, 32, 32) &&
       make_map(&t.lo, lo, p->batch, p->rows, p->cols, l.ldx, 32, 32);
  if (flat)
    ok = ok && make_map(&t.out, update, p->batch, p->rows, p->cols, p->cols, 32, 32, true);
  else
    t.out = t.lo;  // not read
  if (!ok) return NVFP4_ERR_CUDA;

  NsArgs gram = {}, poly, upd;
  gram.m = gram.n = (int)l.m;
  gram.k = (int)l.n;
  gram.a_mn = gram.b_mn = tall;
  gram.symmetric = 1;
  gram.din = gram.dout = d;
  gram.dstride = l.dstride;
  gram.last = -1;
  poly = gram;
  poly.k = (int)l.m;
  poly.a_mn = poly.b_mn = 0;
  poly.loads = poly.by_row = poly.by_col = 1;
  poly.dout = db;
  upd = poly;
  upd.m = (int)p->rows;
  upd.n = (int)p->cols;
  upd.b_mn = !tall;
  upd.symmetric = 0;
  upd.loads = 2;
  upd.by_row = !tall;
  upd.by_col = tall;
  upd.din = db;
  upd.out = static_cast<__nv_bfloat16*>(update);
  upd.out_boxes = flat;

  if (whole) {
    WholeArgs a = {};
    a.e = e;
    a.gram = gram;
    a.poly = poly;
    a.update = upd;
    a.bars = reinterpret_cast<unsigned int*>(reinterpret_cast<uint8_t*>(e.partial) +
                                             up1k((size_t)p->batch * kMaxParts * 4));
    a.gram.tickets = a.bars + kTicketWord;
    a.gram.part = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(a.bars) + kBarBytes);
    a.batch = (int)p->batch;
    a.steps = p->steps;
    a.flat = flat;
    std::copy(p->coefs, p->coefs + 3 * p->steps, a.coefs);
    if (bn == 64)
      return wide ? launch_whole<64, true>(t, a, dev.sm_count, s)
                  : launch_whole<64, false>(t, a, dev.sm_count, s);
    return wide ? launch_whole<128, true>(t, a, dev.sm_count, s)
                : launch_whole<128, false>(t, a, dev.sm_count, s);
  }

  const int64_t want = std::max<int64_t>(1, (e.size + kEwThreads * 16 - 1) / (kEwThreads * 16));
  const int64_t fit = std::max<int64_t>(1, (int64_t)dev.sm_count * 8 / p->batch);
  e.parts = (int)std::min<int64_t>({want, fit, kMaxParts});
  const dim3 grid((unsigned)e.parts, (unsigned)p->batch);
  auto k1 = wide ? momentum_kernel<true> : momentum_kernel<false>;
  auto k2 = wide ? (flat ? start_kernel<true, true> : start_kernel<true, false>)
                 : (flat ? start_kernel<false, true> : start_kernel<false, false>);
  if (launch_pdl(k1, grid, kEwThreads, 0, s, e) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (launch_pdl(k2, grid, kEwThreads, 0, s, e) != cudaSuccess) return NVFP4_ERR_CUDA;
  for (int i = 0; i < p->steps; ++i) {
    const int x = i & 1;
    const bool last = i == p->steps - 1;
    const float* abc = p->coefs + 3 * i;
    set_coefs(gram, 0, abc, last);
    set_coefs(poly, 1, abc, last);
    set_coefs(upd, 2, abc, last);
    // every launch goes through the matrices the other way than the one before, whose
    // last results are in L2 (64 x [1024, 2048]: 2547 us, 2570 without)
    gram.last = upd.last = i & 1 ? (int)p->batch - 1 : -1;
    poly.last = i & 1 ? -1 : (int)p->batch - 1;
    st = launch_ns(t.gram_a[x], t.gram_b[x], t.e, t.e, t.e, t.e, gram, p->batch,
                          dev.sm_count, s);
    if (st != NVFP4_OK) return st;
    st = launch_ns(t.poly_a, t.poly_b, t.e, t.e, t.f, t.f, poly, p->batch, dev.sm_count, s);
    if (st != NVFP4_OK) return st;
    st = launch_ns(t.upd_a[x], t.upd_b[x], t.x[x], t.lo, last ? t.out : t.x[x ^ 1], t.lo, upd,
                         p->batch, dev.sm_count, s);
    if (st != NVFP4_OK) return st;
  }
  return NVFP4_OK;
}
