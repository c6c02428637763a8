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
#include <cmath>

#include "muon_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kTile = 256;  // rows and columns of a CTA pair's tile
constexpr int kBK = 64;     // contraction elements of a stage, 128 bytes

// What a product computes and what becomes of it.
enum {
  kGram = 0,    // E, D of X X^T; symmetric
  kPoly = 1,    // F, D' from E E; symmetric
  kUpdate = 2,  // X' = (a + d') X + F X
  kFinal = 3    // the same, stored as bf16
};

struct NsArgs {
  int m, n, k;             // the product's rows, columns and contraction
  int tiles_m, tiles_n;
  int tiles_per, tiles;    // of a matrix, of all
  float a, b, c;
  int by_col;              // update: d' belongs to the columns (tall matrices)
  const float* din;        // poly: d; update: d'
  float* dout;             // gram: d; poly: d'
  int64_t dstride;         // from one matrix's diagonal to the next's
  __nv_bfloat16* out;      // final
  int out_boxes;           // final: rows are whole multiples of 16 bytes
};

// A warp goes on only together: its lanes may give up at a wait one by one.
NVFP4_DEV bool all_waited(bool ok) { return __all_sync(0xFFFFFFFFu, ok); }

// An MN-major operand lies in boxes of 64 (along M or N) x 64 (along K).
constexpr uint32_t kBoxMN = 64 * kBK * 2;

NVFP4_DEV void tc_mma_pair_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                               uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
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

// Tile t of a matrix: by rows of the lower triangle where the result is
// symmetric, else with the matrix's smaller side running fastest: tiles at work
// together then read X, the operand that L2 may not hold, once (14336 x 4096: an
// update 375 us the other way round, 488 ns a stage).
template <int KIND>
NVFP4_DEV void tile_of(int t, const NsArgs& a, int& tm, int& tn) {
  if (KIND <= kPoly) {
    tm = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
    while (tm * (tm + 1) / 2 > t) --tm;
    tn = t - tm * (tm + 1) / 2;
  } else {
    const int fast = min(a.tiles_m, a.tiles_n), slow = t / fast;
    tm = a.tiles_m > a.tiles_n ? slow : t - slow * fast;
    tn = a.tiles_m > a.tiles_n ? t - slow * fast : slow;
  }
}

// =============================================================================
// CTA-pair kernel: persistent pairs, tiles of 256 x 256, contraction 64 a stage
// (tcgen05 cta_group::2 kind::f16, K = 16 an instruction).  CTA r loads rows
// [128 r, 128 r + 128) of A and of B; two accumulators in tensor memory, so a
// tile's epilogue runs under the next one's MMAs.  8 epilogue warps of each CTA
// take 32 rows x 32 columns at a time through a slot of two boxes: what the
// chunk needs (E, or X's two halves) comes in ahead by tensor loads, the results
// go out of the same boxes by tensor stores.  Of a symmetric product the tiles
// on and below the diagonal are computed, and the others are their transposes,
// through ldmatrix and stmatrix.  Rows, columns and contraction behind a
// matrix's end are filled with zeros by the loads and left out by the stores.
// =============================================================================
template <int KIND>
struct NsLayout {
  static constexpr int kStages = KIND == kGram ? 5 : 4;
  static constexpr int kSlots = KIND == kGram ? 2 : 3;  // of an epilogue warp
  static constexpr uint32_t kA = 128 * kBK * 2, kB = kA;
  static constexpr uint32_t kBox = 32 * 64, kSlot = 2 * kBox;
  static constexpr uint32_t offA = 0, offB = offA + kStages * kA;
  static constexpr uint32_t offSlots = offB + kStages * kB;
  static constexpr uint32_t offBar = offSlots + 8 * kSlots * kSlot;
  // full, empty per stage, accumulator full and empty, and the drains' barrier
  // where pair_leave looks for it; then one per epilogue warp and slot
  static constexpr uint32_t kAccBar = 2 * kStages, kDrainBar = 4 * kStages + 2;
  static constexpr uint32_t kSlotBar = kDrainBar + 3;
  static constexpr uint32_t offMisc = offBar + (kSlotBar + 8 * kSlots) * 8;
  static constexpr uint32_t kAlloc = offMisc + 16 + 1024;
  static constexpr int kThreads = 384;
  static_assert(kAlloc <= 232448, "shared memory overflow");
  static_assert(offSlots % 1024 == 0 && kAccBar + 4 <= kDrainBar, "layout");
};

template <int KIND, bool AMN, bool BMN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NsLayout<KIND>::kThreads, 1)
    ns_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmIn0,
                   const __grid_constant__ CUtensorMap tmIn1,
                   const __grid_constant__ CUtensorMap tmOut0,
                   const __grid_constant__ CUtensorMap tmOut1, const NsArgs args) {
  using L = NsLayout<KIND>;
  constexpr int S = L::kStages;
  constexpr bool kSym = KIND <= kPoly;
  constexpr int kLoads = KIND == kGram ? 0 : KIND == kPoly ? 1 : 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::offBar;
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (S + s); };
  auto acc_full = [&](uint32_t b) { return bar0 + 8u * (L::kAccBar + b); };
  auto acc_empty = [&](uint32_t b) { return bar0 + 8u * (L::kAccBar + 2 + b); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::offMisc + 4);
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t peer_abort = mapa_shared(smem_u32(smem + L::offMisc + 4), rank ^ 1u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.x / 2, num_units = gridDim.x / 2;
  const uint32_t fills = sbase + L::offMisc + 8, inject = fills + 4;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 16);  // 8 epilogue warps in each CTA
    }
    mbar_init(bar0 + 8u * L::kDrainBar, 1);
    for (int w = 0; w < 8 * L::kSlots; ++w) mbar_init(bar0 + 8u * (L::kSlotBar + w), 1);
    *abort_flag = 0;
    st_shared_u32(inject, injected());
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  griddep_wait();
  const uint32_t tmem = *tmem_slot;
  const int num_kb = (args.k + kBK - 1) / kBK;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      prefetch_tmap(&tmA);
      prefetch_tmap(&tmB);
      uint32_t s = 0, ph = 0, count = 0;
      bool ok = !(ld_shared_u32(inject) & kStall);
      for (int tile = unit; ok && tile < args.tiles; tile += num_units) {
        const int z = tile / args.tiles_per;
        int tm, tn;
        tile_of<KIND>(tile - z * args.tiles_per, args, tm, tn);
        const int a0 = tm * kTile + (int)rank * 128, b0 = tn * kTile + (int)rank * 128;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!wait_bounded_pair(empty_bar(s), ph ^ 1u, abort_flag, peer_abort, 0x71u)) {
            ok = false;
            break;
          }
          ++count;
          const uint32_t fb = mapa_shared(full_bar(s), 0);
          const uint32_t sa = sbase + L::offA + s * L::kA, sb = sbase + L::offB + s * L::kB;
          if (leader) mbar_arrive_expect_tx(full_bar(s), 2 * (L::kA + L::kB));
          if (AMN) {
            tma_load_3d_pair(sa, &tmA, fb, a0, kb * kBK, z);
            tma_load_3d_pair(sa + kBoxMN, &tmA, fb, a0 + 64, kb * kBK, z);
          } else {
            tma_load_3d_pair(sa, &tmA, fb, kb * kBK, a0, z);
          }
          if (BMN) {
            tma_load_3d_pair(sb, &tmB, fb, b0, kb * kBK, z);
            tma_load_3d_pair(sb + kBoxMN, &tmB, fb, b0 + 64, kb * kBK, z);
          } else {
            tma_load_3d_pair(sb, &tmB, fb, kb * kBK, b0, z);
          }
          if (++s == S) { s = 0; ph ^= 1u; }
        }
      }
      st_shared_u32(fills, count);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------------------------------------------------------- MMA
      constexpr uint32_t idesc = idesc_f16(256, kTile, AMN, BMN);
      uint32_t s = 0, ph = 0, it = 0;
      bool ok = !quits_pair(ld_shared_u32(inject), abort_flag, peer_abort);
      for (int tile = unit; ok && tile < args.tiles; tile += num_units, ++it) {
        const uint32_t b = it & 1u;
        if (!wait_bounded_pair(acc_empty(b), ((it >> 1) & 1u) ^ 1u, abort_flag, peer_abort,
                               0x72u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!wait_bounded_pair(full_bar(s), ph, abort_flag, peer_abort, 0x74u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = sbase + L::offA + s * L::kA, sb = sbase + L::offB + s * L::kB;
          const int left = args.k - kb * kBK;
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j) {
            if (16 * j >= left) break;
            const uint64_t ad = AMN ? smem_desc_mn(sa + 2048 * j, kBoxMN) : smem_desc_sw128(sa + 32 * j);
            const uint64_t bd = BMN ? smem_desc_mn(sb + 2048 * j, kBoxMN) : smem_desc_sw128(sb + 32 * j);
            tc_mma_pair_f16(tmem + b * kTile, ad, bd, idesc, kb | j ? 1u : 0u);
          }
          st_shared_u8(inject + warp, 1u);
          tc_commit_pair(empty_bar(s), (uint16_t)3);
          if (++s == S) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(acc_full(b), (uint16_t)3);
      }
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------------- epilogue
    const int ew = warp - 4, q = warp & 3, h = ew >> 2;
    uint8_t* slots = smem + L::offSlots + ew * (L::kSlots * L::kSlot);
    const uint32_t slot_bar = bar0 + 8u * (L::kSlotBar + ew * L::kSlots);
    if (lane == 0) {
      prefetch_tmap(&tmOut0);
      prefetch_tmap(&tmOut1);
    }
    // where this warp's chunks of a tile lie, and how many there are
    auto place = [&](int tile, int& x, int& y, int& z, int& tm, int& tn) {
      z = tile / args.tiles_per;
      tile_of<KIND>(tile - z * args.tiles_per, args, tm, tn);
      y = tm * kTile + (int)rank * 128 + q * 32;
      x = tn * kTile + h * 128;
      return y < args.m && x < args.n ? min(4, (args.n - x + 31) / 32) : 0;
    };
    // the loads run up to kSlots - 1 chunks ahead, over the tiles
    int ltile = unit, lc = 0;
    uint32_t loaded = 0;
    bool lmore = kLoads > 0;
    auto load_next = [&]() {
      if (!lmore) return;
      int x, y, z, tm, tn, count = 0;
      while (ltile < args.tiles && lc >= (count = place(ltile, x, y, z, tm, tn))) {
        ltile += num_units;
        lc = 0;
      }
      if (ltile >= args.tiles) {
        lmore = false;
        return;
      }
      if (lane == 0) {
        const uint32_t s = loaded % L::kSlots, bar = slot_bar + 8u * s;
        const uint32_t to = smem_u32(slots + s * L::kSlot);
        mbar_arrive_expect_tx(bar, kLoads * L::kBox);
        tma_load_3d(to, &tmIn0, bar, x + lc * 32, y, z);
        if (kLoads > 1) tma_load_3d(to + L::kBox, &tmIn1, bar, x + lc * 32, y, z);
      }
      ++loaded;
      ++lc;
    };
    for (int i = 0; i < L::kSlots - 1; ++i) load_next();
    uint32_t it = 0, used = 0;
    bool ok = true;
    for (int tile = unit; ok && tile < args.tiles; tile += num_units, ++it) {
      const uint32_t b = it & 1u;
      int x0, y, z, tm, tn;
      const int count = place(tile, x0, y, z, tm, tn);
      if (!all_waited(wait_bounded_pair(acc_full(b), (it >> 1) & 1u, abort_flag, peer_abort,
                                        0x73u))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool mirror = kSym && tm != tn;
      const float* din = args.din + (int64_t)z * args.dstride;
      const int row = y + lane;
      float di = 0.0f;
      if ((KIND == kPoly || (KIND >= kUpdate && !args.by_col)) && row < args.m) di = din[row];
      for (int c = 0; c < count; ++c, ++used) {
        const uint32_t s = used % L::kSlots;
        uint8_t* box = slots + s * L::kSlot;
        const int x = x0 + c * 32;
        // the slot of the chunk before last is free once its stores have read it
        if (lane == 0) {
          if (kLoads)
            bulk_wait_group_read<0>();
          else
            bulk_wait_group_read<L::kSlots - 1>();
        }
        __syncwarp();
        load_next();
        uint32_t r[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + b * kTile + (uint32_t)(h * 128 + c * 32), r);
        uint32_t in0[16], in1[16];
        if (kLoads) {
          if (!all_waited(wait_bounded_pair(slot_bar + 8u * s, (used / L::kSlots) & 1u, abort_flag,
                                            peer_abort, 0x75u))) {
            ok = false;
            break;
          }
          box_get(box, lane, in0);
          if (kLoads > 1) box_get(box + L::kBox, lane, in1);
        }
        tmem_ld_wait();
        uint32_t w0[16], w1[16];
        float v[32];
        if constexpr (KIND == kGram) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]) * kUnscale;
          if (x == y) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e == lane) {
                if (row < args.m) args.dout[(int64_t)z * args.dstride + row] = v[e] * kUnscale;
                v[e] = 0.0f;
              }
          }
        } else if constexpr (KIND == kPoly) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 f = unpack_f16x2(in0[e]);
            const float2 dj = *reinterpret_cast<const float2*>(din + x + 2 * e);
            v[2 * e] = args.b * f.x +
                       args.c * (__uint_as_float(r[2 * e]) * kUnscale + (di + dj.x) * f.x);
            v[2 * e + 1] = args.b * f.y +
                           args.c * (__uint_as_float(r[2 * e + 1]) * kUnscale + (di + dj.y) * f.y);
          }
          if (x == y) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e == lane) {
                const float sq = __uint_as_float(r[e]) * (kUnscale * kUnscale);
                if (row < args.m)
                  args.dout[(int64_t)z * args.dstride + row] = args.b * di + args.c * (di * di + sq);
                v[e] = 0.0f;
              }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 hi = unpack_f16x2(in0[e]), lo = unpack_f16x2(in1[e]);
            float2 d = make_float2(di, di);
            if (args.by_col) d = *reinterpret_cast<const float2*>(din + x + 2 * e);
            v[2 * e] = (args.a + d.x) * (hi.x + lo.x) + __uint_as_float(r[2 * e]) * kUnscale;
            v[2 * e + 1] =
                (args.a + d.y) * (hi.y + lo.y) + __uint_as_float(r[2 * e + 1]) * kUnscale;
          }
        }
        if constexpr (KIND == kFinal) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w0[e] = pack_bf16x2(v[2 * e] * kUnscale, v[2 * e + 1] * kUnscale);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) w0[e] = pack_f16x2(v[2 * e], v[2 * e + 1]);
        }
        if constexpr (KIND == kUpdate) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 hi = unpack_f16x2(w0[e]);
            w1[e] = pack_f16x2(v[2 * e] - hi.x, v[2 * e + 1] - hi.y);
          }
        }
        __syncwarp();
        box_put(box, lane, w0);
        if (KIND == kUpdate) box_put(box + L::kBox, lane, w1);
        __syncwarp();
        if (mirror) {
          box_transpose(smem_u32(box), smem_u32(box + L::kBox), lane);
          __syncwarp();
        }
        if (KIND == kFinal && !args.out_boxes) {
          // rows of the result that do not start on 16 bytes: a row at a time
          const int rows = min(32, args.m - y);
          for (int i = 0; i < rows; ++i) {
            const uint16_t u = *reinterpret_cast<const uint16_t*>(box + box_piece(i, lane >> 3) +
                                                                  (lane & 7) * 2);
            if (x + lane < args.n)
              reinterpret_cast<uint16_t*>(args.out)[((int64_t)z * args.m + y + i) * args.n + x +
                                                    lane] = u;
          }
          __syncwarp();
        } else {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmOut0, smem_u32(box), x, y, z);
            if (mirror) tma_store_3d(&tmOut0, smem_u32(box + L::kBox), y, x, z);
            if (KIND == kUpdate) tma_store_3d(&tmOut1, smem_u32(box + L::kBox), x, y, z);
            bulk_commit_group();
          }
        }
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(acc_empty(b), 0));
    }
    // given up: the chunks sent for have landed before the block ends
    for (; kLoads && used < loaded; ++used)
      wait_drain(slot_bar + 8u * (used % L::kSlots), (used / L::kSlots) & 1u);
    if (lane == 0) bulk_wait_group<0>();
  }

  tc_fence_before();
  pair_leave<L, S, 2, false>(L::kA + L::kB);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(ld_shared_u32(sbase + L::offMisc), kTmemCols);
  }
}

// ---- momentum and start ----------------------------------------------------------
// Two passes over the gradient and the momentum, bound by memory: the first
// writes V and sums U's squares (one partial sum a CTA, a matrix's are added in a
// fixed order), the second computes U again from V and G, scales it and writes
// its two halves.
constexpr int kEwThreads = 256, kEwUnroll = 4;

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
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kEwThreads / 32; ++w) s += red[w];
  return s;
}

// VEC: a matrix has a multiple of 4 elements.
template <bool WIDE, bool VEC>
__global__ void __launch_bounds__(kEwThreads) momentum_kernel(const MomentumArgs a) {
  __shared__ float red[kEwThreads / 32];
  griddep_wait();
  const int64_t base = (int64_t)blockIdx.y * a.size;
  const int64_t stride = (int64_t)gridDim.x * kEwThreads;
  float sum = 0.0f;
  if (VEC) {
    const int64_t n4 = a.size / 4;
    for (int64_t i = (int64_t)blockIdx.x * kEwThreads + threadIdx.x; i < n4;
         i += kEwUnroll * stride) {
      float4 g[kEwUnroll], v[kEwUnroll];
#pragma unroll
      for (int u = 0; u < kEwUnroll; ++u) {
        const int64_t at = base + 4 * (i + u * stride);
        if (i + u * stride < n4) {
          g[u] = grad4_at<WIDE>(a.grad, at);
          v[u] = *reinterpret_cast<const float4*>(a.momentum + at);
        }
      }
#pragma unroll
      for (int u = 0; u < kEwUnroll; ++u) {
        const int64_t at = base + 4 * (i + u * stride);
        if (i + u * stride >= n4) continue;
        v[u].x = fmaf(a.mu, v[u].x, g[u].x);
        v[u].y = fmaf(a.mu, v[u].y, g[u].y);
        v[u].z = fmaf(a.mu, v[u].z, g[u].z);
        v[u].w = fmaf(a.mu, v[u].w, g[u].w);
        *reinterpret_cast<float4*>(a.momentum + at) = v[u];
        if (a.nesterov) {
          v[u].x = fmaf(a.mu, v[u].x, g[u].x);
          v[u].y = fmaf(a.mu, v[u].y, g[u].y);
          v[u].z = fmaf(a.mu, v[u].z, g[u].z);
          v[u].w = fmaf(a.mu, v[u].w, g[u].w);
        }
        sum += (v[u].x * v[u].x + v[u].y * v[u].y) + (v[u].z * v[u].z + v[u].w * v[u].w);
      }
    }
  } else {
    for (int64_t i = (int64_t)blockIdx.x * kEwThreads + threadIdx.x; i < a.size; i += stride) {
      const float g = grad_at<WIDE>(a.grad, base + i);
      float v = fmaf(a.mu, a.momentum[base + i], g);
      a.momentum[base + i] = v;
      if (a.nesterov) v = fmaf(a.mu, v, g);
      sum = fmaf(v, v, sum);
    }
  }
  const float s = block_sum(sum, red);
  if (threadIdx.x == 0) a.partial[(int64_t)blockIdx.y * a.parts + blockIdx.x] = s;
}

// VEC: rows of a multiple of 8 elements, so hi and lo are laid out as the matrix.
template <bool WIDE, bool VEC>
__global__ void __launch_bounds__(kEwThreads) start_kernel(const MomentumArgs a) {
  __shared__ float red[kEwThreads / 32];
  griddep_wait();
  float sum = 0.0f;
  for (int p = threadIdx.x; p < a.parts; p += kEwThreads)
    sum += a.partial[(int64_t)blockIdx.y * a.parts + p];
  const float scale = kScale / fmaxf(sqrtf(block_sum(sum, red)), a.eps);
  const int64_t base = (int64_t)blockIdx.y * a.size, to = (int64_t)blockIdx.y * a.padded;
  const int64_t stride = (int64_t)gridDim.x * kEwThreads;
  if (VEC) {
    const int64_t n4 = a.size / 4;
    for (int64_t i = (int64_t)blockIdx.x * kEwThreads + threadIdx.x; i < n4;
         i += kEwUnroll * stride) {
      float4 g[kEwUnroll], v[kEwUnroll];
#pragma unroll
      for (int u = 0; u < kEwUnroll; ++u) {
        const int64_t at = base + 4 * (i + u * stride);
        if (i + u * stride < n4) {
          if (a.nesterov) g[u] = grad4_at<WIDE>(a.grad, at);
          v[u] = *reinterpret_cast<const float4*>(a.momentum + at);
        }
      }
#pragma unroll
      for (int u = 0; u < kEwUnroll; ++u) {
        const int64_t e = 4 * (i + u * stride);
        if (i + u * stride >= n4) continue;
        if (a.nesterov) {
          v[u].x = fmaf(a.mu, v[u].x, g[u].x);
          v[u].y = fmaf(a.mu, v[u].y, g[u].y);
          v[u].z = fmaf(a.mu, v[u].z, g[u].z);
          v[u].w = fmaf(a.mu, v[u].w, g[u].w);
        }
        v[u].x *= scale;
        v[u].y *= scale;
        v[u].z *= scale;
        v[u].w *= scale;
        const uint2 h = make_uint2(pack_f16x2(v[u].x, v[u].y), pack_f16x2(v[u].z, v[u].w));
        const float2 h0 = unpack_f16x2(h.x), h1 = unpack_f16x2(h.y);
        *reinterpret_cast<uint2*>(a.hi + to + e) = h;
        *reinterpret_cast<uint2*>(a.lo + to + e) =
            make_uint2(pack_f16x2(v[u].x - h0.x, v[u].y - h0.y),
                       pack_f16x2(v[u].z - h1.x, v[u].w - h1.y));
        if (a.zero) {
          if (WIDE)
            *reinterpret_cast<float4*>(static_cast<float*>(a.grad) + base + e) =
                make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.grad) + base + e) =
                make_uint2(0u, 0u);
        }
      }
    }
  } else {
    for (int64_t i = (int64_t)blockIdx.x * kEwThreads + threadIdx.x; i < a.size; i += stride) {
      float v = a.momentum[base + i];
      if (a.nesterov) v = fmaf(a.mu, v, grad_at<WIDE>(a.grad, base + i));
      v *= scale;
      const uint32_t row = (uint32_t)i / (uint32_t)a.cols, col = (uint32_t)i - row * a.cols;
      const int64_t at = to + (int64_t)row * a.ld + col;
      const __half h = __float2half_rn(v);
      a.hi[at] = h;
      a.lo[at] = __float2half_rn(v - __half2float(h));
      if (a.zero) {
        if (WIDE)
          static_cast<float*>(a.grad)[base + i] = 0.0f;
        else
          static_cast<uint16_t*>(a.grad)[base + i] = 0;
      }
    }
  }
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

template <int KIND, bool AMN, bool BMN>
nvfp4_status launch_ns(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& in0,
                       const CUtensorMap& in1, const CUtensorMap& out0, const CUtensorMap& out1,
                       NsArgs a, int64_t batch, int sms, cudaStream_t stream) {
  using L = NsLayout<KIND>;
  static GemmLaunchState ls;
  auto kern = ns_pair_kernel<KIND, AMN, BMN>;
  const int units = gemm_setup(ls, kern, L::kAlloc, L::kThreads, 0, 2, sms);
  if (units <= 0) return NVFP4_ERR_CUDA;
  a.tiles_m = (a.m + kTile - 1) / kTile;
  a.tiles_n = (a.n + kTile - 1) / kTile;
  a.tiles_per = KIND <= kPoly ? a.tiles_m * (a.tiles_m + 1) / 2 : a.tiles_m * a.tiles_n;
  a.tiles = (int)(a.tiles_per * batch);
  return cuda_status(launch_pdl(kern, 2 * std::min(units, a.tiles), L::kThreads, L::kAlloc, stream,
                                ma, mb, in0, in1, out0, out1, a));
}

// Where the parts of a workspace lie.
struct Layout {
  int64_t m, n;          // the matrix's smaller and larger side
  int64_t ldx, ldm, dstride;
  size_t x_bytes, g_bytes, d_bytes;
  size_t total;
  bool panel;
};
constexpr int kMaxParts = 1024;
constexpr int64_t kMaxSide = 1 << 20;

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
                            up1k((size_t)batch * kMaxParts * 4);
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
  const int64_t want = std::max<int64_t>(1, (e.size + kEwThreads * 16 - 1) / (kEwThreads * 16));
  const int64_t fit = std::max<int64_t>(1, (int64_t)dev.sm_count * 8 / p->batch);
  e.parts = (int)std::min<int64_t>({want, fit, kMaxParts});
  const dim3 grid((unsigned)e.parts, (unsigned)p->batch);
  const bool vec1 = e.size % 4 == 0, vec2 = p->cols % 8 == 0;
  auto k1 = wide ? (vec1 ? momentum_kernel<true, true> : momentum_kernel<true, false>)
                 : (vec1 ? momentum_kernel<false, true> : momentum_kernel<false, false>);
  auto k2 = wide ? (vec2 ? start_kernel<true, true> : start_kernel<true, false>)
                 : (vec2 ? start_kernel<false, true> : start_kernel<false, false>);
  if (launch_pdl(k1, grid, kEwThreads, 0, s, e) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (launch_pdl(k2, grid, kEwThreads, 0, s, e) != cudaSuccess) return NVFP4_ERR_CUDA;

  const bool tall = p->rows > p->cols;
  CUtensorMap xk[2], xmn[2], xbox[2], lobox, ek, fk, ebox, fbox, obox;
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    ok = ok && make_map(&xk[i], hi[i], p->batch, p->rows, p->cols, l.ldx, 64, 128);
    ok = ok && make_map(&xmn[i], hi[i], p->batch, p->rows, p->cols, l.ldx, 64, 64);
    ok = ok && make_map(&xbox[i], hi[i], p->batch, p->rows, p->cols, l.ldx, 32, 32);
  }
  ok = ok && make_map(&lobox, lo, p->batch, p->rows, p->cols, l.ldx, 32, 32);
  ok = ok && make_map(&ek, E, p->batch, l.m, l.m, l.ldm, 64, 128);
  ok = ok && make_map(&fk, F, p->batch, l.m, l.m, l.ldm, 64, 128);
  ok = ok && make_map(&ebox, E, p->batch, l.m, l.m, l.ldm, 32, 32);
  ok = ok && make_map(&fbox, F, p->batch, l.m, l.m, l.ldm, 32, 32);
  const bool out_boxes = p->cols % 8 == 0;
  if (out_boxes)
    ok = ok && make_map(&obox, update, p->batch, p->rows, p->cols, p->cols, 32, 32, true);
  else
    obox = lobox;  // not read
  if (!ok) return NVFP4_ERR_CUDA;

  for (int i = 0; i < p->steps; ++i) {
    const int x = i & 1;
    NsArgs a = {};
    a.a = p->coefs[3 * i];
    a.b = p->coefs[3 * i + 1];
    a.c = p->coefs[3 * i + 2];
    a.dstride = l.dstride;
    a.m = a.n = (int)l.m;
    a.k = (int)l.n;
    a.din = d;
    a.dout = d;
    st = tall ? launch_ns<kGram, true, true>(xmn[x], xmn[x], ebox, ebox, ebox, ebox, a, p->batch,
                                             dev.sm_count, s)
              : launch_ns<kGram, false, false>(xk[x], xk[x], ebox, ebox, ebox, ebox, a, p->batch,
                                               dev.sm_count, s);
    if (st != NVFP4_OK) return st;
    a.k = (int)l.m;
    a.din = d;
    a.dout = db;
    st = launch_ns<kPoly, false, false>(ek, ek, ebox, ebox, fbox, fbox, a, p->batch, dev.sm_count,
                                        s);
    if (st != NVFP4_OK) return st;
    a.m = (int)p->rows;
    a.n = (int)p->cols;
    a.din = db;
    a.by_col = tall;
    a.out = static_cast<__nv_bfloat16*>(update);
    a.out_boxes = out_boxes;
    const bool last = i == p->steps - 1;
    if (tall)
      st = last ? launch_ns<kFinal, false, false>(xk[x], fk, xbox[x], lobox, obox, obox, a,
                                                  p->batch, dev.sm_count, s)
                : launch_ns<kUpdate, false, false>(xk[x], fk, xbox[x], lobox, xbox[x ^ 1], lobox, a,
                                                   p->batch, dev.sm_count, s);
    else
      st = last ? launch_ns<kFinal, false, true>(fk, xmn[x], xbox[x], lobox, obox, obox, a,
                                                 p->batch, dev.sm_count, s)
                : launch_ns<kUpdate, false, true>(fk, xmn[x], xbox[x], lobox, xbox[x ^ 1], lobox, a,
                                                  p->batch, dev.sm_count, s);
    if (st != NVFP4_OK) return st;
  }
  return NVFP4_OK;
}
