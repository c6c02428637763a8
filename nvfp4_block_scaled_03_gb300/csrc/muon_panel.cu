// muon_panel.cu -- orthogonalised momentum (muon.cu) of matrices whose smaller side
// has at most 128 rows or columns: one launch that keeps the matrix on chip.
//
// X [m, n], m <= 128 the smaller side (a tall matrix is turned as it is loaded), is
// cut along n into blocks of 64 columns; a team of CTAs shares a matrix, a run of
// blocks each, held in shared memory as two f16 halves from the momentum's first
// read to the update's write.  A step is, for every CTA:
//   G = its blocks' part of X X^T  (tensor cores, FP32 in tensor memory)
//   the team's parts are added in a fixed order, through L2: all of them by every CTA
//     for itself where they are few (one team barrier), else a share by each CTA, whose
//     sums the others read (two)
//   E E, then F and the diagonals as in muon.cu, by every CTA for itself
//   X <- (a + d'_i) X + F X of its own blocks, in place
// A block, rows of 128 bytes with the 128-byte swizzle, is a K-major operand of the
// Gram product and an MN-major one of F X: one image serves both.  Rows behind m are
// zeros up to a multiple of 16; what an operand of 128 rows reads behind those (E, the
// blocks' first halves and their second halves follow one another) reaches rows of the
// result that nobody looks at.  For m up to 64 F's rows stand there again, so that every
// quarter of tensor memory, and with it every warp, has a share of the columns of F X.
//
// What bounds it, and measured: a step's chain of waits.  64 x 4096 on a cluster of 16
// takes 49 us (146 by the kernels of muon.cu, floor 0.5): 6 to load, then five steps of 8:
// 1.0 for X X^T, 3.4 until all CTAs have E (one meeting, 16 parts through L2), 0.5 for
// E E, 0.9 for F, 2.0 for F X.  Stacks go through it in rounds of what fits the SMs:
// 57 x [102, 1136] 146 us (199), 64 x [100, 9000] 965 to 1030 (1143; floor 118).
#include <algorithm>

#include "muon_common.cuh"

namespace nvfp4 {
namespace {

constexpr int kPanelThreads = 512, kColWarps = kPanelThreads / 128;
constexpr int kMaxM = 128;
constexpr uint32_t kMisc = 2048;
constexpr uint32_t kPanelSmem = 232448;
constexpr int kBarStride = 32;           // words between two teams' counters
constexpr int kPanelSms = 148;           // a plan has no more CTAs a matrix than this
// Up to so many values in a team's parts every CTA adds all of them.  A step has one
// barrier then, in front of the reads, and nothing keeps the next step's parts of a fast
// CTA from being stored while a slow one still reads: every other step's go to a second
// set of places, whose readers, a step before, are behind that barrier.  (Two matrices'
// steps have the barrier of the norm between them.)
// Measured (us; all of them by every CTA, a share each): clusters below the limit
// 16 x 2000 33, 37; 128 x 256 on 4 CTAs 53, 60; at it 64 x 4096 on 16 48.8, 49.5; beyond
// 128 x 512 on 8 60.4, 59.4; 80 x 4096 on 16 76, 58.  Teams of many CTAs would have the
// shares from less on: 16 x 60000 on 152 107, 85.
constexpr int64_t kOwnSum = 65536;

struct PanelArgs {
  void* grad;
  float* momentum;
  __nv_bfloat16* update;
  float4* part[2];     // [teams][ctas][mp / 4][m]: a CTA's part of X X^T, 4 columns each
  float4* sum;         // [teams][mp / 4][m]
  float* norm;         // [teams][ctas]
  unsigned int* bars;  // [teams], a counter each, zero at the start
  int m, mp, n;        // mp: m up to a multiple of 16
  int e_block;         // bytes of 64 columns of E or F
  int blocks;          // of 64 columns, of the matrix
  int room;            // blocks that a CTA has room for
  int ctas, teams, batch;
  int rows;            // between two copies of F's rows: 32, 64 or 128
  int cluster;         // a team is a cluster
  int shared_sum;      // each CTA adds a share of the parts; else all of them itself
  int tall, nesterov, zero, steps;
  float mu, eps;
  float coefs[3 * NVFP4_MUON_MAX_STEPS];
};

NVFP4_DEV void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Byte offset of 16-byte piece p of row i in a block.
NVFP4_DEV uint32_t piece_at(int i, int p) { return (uint32_t)(i * 128 + ((p ^ (i & 7)) << 4)); }

// What a CTA works with.
struct Panel {
  uint8_t *e, *hi, *lo;
  float *d, *dp;       // diagonals: d of A, a + d' of the step
  float* red;
  volatile int* abort_flag;
  unsigned int* bar;   // the team's counter
  unsigned int target;
  uint32_t mbar, phase, tmem;
  int team, rank, nb;  // nb: this CTA's blocks
  bool ok;
};

// All CTAs of a team meet; what each wrote to global memory before is visible to the
// others behind it.  False (for the whole CTA) when the wait ran out.  A cluster has
// its own barrier, which does not wait for CTAs that have left.
NVFP4_DEV bool team_barrier(Panel& s, const PanelArgs& a) {
  if (a.cluster) {
    __syncwarp();
    cluster_sync();
    return true;
  }
  __syncthreads();
  if (a.ctas > 1 && threadIdx.x == 0) {
    s.target += a.ctas;
    const bool lost = (injected() & kStall) != 0 && s.rank == 0;
    if (!lost) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(s.bar) : "memory");
    const uint64_t t0 = globaltimer_ns();
    const uint64_t limit = *reinterpret_cast<volatile unsigned long long*>(&g_gemm_wait_ns);
    while (true) {
      unsigned int v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(s.bar) : "memory");
      if (v >= s.target) break;
      if (globaltimer_ns() - t0 > limit) {
        *s.abort_flag = 1;
        atomicCAS(&g_gemm_error, 0u, 0x81u);
        break;
      }
    }
  }
  __syncthreads();
  return *s.abort_flag == 0;
}

// Every thread waits for the MMAs that thread 0 committed.
NVFP4_DEV bool wait_mma(Panel& s, uint32_t which) {
  const bool ok = wait_bounded(s.mbar + 8u * which, (s.phase >> which) & 1u, s.abort_flag, 0x82u);
  s.phase ^= 1u << which;
  tc_fence_after();
  return ok;
}

// The matrix's block run, values (i, 8 k ..): f(row i, first column k in the matrix,
// byte offset of the piece).
template <class F>
NVFP4_DEV void for_pieces(const Panel& s, const PanelArgs& a, int first, F f) {
  const int per = s.nb * 8;  // pieces of a row
  const int count = a.mp * per;
#pragma unroll 2
  for (int x = threadIdx.x; x < count; x += kPanelThreads) {
    int i, p;
    if (a.tall) {
      p = x / a.mp;
      i = x - p * a.mp;
    } else {
      i = x / per;
      p = x - i * per;
    }
    f(i, (first * 8 + p) * 8, (uint32_t)(p >> 3) * (uint32_t)(a.mp * 128) + piece_at(i, p & 7));
  }
}

NVFP4_DEV float block_total(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kPanelThreads / 32; ++w) t += red[w];
  return t;
}

// Momentum of one value and the direction U of the step.
NVFP4_DEV float momentum_of(const PanelArgs& a, float g, float& v) {
  v = fmaf(a.mu, v, g);
  return a.nesterov ? fmaf(a.mu, v, g) : v;
}

template <bool WIDE>
NVFP4_DEV void zero_grad(const PanelArgs& a, int64_t at) {
  if (WIDE)
    static_cast<float*>(a.grad)[at] = 0.0f;
  else
    static_cast<uint16_t*>(a.grad)[at] = 0;
}

// Whether rows are kept whole with a width that 16-byte pieces do not divide.  A lane
// then takes a column in global memory, not a piece of eight values one at a time, and the
// update goes out by way of shared memory: 60 x [101, 2137] 502 -> 414 us (60 x [104, 2144]
// 325), [37, 11654] 111 -> 90.
NVFP4_DEV bool ragged(const PanelArgs& a) { return !a.tall && a.n % 8 != 0; }

// f(row i, column in the matrix, byte offset of the value, turn) in the own blocks, for
// TURNS items of a warp from `item` on: 32 columns of a row each.
template <int TURNS, class F>
NVFP4_DEV void for_columns(const Panel& s, const PanelArgs& a, int first, int item, F f) {
  const int per = 2 * s.nb, lane = threadIdx.x & 31;
#pragma unroll
  for (int t = 0; t < TURNS; ++t) {
    const int x = item + t * (kPanelThreads / 32);
    const int i = x / per, col = (x - i * per) * 32 + lane;
    f(i, first * 64 + col,
      (uint32_t)(col >> 6) * (uint32_t)(a.mp * 128) + piece_at(i, (col & 63) >> 3) +
          2u * (col & 7), t);
  }
}

// Momentum and X's start.  Until the norm is known, a value's FP32 bits lie in the
// places of its two halves.
template <bool WIDE>
NVFP4_DEV bool load_matrix(Panel& s, const PanelArgs& a, int mat, int first) {
  const int64_t base = (int64_t)mat * a.m * a.n;
  float sum = 0.0f;
  if (ragged(a)) {
    constexpr int kTurns = 8;
    const int items = a.mp * s.nb * 2;
    for (int x = threadIdx.x >> 5; x < items; x += kTurns * (kPanelThreads / 32)) {
      float g[kTurns], v[kTurns];
      for_columns<kTurns>(s, a, first, x, [&](int i, int k, uint32_t, int t) {
        g[t] = v[t] = 0.0f;
        if (i < a.m && k < a.n) {
          g[t] = grad_at<WIDE>(a.grad, base + (int64_t)i * a.n + k);
          v[t] = a.momentum[base + (int64_t)i * a.n + k];
        }
      });
      for_columns<kTurns>(s, a, first, x, [&](int i, int k, uint32_t at, int t) {
        const float u = momentum_of(a, g[t], v[t]);
        if (i < a.m && k < a.n) {
          a.momentum[base + (int64_t)i * a.n + k] = v[t];
          if (a.zero) zero_grad<WIDE>(a, base + (int64_t)i * a.n + k);
        }
        sum = fmaf(u, u, sum);
        if (i < a.mp) {
          *reinterpret_cast<uint16_t*>(s.hi + at) = (uint16_t)(__float_as_uint(u) >> 16);
          *reinterpret_cast<uint16_t*>(s.lo + at) = (uint16_t)__float_as_uint(u);
        }
      });
    }
  } else {
    for_pieces(s, a, first, [&](int i, int k, uint32_t at) {
      float g[8] = {}, v[8] = {};
      const int live = i < a.m ? min(8, a.n - k) : 0;
      const int64_t step = a.tall ? a.m : 1;
      const int64_t from = base + (a.tall ? (int64_t)k * a.m + i : (int64_t)i * a.n + k);
      if (a.tall) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < live) {
            g[j] = grad_at<WIDE>(a.grad, from + j * step);
            v[j] = a.momentum[from + j * step];
          }
      } else if (live > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 x = grad4_at<WIDE>(a.grad, from + 4 * h);
          const float4 y = *reinterpret_cast<const float4*>(a.momentum + from + 4 * h);
          g[4 * h] = x.x, g[4 * h + 1] = x.y, g[4 * h + 2] = x.z, g[4 * h + 3] = x.w;
          v[4 * h] = y.x, v[4 * h + 1] = y.y, v[4 * h + 2] = y.z, v[4 * h + 3] = y.w;
        }
      }
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = momentum_of(a, g[j], v[j]);
        sum = fmaf(u, u, sum);
        w[j] = __float_as_uint(u);
      }
      if (a.tall) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < live) a.momentum[from + j * step] = v[j];
      } else if (live > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4*>(a.momentum + from + 4 * h) =
              make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
      }
      if (a.zero)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < live) zero_grad<WIDE>(a, from + j * step);
      *reinterpret_cast<uint4*>(s.hi + at) =
          make_uint4(__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632),
                     __byte_perm(w[4], w[5], 0x7632), __byte_perm(w[6], w[7], 0x7632));
      *reinterpret_cast<uint4*>(s.lo + at) =
          make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410),
                     __byte_perm(w[4], w[5], 0x5410), __byte_perm(w[6], w[7], 0x5410));
    });
  }
  float total = block_total(sum, s.red);
  if (a.ctas > 1) {
    float* norm = a.norm + s.team * a.ctas;
    if (threadIdx.x == 0) norm[s.rank] = total;
    if (!team_barrier(s, a)) return false;
    float t = 0.0f;
    for (int c = threadIdx.x; c < a.ctas; c += kPanelThreads) t += __ldcg(norm + c);
    total = block_total(t, s.red);
  }
  const float scale = start_scale(total, a.eps);
  for_pieces(s, a, first, [&](int, int, uint32_t at) {
    const uint4 h = *reinterpret_cast<const uint4*>(s.hi + at);
    const uint4 l = *reinterpret_cast<const uint4*>(s.lo + at);
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = __uint_as_float(__byte_perm(lw[e], hw[e], 0x5410)) * scale;
      const float y = __uint_as_float(__byte_perm(lw[e], hw[e], 0x7632)) * scale;
      ph[e] = pack_f16x2(x, y);
      const float2 f = unpack_f16x2(ph[e]);
      pl[e] = pack_f16x2(x - f.x, y - f.y);
    }
    *reinterpret_cast<uint4*>(s.hi + at) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
    *reinterpret_cast<uint4*>(s.lo + at) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
  });
  return true;
}

// The sum of a team's parts at one place, in the CTAs' order.
NVFP4_DEV float4 add_parts(const float4* at, int ctas, int stride) {
  float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 16
  for (int c = 0; c < ctas; ++c) {
    const float4 u = __ldcg(at + (int64_t)c * stride);
    t.x += u.x;
    t.y += u.y;
    t.z += u.z;
    t.w += u.w;
  }
  return t;
}

// 8 columns from j0 on of row i of E, in f16 with 2^12; the diagonal goes to d.
NVFP4_DEV void put_e(const Panel& s, const PanelArgs& a, int i, int j0, const float4 u,
                     const float4 v) {
  float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] *= kUnscale;
    if (j0 + e == i) {
      s.d[i] = x[e] * kUnscale;
      x[e] = 0.0f;
    }
  }
  *reinterpret_cast<uint4*>(s.e + (j0 >> 6) * a.e_block + piece_at(i, (j0 & 63) >> 3)) =
      make_uint4(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]), pack_f16x2(x[4], x[5]),
                 pack_f16x2(x[6], x[7]));
}

// E of the sum of `count` parts: 16 loads of a thread in flight, of one piece of 8
// columns where there are no more pieces than threads, else of four.
NVFP4_DEV void make_e(const Panel& s, const PanelArgs& a, const float4* parts, int count) {
  const int pieces = a.m * a.mp / 8, quads = 2 * pieces;
  if (pieces <= kPanelThreads) {
    const int x = threadIdx.x, p = x / a.m;
    if (x < pieces) {
      const float4* at = parts + p * a.m + x;  // 2 p m + i
      const float4 u = add_parts(at, count, quads), v = add_parts(at + a.m, count, quads);
      put_e(s, a, x - p * a.m, 8 * p, u, v);
    }
    return;
  }
  for (int x0 = threadIdx.x; x0 < pieces; x0 += 4 * kPanelThreads) {
    float4 t[4][2];
    int at[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = min(x0 + k * kPanelThreads, pieces - 1), p = x / a.m;
      at[k] = p * a.m + x;  // 2 p m + i
      t[k][0] = t[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll 2
    for (int c = 0; c < count; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 u = __ldcg(parts + (int64_t)c * quads + at[k] + h * a.m);
          t[k][h].x += u.x;
          t[k][h].y += u.y;
          t[k][h].z += u.z;
          t[k][h].w += u.w;
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = x0 + k * kPanelThreads, p = x / a.m;
      if (x < pieces) put_e(s, a, x - p * a.m, 8 * p, t[k][0], t[k][1]);
    }
  }
}

template <bool WIDE>
__global__ void __launch_bounds__(kPanelThreads, 1) panel_kernel(const PanelArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t block_bytes = (uint32_t)a.mp * 128;
  Panel s;
  s.e = smem;
  const uint32_t e_bytes = a.e_block * ((a.mp + 63) / 64);
  s.hi = smem + e_bytes;
  s.lo = s.hi + a.room * block_bytes;
  uint8_t* misc = smem + kPanelSmem - 1024 - kMisc;
  s.d = reinterpret_cast<float*>(misc);
  s.dp = s.d + kMaxM;
  s.red = s.dp + kMaxM;
  s.mbar = smem_u32(misc + 1536);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 1568);
  s.abort_flag = reinterpret_cast<volatile int*>(misc + 1572);
  s.team = blockIdx.x / a.ctas;
  s.rank = blockIdx.x - s.team * a.ctas;
  s.bar = a.bars + s.team * kBarStride;
  s.target = 0;
  s.phase = 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = warp & 3, h = warp >> 2;
  const int first = (int)((int64_t)a.blocks * s.rank / a.ctas);
  s.nb = (int)((int64_t)a.blocks * (s.rank + 1) / a.ctas) - first;
  if (tid == 0) {
    mbar_init(s.mbar, 1);
    mbar_init(s.mbar + 8, 1);
    *s.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  for (uint32_t i = tid * 16; i < e_bytes; i += kPanelThreads * 16)
    *reinterpret_cast<uint4*>(s.e + i) = make_uint4(0u, 0u, 0u, 0u);
  if (tid < kMaxM) s.d[tid] = s.dp[tid] = 0.0f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  s.tmem = *tmem_slot;
  const uint32_t tmem = s.tmem, hi = smem_u32(s.hi), e = smem_u32(s.e);
  const uint32_t rows = tmem + ((uint32_t)(q * 32) << 16);  // this warp's lanes
  const int row = q * 32 + lane;
  const uint32_t idesc_mm = idesc_f16(128, a.mp, false, false);
  const int chunks = (s.nb + 3) / 4;
  bool ok = true;

  for (int mat = s.team; ok && mat < a.batch; mat += a.teams) {
    ok = WIDE ? load_matrix<true>(s, a, mat, first) : load_matrix<false>(s, a, mat, first);
    for (int step = 0; ok && step < a.steps; ++step) {
      const float ca = a.coefs[3 * step], cb = a.coefs[3 * step + 1], cc = a.coefs[3 * step + 2];
      // ---- X X^T of the own blocks
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        for (int b = 0; b < s.nb; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t d = smem_desc_sw128(hi + b * block_bytes + 32 * j);
            tc_mma_f16(tmem, d, d, idesc_mm, b | j ? 1u : 0u);
          }
        tc_commit(s.mbar);
      }
      ok = __syncthreads_and(wait_mma(s, 0));
      if (!ok) break;
      // this warp's columns of the part, 4 of 32 rows at a time
      const int quads = a.m * a.mp / 4;
      float4* parts = a.part[step & 1] + (int64_t)s.team * a.ctas * quads;
      if (q * 32 < a.m && 32 * h < a.mp) {
        uint32_t r[32];
        tmem_ld32(rows + 32 * h, r);
        tmem_ld_wait();
        if (row < a.m)
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (32 * h + 4 * x < a.mp) {
              const float4 v = make_float4(__uint_as_float(r[4 * x]), __uint_as_float(r[4 * x + 1]),
                                           __uint_as_float(r[4 * x + 2]),
                                           __uint_as_float(r[4 * x + 3]));
              __stcg(parts + (int64_t)s.rank * quads + (8 * h + x) * a.m + row, v);
            }
      }
      ok = team_barrier(s, a);
      if (!ok) break;
      const float4* sum = a.sum + (int64_t)s.team * quads;
      if (a.shared_sum) {
        const int q0 = (int)((int64_t)quads * s.rank / a.ctas);
        const int q1 = (int)((int64_t)quads * (s.rank + 1) / a.ctas);
        for (int x = q0 + tid; x < q1; x += kPanelThreads)
          __stcg(const_cast<float4*>(sum) + x, add_parts(parts + x, a.ctas, quads));
        ok = team_barrier(s, a);
        if (!ok) break;
      }
      make_e(s, a, a.shared_sum ? sum : parts, a.shared_sum ? 1 : a.ctas);
      // ---- E E, then F in E's place
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        for (int k = 0; k < a.mp; k += 16) {
          const uint64_t d = smem_desc_sw128(e + (k >> 6) * a.e_block + (k & 63) * 2);
          tc_mma_f16(tmem, d, d, idesc_mm, k ? 1u : 0u);
        }
        tc_commit(s.mbar);
      }
      ok = __syncthreads_and(wait_mma(s, 0));
      if (!ok) break;
      if (q * 32 < a.m)
        for (int c0 = 32 * h; c0 < a.mp; c0 += 32 * kColWarps) {
          uint32_t r[32];
          tmem_ld32(rows + c0, r);
          tmem_ld_wait();
          if (row < a.m) {
            const float di = s.d[row];
            uint8_t* block = s.e + (c0 >> 6) * a.e_block;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              uint4* at = reinterpret_cast<uint4*>(block + piece_at(row, ((c0 & 63) >> 3) + p));
              const uint4 u = *at;
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
              uint32_t f[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int j = c0 + 8 * p + 2 * x;
                const float2 ev = unpack_f16x2(w[x]);
                const float r0 = __uint_as_float(r[8 * p + 2 * x]);
                const float r1 = __uint_as_float(r[8 * p + 2 * x + 1]);
                float f0 = 0.0f, f1 = 0.0f;
                if (j < a.m) f0 = cb * ev.x + cc * (r0 * kUnscale + (di + s.d[j]) * ev.x);
                if (j + 1 < a.m) f1 = cb * ev.y + cc * (r1 * kUnscale + (di + s.d[j + 1]) * ev.y);
                const float sq = (j == row ? r0 : r1) * (kUnscale * kUnscale);
                if (j == row || j + 1 == row) s.dp[row] = ca + (cb * di + cc * (di * di + sq));
                if (j == row) f0 = 0.0f;
                if (j + 1 == row) f1 = 0.0f;
                f[x] = pack_f16x2(f0, f1);
              }
              *at = make_uint4(f[0], f[1], f[2], f[3]);
              for (int c = a.rows; c < 128; c += a.rows)
                *reinterpret_cast<uint4*>(block + piece_at(row + c, ((c0 & 63) >> 3) + p)) = *at;
            }
          }
        }
      // ---- X <- (a + d') X + F X, 256 columns at a time
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      auto issue = [&](int c) {
        tc_fence_after();
        const int nb = min(4, s.nb - 4 * c);
        const uint32_t idesc = idesc_f16(128, 64 * nb, false, true);
        for (int k = 0; k < a.mp; k += 16)
          tc_mma_f16(tmem + (c & 1) * 256,
                     smem_desc_sw128(e + (k >> 6) * a.e_block + (k & 63) * 2),
                     smem_desc_mn(hi + 4 * c * block_bytes + k * 128, block_bytes), idesc,
                     k ? 1u : 0u);
        tc_commit(s.mbar + 8u * (c & 1));
      };
      if (tid == 0) {
        issue(0);
        if (chunks > 1) issue(1);
      }
      const bool last = step == a.steps - 1, odd = ragged(a);
      for (int c = 0; c < chunks; ++c) {
        ok = __syncthreads_and(wait_mma(s, c & 1));
        if (!ok) break;
        const int cols = 64 * min(4, s.nb - 4 * c);
        // the quarters of tensor memory that hold a copy of the rows share the columns
        const int copies = 128 / a.rows, mine = q * 32 % a.rows, row = mine + lane;
        if (mine < a.m) {
          const float dp = s.dp[row];
          for (int col = 32 * (h * copies + q * 32 / a.rows); col < cols;
               col += 32 * kColWarps * copies) {
            uint32_t r[32];
            tmem_ld32(rows + (c & 1) * 256 + col, r);
            tmem_ld_wait();
            const uint32_t block = (uint32_t)(4 * c + (col >> 6)) * block_bytes;
            const int k0 = (first + 4 * c) * 64 + col;  // in the matrix
            const int64_t out = (int64_t)mat * a.m * a.n +
                                (a.tall ? (int64_t)k0 * a.m + row : (int64_t)row * a.n + k0);
            if (row < a.m)
#pragma unroll
              for (int p = 0; p < 4; ++p) {
                const uint32_t at = block + piece_at(row, ((col & 63) >> 3) + p);
                const uint4 uh = *reinterpret_cast<const uint4*>(s.hi + at);
                const uint4 ul = *reinterpret_cast<const uint4*>(s.lo + at);
                const uint32_t wh[4] = {uh.x, uh.y, uh.z, uh.w}, wl[4] = {ul.x, ul.y, ul.z, ul.w};
                uint32_t oh[4], ol[4];
                float v[8];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float2 fh = unpack_f16x2(wh[x]), fl = unpack_f16x2(wl[x]);
                  v[2 * x] = dp * (fh.x + fl.x) + __uint_as_float(r[8 * p + 2 * x]) * kUnscale;
                  v[2 * x + 1] =
                      dp * (fh.y + fl.y) + __uint_as_float(r[8 * p + 2 * x + 1]) * kUnscale;
                  oh[x] = pack_f16x2(v[2 * x], v[2 * x + 1]);
                  const float2 g = unpack_f16x2(oh[x]);
                  ol[x] = pack_f16x2(v[2 * x] - g.x, v[2 * x + 1] - g.y);
                }
                if (!last) {
                  *reinterpret_cast<uint4*>(s.hi + at) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
                  *reinterpret_cast<uint4*>(s.lo + at) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
                } else if (odd) {
                  // to shared memory in X's place, from where whole lines go out below
                  *reinterpret_cast<uint4*>(s.hi + at) =
                      make_uint4(pack_bf16x2(v[0] * kUnscale, v[1] * kUnscale),
                                 pack_bf16x2(v[2] * kUnscale, v[3] * kUnscale),
                                 pack_bf16x2(v[4] * kUnscale, v[5] * kUnscale),
                                 pack_bf16x2(v[6] * kUnscale, v[7] * kUnscale));
                } else if (!a.tall) {
                  if (k0 + 8 * p < a.n)
                    *reinterpret_cast<uint4*>(a.update + out + 8 * p) = make_uint4(
                        pack_bf16x2(v[0] * kUnscale, v[1] * kUnscale),
                        pack_bf16x2(v[2] * kUnscale, v[3] * kUnscale),
                        pack_bf16x2(v[4] * kUnscale, v[5] * kUnscale),
                        pack_bf16x2(v[6] * kUnscale, v[7] * kUnscale));
                } else {
#pragma unroll
                  for (int x = 0; x < 8; ++x)
                    if (k0 + 8 * p + x < a.n)
                      a.update[out + (int64_t)(8 * p + x) * a.m] =
                          __float2bfloat16_rn(v[x] * kUnscale);
                }
              }
          }
        }
        tc_fence_before();
        __syncthreads();
        if (tid == 0 && c + 2 < chunks) issue(c + 2);
      }
      if (ok && last && odd) {
        const int items = a.m * s.nb * 2;
        for (int x = warp; x < items; x += kPanelThreads / 32)
          for_columns<1>(s, a, first, x, [&](int i, int k, uint32_t at, int) {
            if (k < a.n)
              a.update[(int64_t)mat * a.m * a.n + (int64_t)i * a.n + k] =
                  *reinterpret_cast<const __nv_bfloat16*>(s.hi + at);
          });
        __syncthreads();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // given up at a wait: what thread 0 issued has finished before its memory is freed
  if (!ok && tid == 0) {
    tc_commit(s.mbar);
    wait_drain(s.mbar, (s.phase & 1u));
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// How a call is spread over a device's SMs.
struct PanelPlan {
  int m, mp, n, e_block, blocks, room, least, ctas, teams;
  bool cluster, shared_sum;
};
// wide: how many clusters of 16 a device has room for (0: not known).
PanelPlan panel_plan(int64_t batch, int64_t rows, int64_t cols, int sms, int wide) {
  PanelPlan l;
  l.m = (int)std::min(rows, cols);
  l.n = (int)std::max(rows, cols);
  l.mp = (l.m + 15) / 16 * 16;
  l.blocks = (l.n + 63) / 64;
  l.e_block = 128 * (l.m > 64 ? l.mp : 128);  // with copies 128 rows
  l.room = (int)((kPanelSmem - 1024 - kMisc - l.e_block * ((l.mp + 63) / 64)) / (l.mp * 256));
  l.least = (l.blocks + l.room - 1) / l.room;
  // Teams that fit a cluster are one, for its barrier (a team of 64 CTAs by counters
  // took 72 us for 64 x 4096, a cluster of 8 63, of 16 52); a matrix is spread over as
  // many CTAs of one as the stack leaves.  Clusters of 16 only where all are resident
  // at once: 8 x [128, 4096] take 142 us in them, 104 with teams of 19.
  const int spread = (int)std::min<int64_t>(l.blocks, std::max<int64_t>(1, sms / batch));
  const bool sixteen = batch <= wide;
  l.cluster = l.least <= (sixteen ? 16 : 8);
  if (l.cluster) {
    const int most = std::min(spread, sixteen ? 16 : 8);
    for (l.ctas = 1; l.ctas < l.least || 2 * l.ctas <= most;) l.ctas *= 2;
  } else {
    l.ctas = std::max(l.least, spread);
  }
  l.teams = (int)std::min<int64_t>(batch, std::max(1, sms / l.ctas));
  l.shared_sum = (int64_t)l.ctas * l.m * l.mp > kOwnSum;
  return l;
}

size_t panel_bytes(const PanelPlan& l, size_t* sum, size_t* norm, size_t* bars) {
  const size_t square = (size_t)l.m * l.mp * 4;
  *sum = up1k((size_t)l.teams * l.ctas * square);
  *norm = *sum + up1k((size_t)l.teams * (l.shared_sum ? 1 : l.ctas) * square);
  *bars = *norm + up1k((size_t)l.teams * l.ctas * 4);
  return *bars + up1k((size_t)l.teams * kBarStride * 4);
}

}  // namespace

bool muon_panel_fits(int64_t rows, int64_t cols) {
  if (std::min(rows, cols) > kMaxM) return false;
  return panel_plan(1, rows, cols, kPanelSms, 0).least <= kPanelSms;
}

// Enough for any plan: at most kMaxSms CTAs, so as many parts, sums (or second parts) and
// counters.
size_t muon_panel_workspace(int64_t rows, int64_t cols) {
  const int64_t m = std::min(rows, cols);
  const size_t square = (size_t)m * ((m + 15) / 16 * 16) * 4;
  return 2 * up1k(kMaxSms * square) + up1k(kMaxSms * 4) + up1k((size_t)kMaxSms * kBarStride * 4);
}

nvfp4_status muon_panel(const MuonCall& c) {
  auto kern = c.wide ? panel_kernel<true> : panel_kernel<false>;
  static GemmLaunchState ls[2][5];
  auto resident = [&](int cluster) {  // clusters that a device holds at once
    int log = 0;
    while ((1 << log) < cluster) ++log;
    return gemm_setup(ls[c.wide][log], kern, kPanelSmem, kPanelThreads, 0, cluster, c.sms);
  };
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  const int sms = std::min(c.sms, kMaxSms);
  PanelPlan l = panel_plan(c.p->batch, c.p->rows, c.p->cols, sms, resident(16));
  if (l.ctas > sms) return NVFP4_ERR_CUDA;
  const int fit = resident(l.cluster ? l.ctas : 1);
  if (fit <= 0) return NVFP4_ERR_CUDA;
  if (l.cluster && l.ctas > 1) l.teams = std::min(l.teams, fit);
  size_t sum, norm, bars;
  panel_bytes(l, &sum, &norm, &bars);
  uint8_t* w = static_cast<uint8_t*>(c.workspace);
  PanelArgs a = {};
  a.grad = c.grad;
  a.momentum = c.momentum;
  a.update = c.update;
  a.part[0] = reinterpret_cast<float4*>(w);
  a.part[1] = reinterpret_cast<float4*>(l.shared_sum ? w : w + sum);
  a.sum = reinterpret_cast<float4*>(w + sum);
  a.norm = reinterpret_cast<float*>(w + norm);
  a.bars = reinterpret_cast<unsigned int*>(w + bars);
  a.m = l.m;
  a.rows = l.m <= 32 ? 32 : l.m <= 64 ? 64 : 128;
  a.mp = l.mp;
  a.e_block = l.e_block;
  a.n = l.n;
  a.blocks = l.blocks;
  a.room = l.room;
  a.ctas = l.ctas;
  a.teams = l.teams;
  a.cluster = l.cluster;
  a.shared_sum = l.shared_sum;
  a.batch = (int)c.p->batch;
  a.tall = c.p->rows > c.p->cols;
  a.nesterov = c.p->nesterov;
  a.zero = c.zero;
  a.steps = c.p->steps;
  a.mu = c.p->mu;
  a.eps = c.p->eps;
  std::copy(c.p->coefs, c.p->coefs + 3 * c.p->steps, a.coefs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(l.teams * l.ctas));
  cfg.blockDim = dim3(kPanelThreads);
  cfg.dynamicSmemBytes = kPanelSmem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr;
  if (l.cluster) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = l.ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  } else {
    if (cudaMemsetAsync(a.bars, 0, (size_t)l.teams * kBarStride * 4, c.stream) != cudaSuccess)
      return NVFP4_ERR_CUDA;
    attr.id = cudaLaunchAttributeCooperative;  // the CTAs of a team wait on one another
    attr.val.cooperative = 1;
  }
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, a));
}

nvfp4_status muon_panel_set_injection(unsigned int stall, unsigned long long wait_ns) {
  if (cudaMemcpyToSymbol(g_gemm_stall, &stall, sizeof(stall)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_gemm_wait_ns, &wait_ns, sizeof(wait_ns)) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return NVFP4_OK;
}

nvfp4_status muon_panel_read_error(unsigned int* code) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemm_error, sizeof(v)) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (v && cudaMemcpyToSymbol(g_gemm_error, &zero, sizeof(zero)) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  *code = v;
  return NVFP4_OK;
}

}  // namespace nvfp4
