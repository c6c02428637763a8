// norm.cu -- the RMS norms on either side of a residual block, fused with the
// block's gate and the residual scales:
//   y = a x + b g (.) n,   n = z r_z w_post,   h = y r_y w_pre,
//   r_v = (mean v^2 + eps)^(-1/2) over a row,
// x the residual stream, z the block's output, g a gate per channel or per
// row, h the next block's input.  One pass reads x and z and writes y and h,
// so closing a block and opening the next costs no second read of y.
//
// Backward from dy and dh, with z^ = z r_z, y^ = y r_y (recomputed from x and
// z in FP32: nothing but the inputs is kept from the forward):
//   u  = dh w_pre,  dY = dy + r_y (u - y^ mean(u y^)),  dx = a dY,  q = b dY,
//   v  = q g w_post,  dz = r_z (v - z^ mean(v z^)),
//   dw_pre = sum_rows dh y^,  dw_post = sum_rows q g z^,
//   dg = sum_rows q z^ w_post (channel gate) or sum_channels (row gate).
// With a gate per channel dw_post = g S and dg = w_post S for one column sum
// S = sum_rows q z^, so two column sums are carried in every form.
//
// All arithmetic is FP32 (two values an instruction: f32x2); x, y, dx, dy are
// bf16 or FP32, z, h, dz, dh bf16, each rounded once.  The kernels move 2 (x, y)
// + 2 (z, h) or 3 + 3 streams and are bound by memory, with the arithmetic
// (about 12 and 25 instructions an element pair) not far behind.
//
// A persistent CTA takes `rpc` rows at a time, whole warps per row (forward one
// from 4104 to 16384 columns, backward one from 2056 on), its weights in
// registers.  Rows arrive by bulk copies in a ring of shared-memory stages, so
// loads run ahead while a row is reduced; a row is read from its stage once per
// pass instead of being held in registers, which leaves those to the weights
// and the column sums.  Long rows (the backward from 8200 columns on, the
// forward from 16392) are read from global memory in each pass.  From 16392 columns on a thread takes 128 of them,
// more than its 64 registers hold: 1.1 KB of spills forward, 2.7 KB backward.
//
// Measured (us, and the time their bytes take at the copy rate): 16384 x 4096
// bf16 forward 84 (80), backward 149 (120); FP32 stream, 8191 x 4096 forward
// 69 (60), backward 102 (90); 4096 x 16384 bf16 118 (80), 230 (120); 2048 x 32768
// 241 (80), 780 (120); 16 x 4096 forward 3.9, launch included.  The bf16
// backward is bound by its arithmetic (0.58 of the issue slots, 16 warps an SM:
// its column sums and weights fill the registers).
//
// The column sums go to per-CTA partials that a second kernel adds in a fixed
// order: no atomics, so results repeat bit for bit.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace nvfp4 {

static __device__ unsigned int g_norm_error;
// Failure injection (nvfp4_debug_inject): bit 0, no rows are loaded; bit 1, each
// CTA's first barrier waits for 16 bytes that do not come.
static __device__ unsigned int g_norm_stall;
static __device__ unsigned long long g_norm_wait_ns = 2000000000ull;

namespace {

constexpr int kVec = 8;           // columns a thread takes at a time
constexpr int kPairs = kVec / 2;  // as pairs
constexpr int kMaxThreads = 512;
constexpr int kMaxVpt = 16;       // 512 threads x 16 x 8 = 65536 columns
constexpr int kRegVpt = 2;        // up to here the weights stay in registers
constexpr int kMaxStages = 4;
constexpr uint64_t kDrainNs = 2000000000ull;

struct NormArgs {
  const void* x;
  const uint16_t* z;
  const float* w_post;
  const float* gate;
  const float* w_pre;
  void* y;
  uint16_t* h;
  int64_t rows;
  int cols;
  int gate_mode;
  float eps, a, b;
  int wpr, rpc;         // warps of a row, rows of a CTA
  int stages;           // of the ring
  uint32_t stage_bytes;
  // backward
  const void* dy;
  const uint16_t* dh;
  void* dx;
  uint16_t* dz;
  float* drow;      // row gate: its gradient [rows]
  float* partials;  // [CTAs x rpc][2][cols]: S or dw_post, then dw_pre
};

struct F8 {
  float2 v[kPairs];
};

NVFP4_DEV F8 zero8() {
  F8 r;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) r.v[i] = make_float2(0.0f, 0.0f);
  return r;
}
NVFP4_DEV float2 both(float s) { return make_float2(s, s); }
NVFP4_DEV F8 load_bf16(const void* p) {
  const uint4 u = *static_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  F8 r;
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    r.v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return r;
}
NVFP4_DEV F8 load_f32(const void* p) {
  const float4 lo = static_cast<const float4*>(p)[0], hi = static_cast<const float4*>(p)[1];
  F8 r;
  r.v[0] = make_float2(lo.x, lo.y);
  r.v[1] = make_float2(lo.z, lo.w);
  r.v[2] = make_float2(hi.x, hi.y);
  r.v[3] = make_float2(hi.z, hi.w);
  return r;
}
NVFP4_DEV void store_bf16(uint16_t* p, const F8& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(f.v[i].x, f.v[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
NVFP4_DEV void store_f32(float* p, const F8& f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(f.v[2].x, f.v[2].y, f.v[3].x, f.v[3].y);
}
template <bool WIDE>
NVFP4_DEV F8 load_stream(const void* p, int c) {
  if constexpr (WIDE) return load_f32(static_cast<const float*>(p) + c);
  return load_bf16(static_cast<const uint16_t*>(p) + c);
}
template <bool WIDE>
NVFP4_DEV void store_stream(void* p, int64_t at, const F8& f) {
  if constexpr (WIDE)
    store_f32(static_cast<float*>(p) + at, f);
  else
    store_bf16(static_cast<uint16_t*>(p) + at, f);
}

// Sums over the threads of a row, one or five at a time: within the warp by
// shuffles, across the row's warps (16 at most) through shared memory with one
// barrier of the CTA.  Every thread gets them and the order is fixed.  The
// calls alternate between two buffers: a buffer is written again only after
// the next call's barrier, which every thread reaches after its reads.
struct Reducer {
  float buf[2][16 * 8];
};
NVFP4_DEV void row_sum(float& v, Reducer& r, int& turn, int wpr, int w0) {
  float* red = r.buf[turn];
  turn ^= 1;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (wpr == 1) return;
  v = (lane & 15) < wpr ? red[w0 + (lane & 15)] : 0.0f;
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
}
// One step of a reduction of two values at once: the lanes with bit `o` clear
// go on with a, the others with b.
NVFP4_DEV float fold2(float a, float b, int o) {
  const bool hi = threadIdx.x & o;
  return (hi ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, hi ? a : b, o);
}
// Five values in 8 + 7 shuffles: each step folds values pairwise into the two
// halves of a lane group, so lane bits 4, 3, 2 end up naming the value.
NVFP4_DEV void row_sum(float (&v)[5], Reducer& r, int& turn, int wpr, int w0) {
  float* red = r.buf[turn];
  turn ^= 1;
  const int lane = threadIdx.x & 31;
  const float v01 = fold2(v[0], v[1], 16), v23 = fold2(v[2], v[3], 16);
  const float v4 = v[4] + __shfl_xor_sync(0xFFFFFFFFu, v[4], 16);
  float t = fold2(fold2(v01, v23, 8), v4 + __shfl_xor_sync(0xFFFFFFFFu, v4, 8), 4);
  t += __shfl_xor_sync(0xFFFFFFFFu, t, 2);
  t += __shfl_xor_sync(0xFFFFFFFFu, t, 1);
  // bit 2 clear: value 2 (bit 3) + (bit 4); set: value 4 (from the lowest such lane)
  if ((lane & 7) == 0) red[(threadIdx.x >> 5) * 8 + ((lane >> 3) & 1) * 2 + (lane >> 4)] = t;
  if (lane == 4) red[(threadIdx.x >> 5) * 8 + 4] = t;
  __syncthreads();
  // lane: value lane % 8 of the warps lane / 8, lane / 8 + 4, ..
  t = 0.0f;
  for (int w = lane >> 3; w < wpr; w += 4) t += red[(w0 + w) * 8 + (lane & 7)];
  t += __shfl_xor_sync(0xFFFFFFFFu, t, 8);
  t += __shfl_xor_sync(0xFFFFFFFFu, t, 16);
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, t, i);
}

// 1 / sqrt(mean square + eps); rsqrtf is within 2 ulp.
NVFP4_DEV float rstd(float sum_sq, float inv_cols, float eps) {
  return rsqrtf(fmaf(sum_sq, inv_cols, eps));
}

// What a kernel is compiled for: both norms, only the one after the block, only
// the one before it; kAsGiven looks at the pointers (long rows).
enum { kBoth = 0, kPostOnly = 1, kPreOnly = 2, kAsGiven = 3 };
template <int PARTS>
NVFP4_DEV bool has_post(const void* p) {
  return PARTS == kAsGiven ? p != nullptr : PARTS != kPreOnly;
}
template <int PARTS>
NVFP4_DEV bool has_pre(const void* p) {
  return PARTS == kAsGiven ? p != nullptr : PARTS != kPostOnly;
}

// The block's weights at column c, with a channel gate in them.
NVFP4_DEV F8 post_weight(const NormArgs& p, int c) {
  F8 w = load_f32(p.w_post + c);
  if (p.gate_mode == NVFP4_GATE_CHANNEL) {
    const F8 g = load_f32(p.gate + c);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) w.v[i] = __fmul2_rn(w.v[i], g.v[i]);
  }
  return w;
}

// ---- the ring of rows --------------------------------------------------------------
// Stage s of the ring holds rpc rows of x, z (and, backward, dy, dh), each
// array behind the other; a bulk copy per array, on the stage's barrier.
// quit_row: where thread 0 gave up (the other threads' word is not read).
struct Ring {
  uint64_t bar[kMaxStages];
  int64_t quit_row[2];
};

template <bool WIDE>
struct RowBytes {
  static constexpr int kStream = WIDE ? 4 : 2;
};

// Issues the copies of the rows from row0 on into a stage.
template <bool WIDE, bool BACK>
NVFP4_DEV void fetch_rows(const NormArgs& p, uint32_t smem, uint32_t bars, int64_t row0,
                          int stage) {
  if (row0 >= p.rows) return;
  constexpr int kS = RowBytes<WIDE>::kStream;
  const int64_t n = min((int64_t)p.rpc, p.rows - row0) * p.cols;
  const int64_t at = row0 * p.cols;
  const uint32_t area = (uint32_t)p.rpc * p.cols;  // elements of an array in the stage
  uint32_t dst = smem + stage * p.stage_bytes;
  const uint32_t bar = bars + 8u * stage;
  uint32_t bytes = (uint32_t)n * kS;
  if (p.z) bytes += (uint32_t)n * 2;
  if (BACK && p.dy) bytes += (uint32_t)n * kS;
  if (BACK && p.dh) bytes += (uint32_t)n * 2;
  mbar_arrive_expect_tx(bar, bytes);
  bulk_load(dst, static_cast<const char*>(p.x) + at * kS, (uint32_t)n * kS, bar);
  dst += area * kS;
  if (p.z) bulk_load(dst, p.z + at, (uint32_t)n * 2, bar);
  dst += area * 2;
  if (BACK) {
    if (p.dy) bulk_load(dst, static_cast<const char*>(p.dy) + at * kS, (uint32_t)n * kS, bar);
    dst += area * kS;
    if (p.dh) bulk_load(dst, p.dh + at, (uint32_t)n * 2, bar);
  }
}

// Where a row's arrays are read: in its stage, or in global memory.
struct RowPtrs {
  const void* x;
  const uint16_t* z;
  const void* dy;
  const uint16_t* dh;
};
template <bool WIDE, bool RING>
NVFP4_DEV RowPtrs row_ptrs(const NormArgs& p, const uint8_t* smem, int stage, int sub,
                           int64_t row) {
  constexpr int kS = RowBytes<WIDE>::kStream;
  RowPtrs r;
  if (RING) {
    const uint32_t area = (uint32_t)p.rpc * p.cols;
    const uint8_t* s = smem + (uint32_t)stage * p.stage_bytes;
    r.x = s + (uint32_t)sub * p.cols * kS;
    s += area * kS;
    r.z = reinterpret_cast<const uint16_t*>(s) + sub * p.cols;
    s += area * 2;
    r.dy = s + (uint32_t)sub * p.cols * kS;
    s += area * kS;
    r.dh = reinterpret_cast<const uint16_t*>(s) + sub * p.cols;
  } else {
    const int64_t at = row * p.cols;
    r.x = static_cast<const char*>(p.x) + at * kS;
    r.z = p.z + at;
    r.dy = static_cast<const char*>(p.dy) + at * kS;
    r.dh = p.dh + at;
  }
  return r;
}

template <bool WIDE, bool BACK>
NVFP4_DEV void start_ring(const NormArgs& p, Ring& ring, uint32_t smem) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(smem_u32(&ring.bar[s]), 1);
    ring.quit_row[0] = -1;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  if (threadIdx.x == 0) {
    const unsigned int stall = *reinterpret_cast<volatile unsigned int*>(&g_norm_stall);
    if (stall & 2u) mbar_expect_tx(smem_u32(ring.bar), 16);
    if (!(stall & 1u))
      for (int s = 0; s < p.stages; ++s)
        fetch_rows<WIDE, BACK>(p, smem, smem_u32(ring.bar),
                               ((int64_t)blockIdx.x + (int64_t)s * gridDim.x) * p.rpc, s);
  }
}

// The rows of a CTA, one set of rpc after the other, and their stages.
struct Walk {
  int64_t row0, step;
  int stage = 0;
  uint32_t phase = 0;
  bool first = true, dead = false;

  NVFP4_DEV explicit Walk(const NormArgs& p)
      : row0((int64_t)blockIdx.x * p.rpc), step((int64_t)gridDim.x * p.rpc) {}
  NVFP4_DEV void next(const NormArgs& p) {
    row0 += step;
    first = false;
    if (++stage == p.stages) stage = 0, phase ^= 1u;
  }
};

// Until the copies that thread 0 issued have landed, with a limit of its own:
// those of the rows at `at`, where it gave up, and of the sets behind them that
// it had sent for -- `stages` from the start, then one short of that, as a
// refill comes after the wait.
NVFP4_DEV void drain_ring(const NormArgs& p, Ring& ring, Walk at) {
  if (*reinterpret_cast<volatile unsigned int*>(&g_norm_stall) & 1u) return;  // there are none
  const uint64_t t0 = globaltimer_ns();
  for (int i = at.first ? 0 : 1; i < p.stages && at.row0 < p.rows; ++i, at.next(p))
    while (!mbar_try_wait(smem_u32(&ring.bar[at.stage]), at.phase) &&
           globaltimer_ns() - t0 <= kDrainNs) {
    }
}

// Wait with a limit.  A copy that never lands sets the error word; from then
// on nothing is loaded or waited for (the results are void, as the error
// says), and no copy outlives the CTA, whose shared memory is handed on: thread
// 0 waits for them at once or (leave_ring) at the end.  The compiler's code for
// rows that do land depends on which: with one norm forward 16384 x 4096 bf16
// takes 43.6 us with the former, 46.7 with the latter; the backward with both
// norms 161 and 148.
template <bool AT_ONCE>
NVFP4_DEV void wait_row(const NormArgs& p, Ring& ring, Walk& at) {
  const uint32_t bar = smem_u32(&ring.bar[at.stage]);
  if (at.dead || mbar_try_wait(bar, at.phase)) return;
  const uint64_t t0 = globaltimer_ns();
  const uint64_t limit = *reinterpret_cast<volatile unsigned long long*>(&g_norm_wait_ns);
  while (!mbar_try_wait(bar, at.phase)) {
    if (globaltimer_ns() - t0 > limit) {
      atomicCAS(&g_norm_error, 0u, 0x50u);
      if constexpr (AT_ONCE) {
        if (threadIdx.x == 0) drain_ring(p, ring, at);
      } else {
        ring.quit_row[threadIdx.x != 0] = at.row0;
      }
      at.dead = true;
      return;
    }
  }
}

template <bool AT_ONCE>
NVFP4_DEV void leave_ring(const NormArgs& p, Ring& ring) {
  if (AT_ONCE || threadIdx.x != 0 || ring.quit_row[0] < 0) return;
  Walk at(p);
  while (at.row0 < ring.quit_row[0]) at.next(p);
  drain_ring(p, ring, at);
}

// Refills the stage of the rows before, once every thread is done with them
// (called behind a barrier of the CTA).
template <bool WIDE, bool BACK>
NVFP4_DEV void refill(const NormArgs& p, Ring& ring, uint32_t smem, const Walk& at) {
  if (threadIdx.x == 0 && !at.first && !at.dead)
    fetch_rows<WIDE, BACK>(p, smem, smem_u32(ring.bar), at.row0 + (p.stages - 1) * at.step,
                           at.stage == 0 ? p.stages - 1 : at.stage - 1);
}

// Where a thread's weights are: in registers up to 8192 columns; beyond, in
// shared memory (w_post with a channel gate in it, then w_pre) where the ring
// does not need it -- the backward, whose rows are too long for two stages --
// else in global memory.  Measured, 4096 x 16384 bf16: forward 117 us with the
// ring, 187 with shared weights instead; backward 249 us with global weights,
// 229 with shared ones.
enum { kInRegs, kInSmem, kInGlobal };
template <int VPT, bool RING>
struct WeightsAt {
  static constexpr int value = VPT <= kRegVpt ? kInRegs : VPT < kMaxVpt && !RING ? kInSmem : kInGlobal;
};
template <int VPT, bool RING>
struct Weights {
  static constexpr int kAt = WeightsAt<VPT, RING>::value;
  F8 post[kAt == kInRegs ? VPT : 1], pre[kAt == kInRegs ? VPT : 1];
  const float* smem;

  NVFP4_DEV Weights(const NormArgs& p, uint8_t* sm, int tid, int tpr, bool has_post, bool has_pre) {
    smem = reinterpret_cast<const float*>(sm);
    if constexpr (kAt == kInRegs) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * tpr + tid) * kVec;
        post[i] = has_post && c < p.cols ? post_weight(p, c) : zero8();
        pre[i] = has_pre && c < p.cols ? load_f32(p.w_pre + c) : zero8();
      }
    } else if constexpr (kAt == kInSmem) {  // one row a CTA: a thread reads what it wrote
      float* w = reinterpret_cast<float*>(sm);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * tpr + tid) * kVec;
        if (c < p.cols) {
          if (has_post) store_f32(w + c, post_weight(p, c));
          if (has_pre) store_f32(w + p.cols + c, load_f32(p.w_pre + c));
        }
      }
    }
  }
  NVFP4_DEV F8 get_post(const NormArgs& p, int i, int c) const {
    if constexpr (kAt == kInRegs) return post[i];
    if constexpr (kAt == kInSmem) return load_f32(smem + c);
    return post_weight(p, c);
  }
  NVFP4_DEV F8 get_pre(const NormArgs& p, int i, int c) const {
    if constexpr (kAt == kInRegs) return pre[i];
    if constexpr (kAt == kInSmem) return load_f32(smem + p.cols + c);
    return load_f32(p.w_pre + c);
  }
};

template <int VPT, bool WIDE, bool RING, int PARTS>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const NormArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Reducer red;
  __shared__ Ring ring;
  const int tpr = p.wpr * 32, sub = threadIdx.x / tpr, tid = threadIdx.x % tpr;
  const int w0 = sub * p.wpr;  // the row's first warp
  const bool post = has_post<PARTS>(p.z), pre = has_pre<PARTS>(p.h);
  const float inv = 1.0f / (float)p.cols;
  if (RING)
    start_ring<WIDE, false>(p, ring, smem_u32(smem));
  else
    griddep_wait();
  const Weights<VPT, RING> weights(p, smem, tid, tpr, post, pre);
  int turn = 0;
  for (Walk at(p); at.row0 < p.rows; at.next(p)) {
    const int64_t row = at.row0 + sub, at0 = row * p.cols;
    const bool live = row < p.rows;
    const RowPtrs in = row_ptrs<WIDE, RING>(p, smem, at.stage, sub, row);
    if (RING) wait_row<PARTS != kBoth>(p, ring, at);
    float k = 0.0f;  // b [g] r_z
    float s;
    float2 q = both(0.0f);
    if (post) {
      if (live)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = (i * tpr + tid) * kVec;
          if (c < p.cols) {
            const F8 z = load_bf16(in.z + c);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) q = __ffma2_rn(z.v[e], z.v[e], q);
          }
        }
      s = q.x + q.y;
      row_sum(s, red, turn, p.wpr, w0);
      if (RING) refill<WIDE, false>(p, ring, smem_u32(smem), at);
      k = rstd(s, inv, p.eps) * p.b;
      if (p.gate_mode == NVFP4_GATE_ROW && live) k *= p.gate[row];
    }
    F8 y[VPT];
    q = both(0.0f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * tpr + tid) * kVec;
      if (live && c < p.cols) {
        y[i] = load_stream<WIDE>(in.x, c);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) y[i].v[e] = __fmul2_rn(y[i].v[e], both(p.a));
        if (post) {
          const F8 z = load_bf16(in.z + c);
          const F8 w = weights.get_post(p, i, c);
#pragma unroll
          for (int e = 0; e < kPairs; ++e)
            y[i].v[e] = __ffma2_rn(both(k), __fmul2_rn(z.v[e], w.v[e]), y[i].v[e]);
        }
#pragma unroll
        for (int e = 0; e < kPairs; ++e) q = __ffma2_rn(y[i].v[e], y[i].v[e], q);
        if (p.y) store_stream<WIDE>(p.y, at0 + c, y[i]);
      }
    }
    if (pre) {
      s = q.x + q.y;
      row_sum(s, red, turn, p.wpr, w0);
      if (RING && !post) refill<WIDE, false>(p, ring, smem_u32(smem), at);
      const float2 ry = both(rstd(s, inv, p.eps));
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * tpr + tid) * kVec;
        if (live && c < p.cols) {
          const F8 w = weights.get_pre(p, i, c);
          F8 h;
#pragma unroll
          for (int e = 0; e < kPairs; ++e)
            h.v[e] = __fmul2_rn(__fmul2_rn(y[i].v[e], ry), w.v[e]);
          store_bf16(p.h + at0 + c, h);
        }
      }
    }
  }
  if (RING) leave_ring<PARTS != kBoth>(p, ring);
}

template <int VPT, bool WIDE, bool RING, int PARTS>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Reducer red;
  __shared__ Ring ring;
  const int tpr = p.wpr * 32, sub = threadIdx.x / tpr, tid = threadIdx.x % tpr;
  const int w0 = sub * p.wpr;  // the row's first warp
  const bool post = has_post<PARTS>(p.z), pre = has_pre<PARTS>(p.dh);
  const float inv = 1.0f / (float)p.cols;
  if (RING)
    start_ring<WIDE, true>(p, ring, smem_u32(smem));
  else
    griddep_wait();
  const Weights<VPT, RING> weights(p, smem, tid, tpr, post, pre);
  F8 acc_post[VPT], acc_pre[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) acc_post[i] = acc_pre[i] = zero8();
  int turn = 0;
  for (Walk at(p); at.row0 < p.rows; at.next(p)) {
    const int64_t row = at.row0 + sub, at0 = row * p.cols;
    const bool live = row < p.rows;
    const RowPtrs in = row_ptrs<WIDE, RING>(p, smem, at.stage, sub, row);
    if (RING) wait_row<false>(p, ring, at);
    float rz = 0.0f, bg = p.b;  // b [g]
    if (post) {
      float2 q = both(0.0f);
      if (live)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = (i * tpr + tid) * kVec;
          if (c < p.cols) {
            const F8 z = load_bf16(in.z + c);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) q = __ffma2_rn(z.v[e], z.v[e], q);
          }
        }
      float sq = q.x + q.y;
      row_sum(sq, red, turn, p.wpr, w0);
      if (RING) refill<WIDE, true>(p, ring, smem_u32(smem), at);
      rz = rstd(sq, inv, p.eps);
      if (p.gate_mode == NVFP4_GATE_ROW && live) bg *= p.gate[row];
    }
    const float k = bg * rz;
    // One column vector: zc = z c (c = w_post [g]), y = a x + k zc, u = dh w_pre.
    struct Cols {
      F8 z, zc, y, dy, dh, u, w;
    };
    auto columns = [&](int i, int c) {
      Cols v;
      v.y = load_stream<WIDE>(in.x, c);
      v.z = v.zc = v.w = v.dh = v.u = zero8();
      v.dy = p.dy ? load_stream<WIDE>(in.dy, c) : zero8();
#pragma unroll
      for (int e = 0; e < kPairs; ++e) v.y.v[e] = __fmul2_rn(v.y.v[e], both(p.a));
      if (post) {
        v.z = load_bf16(in.z + c);
        v.w = weights.get_post(p, i, c);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          v.zc.v[e] = __fmul2_rn(v.z.v[e], v.w.v[e]);
          v.y.v[e] = __ffma2_rn(both(k), v.zc.v[e], v.y.v[e]);
        }
      }
      if (pre) {
        v.dh = load_bf16(in.dh + c);
        const F8 w = weights.get_pre(p, i, c);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) v.u.v[e] = __fmul2_rn(v.dh.v[e], w.v[e]);
      }
      return v;
    };
    // sums over the row: y^2, u y, and zc times dy, u, y
    float2 q[5] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
    if (live)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * tpr + tid) * kVec;
        if (c < p.cols) {
          const Cols v = columns(i, c);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            q[0] = __ffma2_rn(v.y.v[e], v.y.v[e], q[0]);
            q[1] = __ffma2_rn(v.u.v[e], v.y.v[e], q[1]);
            q[2] = __ffma2_rn(v.zc.v[e], v.dy.v[e], q[2]);
            q[3] = __ffma2_rn(v.zc.v[e], v.u.v[e], q[3]);
            q[4] = __ffma2_rn(v.zc.v[e], v.y.v[e], q[4]);
          }
        }
      }
    float s[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) s[i] = q[i].x + q[i].y;
    row_sum(s, red, turn, p.wpr, w0);
    if (RING && !post) refill<WIDE, true>(p, ring, smem_u32(smem), at);
    float ry = 0.0f, m = 0.0f;  // m = r_y^2 mean(u y): dY = dy + r_y (u - y m)
    if (pre) {
      ry = rstd(s[0], inv, p.eps);
      m = ry * ry * s[1] * inv;
    }
    // sum over the row of dY z^ c; dz = k dY c - (r_z^2 b [g] t / cols) z
    const float t = rz * (s[2] + ry * (s[3] - m * s[4]));
    const float2 k2 = both(k), kz = both(-rz * rz * bg * t * inv);
    const float2 r1 = both(ry), r2 = both(-ry * m);
    if (!live) continue;
    if (p.drow && tid == 0) p.drow[row] = p.b * t;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * tpr + tid) * kVec;
      if (c < p.cols) {
        const Cols v = columns(i, c);
        F8 dx, dz;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          const float2 d =
              __ffma2_rn(r1, v.u.v[e], __ffma2_rn(r2, v.y.v[e], v.dy.v[e]));
          acc_pre[i].v[e] = __ffma2_rn(r1, __fmul2_rn(v.dh.v[e], v.y.v[e]), acc_pre[i].v[e]);
          acc_post[i].v[e] = __ffma2_rn(k2, __fmul2_rn(v.z.v[e], d), acc_post[i].v[e]);
          dx.v[e] = __fmul2_rn(d, both(p.a));
          dz.v[e] = __ffma2_rn(k2, __fmul2_rn(d, v.w.v[e]), __fmul2_rn(kz, v.z.v[e]));
        }
        store_stream<WIDE>(p.dx, at0 + c, dx);
        if (post) store_bf16(p.dz + at0 + c, dz);
      }
    }
  }
  float* out = p.partials + ((int64_t)blockIdx.x * p.rpc + sub) * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * tpr + tid) * kVec;
    if (c < p.cols) {
      if (post) store_f32(out + c, acc_post[i]);
      if (pre) store_f32(out + p.cols + c, acc_pre[i]);
    }
  }
  if (RING) leave_ring<false>(p, ring);
}

// Adds the CTAs' partial column sums: a CTA of 8 warps takes 32 columns of
// one of the two sums, each warp every eighth partial.
__global__ void __launch_bounds__(256) norm_bwd_reduce_kernel(const float* partials, int n,
                                                               int cols, const float* w_post,
                                                               const float* gate, float* dw_post,
                                                               float* dgate, float* dw_pre) {
  __shared__ float red[8][33];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const bool pre = blockIdx.y == 1;
  if (!pre && !dw_post) return;
  float s = 0.0f;
  if (c < cols)
    for (int i = warp; i < n; i += 8) s += partials[((int64_t)i * 2 + (pre ? 1 : 0)) * cols + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    s = red[0][lane];
    for (int w = 1; w < 8; ++w) s += red[w][lane];
    if (pre) {
      dw_pre[c] = s;
    } else {
      // a channel gate leaves the sum without it: dw_post = g S, dg = w_post S
      dw_post[c] = gate ? gate[c] * s : s;
      if (dgate) dgate[c] = w_post[c] * s;
    }
  }
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// How a CTA takes rows of `cols` columns: 16 columns a thread, and rows to
// fill 16 warps (forward) or 8 (backward).  Measured, 16384 x 4096 bf16:
// forward 85 us with 16 warps, 98 with 8; backward 153 and 150 (FP32 stream,
// 8191 rows: 115 and 101).  32 columns a thread, their weights read again for
// each row, lose to 16 everywhere they can be compared (forward 106, backward
// 256 us), so they are taken only where 512 threads need them.
struct Shape {
  int vpt, wpr, rpc, threads;
};
Shape row_shape(int64_t cols, bool back) {
  Shape s;
  const int64_t vecs = cols / kVec;
  s.vpt = kRegVpt;
  if (vecs > (int64_t)kMaxThreads * 2) s.vpt = vecs > (int64_t)kMaxThreads * 4 ? kMaxVpt : 4;
  s.wpr = (int)((vecs + 32 * s.vpt - 1) / (32 * s.vpt));
  s.rpc = std::max(1, (back ? 8 : 16) / s.wpr);
  s.threads = s.wpr * s.rpc * 32;
  return s;
}

// Stages of the ring: as many as leave room for two CTAs on an SM, and at
// least two, for which the longest rows that take a ring have room (196 KB:
// backward 8192 columns, forward 16384, FP32 stream).
constexpr uint32_t kHalfSmem = 110 * 1024, kFullSmem = 220 * 1024;
static_assert(2 * 8192 * 12 <= kFullSmem && 2 * 16384 * 6 <= kFullSmem, "two stages");
int ring_stages(uint64_t stage_bytes) {
  return (int)std::max<uint64_t>(2, std::min<uint64_t>(kMaxStages, kHalfSmem / stage_bytes));
}

// Sets the shared-memory limit of a kernel and looks up the CTAs that fit an SM
// (once for each kernel, device and size).
template <auto KERN>
int ctas_per_sm(int threads, uint32_t smem) {
  struct Slot {
    std::atomic<uint64_t> key{0};  // smem and threads, then the answer
  };
  static Slot slots[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const uint64_t want = ((uint64_t)smem << 24) | ((uint64_t)threads << 8);
  const uint64_t have = slots[dev].key.load(std::memory_order_relaxed);
  if ((have & ~0xFFull) == want && (have & 0xFF)) return (int)(have & 0xFF);
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kFullSmem) != cudaSuccess)
    return 0;
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERN, threads, smem) != cudaSuccess || n < 1)
    return 0;
  slots[dev].key.store(want | (uint64_t)std::min(n, 255), std::memory_order_relaxed);
  return n;
}

// The backward's grid is capped so that the partials stay small.
constexpr int kBwdCtasPerSm = 2;

template <int VPT, bool WIDE, bool RING, int PARTS, bool BACK>
constexpr auto row_kernel() {
  if constexpr (BACK)
    return norm_bwd_kernel<VPT, WIDE, RING, PARTS>;
  else
    return norm_fwd_kernel<VPT, WIDE, RING, PARTS>;
}

template <int VPT, bool WIDE, bool RING, int PARTS, bool BACK>
cudaError_t launch_rows(const NormArgs& p, int threads, int sms, cudaStream_t stream, int* grid) {
  constexpr auto kern = row_kernel<VPT, WIDE, RING, PARTS, BACK>();
  const uint32_t smem = RING                                           ? p.stages * p.stage_bytes
                        : WeightsAt<VPT, RING>::value == kInSmem ? (uint32_t)p.cols * 8
                                                                 : 0u;
  int per_sm = ctas_per_sm<kern>(threads, smem);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  if (BACK) per_sm = std::min(per_sm, kBwdCtasPerSm);
  *grid = (int)std::min<int64_t>((p.rows + p.rpc - 1) / p.rpc, (int64_t)per_sm * sms);
  return launch_pdl(kern, *grid, threads, smem, stream, p);
}

template <int VPT, bool WIDE, bool RING, bool BACK>
cudaError_t launch_parts(const NormArgs& p, int threads, int sms, cudaStream_t stream, int* grid) {
  const bool post = p.z != nullptr, pre = p.w_pre != nullptr;
  if (post && pre) return launch_rows<VPT, WIDE, RING, kBoth, BACK>(p, threads, sms, stream, grid);
  if (post) return launch_rows<VPT, WIDE, RING, kPostOnly, BACK>(p, threads, sms, stream, grid);
  return launch_rows<VPT, WIDE, RING, kPreOnly, BACK>(p, threads, sms, stream, grid);
}

template <bool WIDE, bool BACK>
cudaError_t launch_norm(NormArgs& p, int sms, cudaStream_t stream, int* grid) {
  const Shape s = row_shape(p.cols, BACK);
  p.wpr = s.wpr;
  p.rpc = s.rpc;
  const uint64_t row = (uint64_t)p.cols * ((WIDE ? 4 : 2) + 2) * (BACK ? 2 : 1);
  constexpr bool kRing4 = !BACK;
  p.stages = s.vpt == 2 || (s.vpt == 4 && kRing4) ? ring_stages(row * s.rpc) : 0;
  p.stage_bytes = p.stages ? (uint32_t)(row * s.rpc) : 0u;
  if (s.vpt == 2) return launch_parts<2, WIDE, true, BACK>(p, s.threads, sms, stream, grid);
  if (s.vpt == 4) return launch_parts<4, WIDE, kRing4, BACK>(p, s.threads, sms, stream, grid);
  return launch_rows<kMaxVpt, WIDE, false, kAsGiven, BACK>(p, s.threads, sms, stream, grid);
}

nvfp4_status check_norm(const nvfp4_norm_params* q, const void* x, const void* z,
                        const float* w_post, const float* gate, const float* w_pre) {
  if (!q || !x) return NVFP4_ERR_INVALID_ARG;
  if (q->stream_dtype != NVFP4_IN_BF16 && q->stream_dtype != NVFP4_IN_FP32)
    return NVFP4_ERR_INVALID_ARG;
  if (q->gate_mode < NVFP4_GATE_NONE || q->gate_mode > NVFP4_GATE_ROW)
    return NVFP4_ERR_INVALID_ARG;
  if (!z != !w_post || (q->gate_mode != NVFP4_GATE_NONE) != (gate != nullptr) || (gate && !z))
    return NVFP4_ERR_INVALID_ARG;
  if (!z && !w_pre) return NVFP4_ERR_INVALID_ARG;
  if (!(q->eps > 0.0f) || !(q->eps < 3.0e38f)) return NVFP4_ERR_INVALID_ARG;
  if (!(q->x_scale - q->x_scale == 0.0f) || !(q->z_scale - q->z_scale == 0.0f))
    return NVFP4_ERR_INVALID_ARG;  // finite
  if (q->rows <= 0 || q->cols <= 0 || q->cols % kVec ||
      q->cols > (int64_t)kMaxThreads * kMaxVpt * kVec)
    return NVFP4_ERR_SHAPE;
  if (!a16(x) || !a16(z) || !a16(w_post) || !a16(w_pre) ||
      (q->gate_mode == NVFP4_GATE_CHANNEL ? !a16(gate)
                                          : (reinterpret_cast<uintptr_t>(gate) & 3u) != 0))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

NormArgs norm_args(const nvfp4_norm_params* q, const void* x, const void* z, const float* w_post,
                   const float* gate, const float* w_pre) {
  NormArgs p = {};
  p.x = x;
  p.z = static_cast<const uint16_t*>(z);
  p.w_post = w_post;
  p.gate = gate;
  p.w_pre = w_pre;
  p.rows = q->rows;
  p.cols = (int)q->cols;
  p.gate_mode = q->gate_mode;
  p.eps = q->eps;
  p.a = q->x_scale;
  p.b = q->z_scale;
  return p;
}

size_t bwd_workspace(int64_t rows, int64_t cols, int sms) {
  const int64_t rpc = row_shape(cols, true).rpc;
  return (size_t)std::min<int64_t>((rows + rpc - 1) / rpc, (int64_t)kBwdCtasPerSm * sms) * rpc * 2 *
         cols * sizeof(float);
}

}  // namespace

nvfp4_status norm_set_injection(unsigned int stall, unsigned long long wait_ns) {
  if (cudaMemcpyToSymbol(g_norm_stall, &stall, sizeof(stall)) != cudaSuccess ||
      cudaMemcpyToSymbol(g_norm_wait_ns, &wait_ns, sizeof(wait_ns)) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  return NVFP4_OK;
}

nvfp4_status norm_read_error(unsigned int* code) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_norm_error, sizeof(v)) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (v && cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(zero)) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  *code = v;
  return NVFP4_OK;
}

nvfp4_status norm_fwd_impl(const nvfp4_norm_params* q, const void* x, const void* z,
                           const float* w_post, const float* gate, const float* w_pre, void* y,
                           void* h, cudaStream_t stream) {
  nvfp4_status st = check_norm(q, x, z, w_post, gate, w_pre);
  if (st != NVFP4_OK && st != NVFP4_ERR_ALIGN) return st;
  if ((z && !y) || !w_pre != !h) return NVFP4_ERR_INVALID_ARG;
  if (st != NVFP4_OK || !a16(y) || !a16(h)) return st != NVFP4_OK ? st : NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  NormArgs p = norm_args(q, x, z, w_post, gate, w_pre);
  p.y = y;
  p.h = static_cast<uint16_t*>(h);
  int grid = 0;
  return cuda_status(q->stream_dtype == NVFP4_IN_FP32
                         ? launch_norm<true, false>(p, dev.sm_count, stream, &grid)
                         : launch_norm<false, false>(p, dev.sm_count, stream, &grid));
}

nvfp4_status norm_bwd_sizes_impl(int64_t rows, int64_t cols, size_t* workspace_bytes) {
  if (!workspace_bytes) return NVFP4_ERR_INVALID_ARG;
  if (rows <= 0 || cols <= 0 || cols % kVec || cols > (int64_t)kMaxThreads * kMaxVpt * kVec)
    return NVFP4_ERR_SHAPE;
  // the most CTAs the backward launches on any device of this architecture
  *workspace_bytes = bwd_workspace(rows, cols, kMaxSms);
  return NVFP4_OK;
}

nvfp4_status norm_bwd_impl(const nvfp4_norm_params* q, const void* dy, const void* dh,
                           const void* x, const void* z, const float* w_post, const float* gate,
                           const float* w_pre, void* dx, void* dz, float* dw_post, float* dgate,
                           float* dw_pre, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
  nvfp4_status st = check_norm(q, x, z, w_post, gate, w_pre);
  if (st != NVFP4_OK && st != NVFP4_ERR_ALIGN) return st;
  if (!dx || !w_pre != !dh || (!dy && !dh) || !z != !dz || !w_post != !dw_post ||
      !gate != !dgate || !w_pre != !dw_pre)
    return NVFP4_ERR_INVALID_ARG;
  auto a4 = [](const void* t) { return (reinterpret_cast<uintptr_t>(t) & 3u) == 0; };
  if (st != NVFP4_OK || !a16(dy) || !a16(dh) || !a16(dx) || !a16(dz) || !a4(dw_post) ||
      !a4(dgate) || !a4(dw_pre))
    return NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  const int sms = std::min(dev.sm_count, kMaxSms);
  if (!workspace || !a16(workspace) || workspace_bytes < bwd_workspace(q->rows, q->cols, sms))
    return NVFP4_ERR_WORKSPACE;
  NormArgs p = norm_args(q, x, z, w_post, gate, w_pre);
  p.dy = dy;
  p.dh = static_cast<const uint16_t*>(dh);
  p.dx = dx;
  p.dz = static_cast<uint16_t*>(dz);
  p.drow = q->gate_mode == NVFP4_GATE_ROW ? dgate : nullptr;
  p.partials = static_cast<float*>(workspace);
  int grid = 0;
  if ((q->stream_dtype == NVFP4_IN_FP32 ? launch_norm<true, true>(p, sms, stream, &grid)
                                        : launch_norm<false, true>(p, sms, stream, &grid)) !=
      cudaSuccess)
    return NVFP4_ERR_CUDA;
  const bool channel = q->gate_mode == NVFP4_GATE_CHANNEL;
  const int first = z ? 0 : 1, sums = (z ? 1 : 0) + (w_pre ? 1 : 0);
  // blockIdx.y 0 is the post sum, 1 the pre sum; without z only the latter
  const dim3 rgrid((unsigned)((q->cols + 31) / 32), (unsigned)(first + sums));
  return cuda_status(launch_pdl(norm_bwd_reduce_kernel, rgrid, dim3(256), 0, stream,
                                (const float*)p.partials, grid * p.rpc, (int)q->cols, w_post,
                                channel ? gate : (const float*)nullptr, dw_post,
                                channel ? dgate : (float*)nullptr, dw_pre));
}

}  // namespace nvfp4
