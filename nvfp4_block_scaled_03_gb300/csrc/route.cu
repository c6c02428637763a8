// route.cu -- routing of a mixture of experts: the choice of each token's k
// experts and their weights, the plan that orders the chosen rows by expert,
// and the rows' way to the experts (dispatch) and back (combine), with the
// gradients.
//
// Choice: the k largest logits of a row, the largest first, the lowest index
// among equals; compared on the bit patterns (mapped so that unsigned order is
// the floats' order), so the choice is exact.  -inf and NaN are never chosen.
// One warp takes a token, two at a time: lane l holds experts NI l .. NI l + NI
// - 1; each of the k rounds is a local maximum and one warp reduction (redux).
// A bf16 logit leaves 16 bits of its key for the index, so the reduction finds
// both; for FP32 a ballot follows, whose first lane holds the lowest index.
// The instructions of the rounds set the time (16384 tokens, 8 of 128 experts).
//
// Plan: expert e owns rows offsets[e] .. offsets[e] + sizes[e] - 1, in the
// order of (token, slot), and the offsets are multiples of 128, the rows of a
// scale atom.  The first kernel clears `source` and counts each CTA's choices
// per expert, the second turns the counts into running sums over the CTAs, the
// third ranks each CTA's choices warp by warp.  (Two kernels, the last summing
// the counts of the CTAs before it by itself, read 152 x experts counts in
// every CTA: 4096 tokens of 512 experts took 43 us that way.)  No atomic
// decides an order: the plan is the same every time.  Few tokens take one CTA
// and one launch for all of it.
#include <algorithm>
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kWarps = 16;            // that rank a CTA's choices
constexpr int kThreads = kWarps * 32;
constexpr int kChooseWarps = 32;      // that make them
constexpr int kChooseThreads = kChooseWarps * 32;
constexpr int kMaxExperts = 512;
constexpr int kMaxTop = 16;
constexpr int kGroupAlign = 128;
constexpr int kSmallTokens = 2 * kChooseWarps;  // up to here one CTA does it all

struct RouteArgs {
  const void* logits;
  int64_t ld;
  int tokens, experts, top;
  int mode;
  int per_cta;  // tokens of a CTA
  int32_t* expert;
  float* weight;
  int32_t* sizes;
  int32_t* offsets;
  int32_t* row;
  int32_t* source;
  int64_t rows;     // entries of source
  int32_t* counts;  // [CTAs + 1][experts], after the second kernel running sums
  int ctas;
  // backward
  const float* dweight;
  void* dlogits;
};

template <bool WIDE>
NVFP4_DEV float load_logit(const void* p, int64_t at) {
  if (WIDE) return static_cast<const float*>(p)[at];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[at] << 16);
}

// Unsigned key in the order of the floats, 0 for what is never chosen; +-0 are
// equal, and +inf counts as the type's largest finite value.  A bf16 logit's
// key has its expert e in the low half, the lower the larger.
template <bool WIDE>
NVFP4_DEV uint32_t logit_key(float& v, int e) {
  const bool none = !(v > -INFINITY);
  v = none ? -INFINITY : fminf(v, WIDE ? 3.402823466e38f : 3.3895314e38f) + 0.0f;
  const uint32_t b = __float_as_uint(v);
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return none ? 0u : WIDE ? k : (k & 0xFFFF0000u) | (0xFFFFu - (uint32_t)e);
}

NVFP4_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The logits of one token in a warp's registers: value and key of experts
// NI lane + i.
template <int NI, bool WIDE>
NVFP4_DEV void load_token(const RouteArgs& a, int64_t t, int lane, float (&v)[NI],
                          uint32_t (&key)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = NI * lane + i;
    v[i] = e < a.experts ? load_logit<WIDE>(a.logits, t * a.ld + e) : -INFINITY;
    key[i] = logit_key<WIDE>(v[i], e);
  }
}

template <bool WIDE>
NVFP4_DEV float key_value(uint32_t k) {
  const uint32_t b = (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k;
  return __uint_as_float(WIDE ? b : b & 0xFFFF0000u);
}

// The tokens of one of `warps` warps of this CTA: [first, last).  Counted from the
// CTA's first token, which is one: the ends of shares may lie beyond 2^31.
NVFP4_DEV void warp_tokens(const RouteArgs& a, int warps, int& first, int& last) {
  const int per = (a.per_cta + warps - 1) / warps, c0 = blockIdx.x * a.per_cta;
  const int n = min(a.per_cta, a.tokens - c0), w = (int)(threadIdx.x >> 5) * per;
  first = c0 + min(w, n);
  last = c0 + min(w + per, n);
}

// Experts and weights of B tokens from t on, one warp: to global memory, and
// counted in `hist` (shared).
template <int NI, bool WIDE, int B>
NVFP4_DEV void choose_tokens(const RouteArgs& a, int t, int* hist) {
  const int lane = threadIdx.x & 31;
  uint32_t key[B][NI];
  float v[B][NI], top_logit[B], my_logit[B], all[B];
  int my_expert[B];
#pragma unroll
  for (int b = 0; b < B; ++b)
    load_token<NI, WIDE>(a, t + b, lane, v[b], key[b]);
#pragma unroll
  for (int b = 0; b < B; ++b) {
    uint32_t best = key[b][0];
#pragma unroll
    for (int i = 1; i < NI; ++i) best = max(best, key[b][i]);
    top_logit[b] = key_value<WIDE>(max(__reduce_max_sync(0xFFFFFFFFu, best), 1u));
    all[b] = my_logit[b] = 0.0f;
    my_expert[b] = -1;
    if (a.mode == NVFP4_ROUTE_ALL)
#pragma unroll
      for (int i = 0; i < NI; ++i)
        all[b] += key[b][i] ? expf(v[b][i] - top_logit[b]) : 0.0f;
  }
  for (int j = 0; j < a.top; ++j) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      uint32_t best = key[b][0];
#pragma unroll
      for (int i = 1; i < NI; ++i) best = max(best, key[b][i]);
      // m is 0 where nothing is left to choose; then the slot stays empty
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
      int e;
      if (WIDE) {
        int at = 0;
#pragma unroll
        for (int i = NI - 1; i >= 0; --i) at = key[b][i] == m ? i : at;
        const int from = __ffs(__ballot_sync(0xFFFFFFFFu, best == m)) - 1;
        e = NI * from + __shfl_sync(0xFFFFFFFFu, at, from);
      } else {
        e = 0xFFFF - (int)(m & 0xFFFFu);
      }
      const bool slot = lane == j && m != 0u;
      my_expert[b] = slot ? e : my_expert[b];
      my_logit[b] = slot ? key_value<WIDE>(m) : my_logit[b];
#pragma unroll
      for (int i = 0; i < NI; ++i)
        key[b][i] = (WIDE ? e - NI * lane == i : key[b][i] == m) ? 0u : key[b][i];
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const float ex = my_expert[b] >= 0 ? expf(my_logit[b] - top_logit[b]) : 0.0f;
    const float total = warp_sum(a.mode == NVFP4_ROUTE_CHOSEN ? ex : all[b]);
    if (lane < a.top) {
      const int64_t at = (int64_t)(t + b) * a.top + lane;
      a.expert[at] = my_expert[b];
      a.weight[at] = my_expert[b] >= 0 ? ex / total : 0.0f;
      if (my_expert[b] >= 0) atomicAdd(&hist[my_expert[b]], 1);
    }
  }
}

// Step 1 for the tokens of this CTA; this CTA's part of `source` is cleared.
template <int NI, bool WIDE>
NVFP4_DEV void choose(const RouteArgs& a, int* hist) {
  for (int e = threadIdx.x; e < a.experts; e += kChooseThreads) hist[e] = 0;
  for (int64_t r = (int64_t)blockIdx.x * kChooseThreads + threadIdx.x; r < a.rows;
       r += (int64_t)gridDim.x * kChooseThreads)
    a.source[r] = -1;
  __syncthreads();
  int t, t1;
  warp_tokens(a, kChooseWarps, t, t1);
  if (NI <= 8)  // more would not leave registers for two tokens
    for (; t + 1 < t1; t += 2) choose_tokens<NI, WIDE, 2>(a, t, hist);
  for (; t < t1; ++t) choose_tokens<NI, WIDE, 1>(a, t, hist);
  __syncthreads();
}

// Step 2: rows of this CTA's choices.  before[e]: choices of e in the CTAs
// before this one; total[e]: in all.  Both in shared memory; base [kWarps]
// [experts] is scratch.  The slots' experts are read twice (counted, then
// placed): the second time from L1.  The first kWarps warps work.
NVFP4_DEV void assign(const RouteArgs& a, const int* before, const int* total, int* offset,
                      int* base) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = threadIdx.x < kThreads ? threadIdx.x : INT_MAX / 2;  // else beyond every loop
  // offsets: warp 0 scans the padded sizes, 32 experts at a time
  if (warp == 0) {
    int run = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 32) {
      const int e = e0 + lane;
      const int size = e < a.experts ? total[e] : 0;
      const int padded = (size + kGroupAlign - 1) / kGroupAlign * kGroupAlign;
      int s = padded;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
      }
      if (e < a.experts) {
        offset[e] = run + s - padded;
        if (blockIdx.x == 0) {
          a.sizes[e] = size;
          a.offsets[e] = run + s - padded;
        }
      }
      run += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane == 0 && blockIdx.x == 0) a.offsets[a.experts] = run;
  }
  for (int i = tid; i < kWarps * a.experts; i += kThreads) base[i] = 0;
  __syncthreads();
  int t0 = 0, t1 = 0;
  if (warp < kWarps) warp_tokens(a, kWarps, t0, t1);
  int* mine = base + warp * a.experts;
  const int64_t i0 = (int64_t)t0 * a.top, i1 = (int64_t)t1 * a.top;
  for (int64_t i = i0 + lane; i < i1; i += 32) {
    const int e = a.expert[i];
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < a.experts; e += kThreads) {
    int n[kWarps], run = offset[e] + before[e];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) n[w] = base[w * a.experts + e];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      base[w * a.experts + e] = run;
      run += n[w];
    }
  }
  __syncthreads();
  // a token's experts differ, so its slots take their places side by side;
  // the warp's tokens follow one another
  int next = -1;
  if (lane < a.top && t0 < t1) next = a.expert[i0 + lane];
  for (int t = t0; t < t1; ++t) {
    const int64_t i = (int64_t)t * a.top + lane;
    const int e = next;
    if (lane < a.top) {
      if (t + 1 < t1) next = a.expert[i + a.top];
      int r = -1;
      if (e >= 0) {
        r = mine[e]++;
        if (r < a.rows) a.source[r] = (int32_t)i;
      }
      a.row[i] = r;
    }
    __syncwarp();
  }
}

template <int NI, bool WIDE>
__global__ void __launch_bounds__(kChooseThreads) route_choose_kernel(const RouteArgs a) {
  __shared__ int hist[kMaxExperts];
  griddep_wait();
  choose<NI, WIDE>(a, hist);
  for (int e = threadIdx.x; e < a.experts; e += kChooseThreads)
    a.counts[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

struct AssignSmem {
  int before[kMaxExperts], total[kMaxExperts], offset[kMaxExperts];
  int base[kWarps * kMaxExperts];
};

// counts [CTAs][experts] becomes its running sums over the CTAs, without the
// CTA's own, and the totals behind them.  A CTA takes 32 experts (lanes), its
// 32 warps up to five CTAs' counts each.
__global__ void __launch_bounds__(1024) route_scan_kernel(const RouteArgs a) {
  constexpr int kPer = (kMaxSms + 31) / 32;
  __shared__ int part[32][33];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  int n[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = warp * kPer + i;
    n[i] = e < a.experts && b < a.ctas ? a.counts[(int64_t)b * a.experts + e] : 0;
    sum += n[i];
  }
  part[warp][lane] = sum;
  __syncthreads();
  // warp w scans expert w of the 32 over the parts
  int v = part[lane][warp];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  part[lane][warp] = v;
  __syncthreads();
  int run = part[warp][lane] - sum;
  if (e >= a.experts) return;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = warp * kPer + i;
    if (b < a.ctas) a.counts[(int64_t)b * a.experts + e] = run;
    run += n[i];
  }
  if (warp == 31) a.counts[(int64_t)a.ctas * a.experts + e] = run;
}

__global__ void __launch_bounds__(kThreads) route_assign_kernel(const RouteArgs a) {
  __shared__ AssignSmem s;
  griddep_wait();
  for (int e = threadIdx.x; e < a.experts; e += kThreads) {
    s.before[e] = a.counts[(int64_t)blockIdx.x * a.experts + e];
    s.total[e] = a.counts[(int64_t)a.ctas * a.experts + e];
  }
  __syncthreads();
  assign(a, s.before, s.total, s.offset, s.base);
}

template <int NI, bool WIDE>
__global__ void __launch_bounds__(kChooseThreads) route_small_kernel(const RouteArgs a) {
  __shared__ AssignSmem s;
  griddep_wait();
  choose<NI, WIDE>(a, s.total);
  for (int e = threadIdx.x; e < a.experts; e += kChooseThreads) s.before[e] = 0;
  __syncthreads();
  assign(a, s.before, s.total, s.offset, s.base);
}

// dl_i = w_i sum_j w_j (dw_i - dw_j) over the chosen (i, j); with the softmax
// over all experts the unchosen, whose weights have no gradient, add their
// share of probability times dw_i, and themselves get -p sum_j w_j dw_j.  The
// differences keep the result exact where one weight is near 1.
// A token's row lies in shared memory: the lanes of its slots put theirs
// into it.
template <int NI, bool WIDE>
__global__ void __launch_bounds__(kThreads) route_bwd_kernel(const RouteArgs a) {
  __shared__ float rows[kWarps][NI * 32];
  griddep_wait();
  const int lane = threadIdx.x & 31;
  float* p = rows[threadIdx.x >> 5];
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  int e = -1;
  float w = 0.0f, dw = 0.0f;
  if (lane < a.top) {
    e = a.expert[t * a.top + lane];
    if (e >= 0 && e < a.experts) {
      w = a.weight[t * a.top + lane];
      dw = a.dweight[t * a.top + lane];
    } else {
      e = -1;
    }
  }
  float apart = 0.0f;
  for (int j = 0; j < a.top; ++j)
    apart += __shfl_sync(0xFFFFFFFFu, w, j) * (dw - __shfl_sync(0xFFFFFFFFu, dw, j));
  float other = 0.0f;  // what an unchosen expert's probability is multiplied by
  if (a.mode == NVFP4_ROUTE_ALL) {
    other = -warp_sum(w * dw);
    float v[NI];
    uint32_t key[NI], best = 0u;
    load_token<NI, WIDE>(a, t, lane, v, key);
#pragma unroll
    for (int i = 0; i < NI; ++i) best = max(best, key[i]);
    const float l = key_value<WIDE>(max(__reduce_max_sync(0xFFFFFFFFu, best), 1u));
    float all = 0.0f, rest = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      v[i] = key[i] ? expf(v[i] - l) : 0.0f;
      p[NI * lane + i] = v[i];
      all += v[i];
    }
    all = warp_sum(all);
    const float inv = all > 0.0f ? 1.0f / all : 0.0f;
    __syncwarp();
    if (e >= 0) p[e] = 0.0f;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      v[i] = p[lane + 32 * i] * inv;
      rest += v[i];
      p[lane + 32 * i] = v[i] * other;
    }
    apart += warp_sum(rest) * dw;
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) p[lane + 32 * i] = 0.0f;
  }
  __syncwarp();
  if (e >= 0) p[e] = w * apart;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = lane + 32 * i;
    if (c < a.experts) {
      if (WIDE)
        static_cast<float*>(a.dlogits)[t * a.experts + c] = p[c];
      else
        static_cast<__nv_bfloat16*>(a.dlogits)[t * a.experts + c] = __float2bfloat16_rn(p[c]);
    }
  }
}

// ---- rows to the experts and back ------------------------------------------------
// A token is taken by `tpr` threads of a 256-thread CTA, a power of two from 32
// on, each 8 columns at a time.  The kernels move rows whole and are bound by
// memory; a token's rows (and weights) are looked up once and all its loads
// are issued before the first is used.  The first CTAs of a grid clear the
// padding rows, eight entries of `source` a warp.
constexpr int kMoveThreads = 256;

struct MoveArgs {
  const uint16_t* in;      // dispatch: x; combine: the experts' rows; its backward: dy
  const uint16_t* rows_in; // combine backward: the experts' rows
  const int32_t* row;
  const int32_t* source;
  const float* weight;
  uint16_t* out;
  float* dweight;
  int64_t tokens, rows;
  int cols, top, tpr;
  unsigned clear_ctas;  // the first CTAs, which clear padding rows
};

NVFP4_DEV void unpack8(const uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
NVFP4_DEV uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
NVFP4_DEV uint4 load8(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
NVFP4_DEV void store8(uint16_t* p, const uint4 v) { *reinterpret_cast<uint4*>(p) = v; }

// The rows of `out` without a source become zero.
constexpr int kClearRows = 8;  // of a warp
NVFP4_DEV void clear_padding(const MoveArgs& a) {
  const int lane = threadIdx.x & 31;
  const int64_t r0 =
      ((int64_t)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * kClearRows;
  const bool pad = lane < kClearRows && r0 + lane < a.rows && a.source[r0 + lane] < 0;
  for (unsigned todo = __ballot_sync(0xFFFFFFFFu, pad); todo; todo &= todo - 1) {
    uint16_t* row = a.out + (r0 + __ffs(todo) - 1) * a.cols;
    for (int c = lane * 8; c < a.cols; c += 256) store8(row + c, make_uint4(0u, 0u, 0u, 0u));
  }
}

// The rows of token t's slots: -1 for none, or for what is not a row of the tensor.
template <int TOP>
NVFP4_DEV void slot_rows(const MoveArgs& a, int64_t t, bool live, int (&r)[TOP]) {
#pragma unroll
  for (int j = 0; j < TOP; ++j) {
    r[j] = live && j < a.top ? a.row[t * a.top + j] : -1;
    if ((uint32_t)r[j] >= (uint64_t)a.rows) r[j] = -1;
  }
}

template <int TOP>
__global__ void __launch_bounds__(kMoveThreads) dispatch_kernel(const MoveArgs a) {
  griddep_wait();
  if (blockIdx.x < a.clear_ctas) return clear_padding(a);
  const int sub = threadIdx.x / a.tpr, tid = threadIdx.x % a.tpr;
  const int64_t t = (int64_t)(blockIdx.x - a.clear_ctas) * (kMoveThreads / a.tpr) + sub;
  if (t >= a.tokens) return;
  int r[TOP];
  slot_rows<TOP>(a, t, true, r);
#pragma unroll 2
  for (int c = tid * 8; c < a.cols; c += a.tpr * 8) {
    const uint4 v = load8(a.in + t * a.cols + c);
#pragma unroll
    for (int j = 0; j < TOP; ++j)
      if (r[j] >= 0) store8(a.out + (int64_t)r[j] * a.cols + c, v);
  }
}

template <int TOP>
__global__ void __launch_bounds__(kMoveThreads) combine_kernel(const MoveArgs a) {
  griddep_wait();
  const int sub = threadIdx.x / a.tpr, tid = threadIdx.x % a.tpr;
  const int64_t t = (int64_t)(blockIdx.x - a.clear_ctas) * (kMoveThreads / a.tpr) + sub;
  if (t >= a.tokens) return;
  int r[TOP];
  float w[TOP];
  slot_rows<TOP>(a, t, true, r);
#pragma unroll
  for (int j = 0; j < TOP; ++j) w[j] = a.weight && j < a.top ? a.weight[t * a.top + j] : 1.0f;
#pragma unroll(TOP <= 4 ? 2 : 1)
  for (int c = tid * 8; c < a.cols; c += a.tpr * 8) {
    uint4 in[TOP];
#pragma unroll
    for (int j = 0; j < TOP; ++j)
      if (r[j] >= 0) in[j] = load8(a.in + (int64_t)r[j] * a.cols + c);
    float s[8] = {};
#pragma unroll
    for (int j = 0; j < TOP; ++j) {
      if (r[j] < 0) continue;
      float v[8];
      unpack8(in[j], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = fmaf(w[j], v[e], s[e]);
    }
    store8(a.out + t * a.cols + c, pack8(s));
  }
}

// do[row] = w dy, dw = <dy, o[row]>: dy is read once for all of a token's
// slots, whose products each thread carries in registers.
template <int TOP>
__global__ void __launch_bounds__(kMoveThreads) combine_bwd_kernel(const MoveArgs a) {
  __shared__ float red[kMoveThreads / 32][TOP];
  griddep_wait();
  if (blockIdx.x < a.clear_ctas) return clear_padding(a);
  const int sub = threadIdx.x / a.tpr, tid = threadIdx.x % a.tpr;
  const int64_t t = (int64_t)(blockIdx.x - a.clear_ctas) * (kMoveThreads / a.tpr) + sub;
  const bool live = t < a.tokens;
  int r[TOP];
  float w[TOP], dot[TOP] = {};
  slot_rows<TOP>(a, t, live, r);
#pragma unroll
  for (int j = 0; j < TOP; ++j) w[j] = r[j] >= 0 ? a.weight[t * a.top + j] : 0.0f;
  if (live) {
#pragma unroll(TOP <= 4 ? 2 : 1)
    for (int c = tid * 8; c < a.cols; c += a.tpr * 8) {
      const uint4 dyv = load8(a.in + t * a.cols + c);
      uint4 in[TOP];
#pragma unroll
      for (int j = 0; j < TOP; ++j)
        if (r[j] >= 0) in[j] = load8(a.rows_in + (int64_t)r[j] * a.cols + c);
      float d[8];
      unpack8(dyv, d);
#pragma unroll
      for (int j = 0; j < TOP; ++j) {
        if (r[j] < 0) continue;
        float v[8];
        unpack8(in[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dot[j] = fmaf(d[e], v[e], dot[j]);
          v[e] = w[j] * d[e];
        }
        store8(a.out + (int64_t)r[j] * a.cols + c, pack8(v));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TOP; ++j) dot[j] = warp_sum(dot[j]);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int j = 0; j < TOP; ++j) red[threadIdx.x >> 5][j] = dot[j];
  __syncthreads();
  if (live && tid < a.top) {
    float s = 0.0f;
    for (int i = 0; i < a.tpr / 32; ++i) s += red[sub * (a.tpr / 32) + i][tid];
    a.dweight[t * a.top + tid] = s;  // 0 for a slot without a row
  }
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool a4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// CTAs of the routing kernels: at most one per SM, and where there are fewer
// tokens than warps on the device, eight a CTA.
int route_ctas(int64_t tokens, int sms) {
  if (tokens <= kSmallTokens) return 1;
  return (int)std::min<int64_t>(std::min(sms, kMaxSms), (tokens + 7) / 8);
}

nvfp4_status check_route(int64_t tokens, int64_t experts, int32_t top) {
  if (tokens <= 0 || tokens > INT32_MAX || experts <= 0 || experts > kMaxExperts || top <= 0 || top > kMaxTop ||
      top > experts)
    return NVFP4_ERR_SHAPE;
  if (route_rows(tokens, experts, top) > INT32_MAX) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

template <int NI, bool WIDE>
cudaError_t launch_route(RouteArgs& a, int ctas, cudaStream_t stream) {
  if (ctas == 1) return launch_pdl(route_small_kernel<NI, WIDE>, 1, kChooseThreads, 0, stream, a);
  const cudaError_t e = launch_pdl(route_choose_kernel<NI, WIDE>, ctas, kChooseThreads, 0, stream, a);
  if (e != cudaSuccess) return e;
  const cudaError_t f = launch_pdl(route_scan_kernel, (a.experts + 31) / 32, 1024, 0, stream, a);
  if (f != cudaSuccess) return f;
  return launch_pdl(route_assign_kernel, ctas, kThreads, 0, stream, a);
}

template <int NI, bool WIDE>
cudaError_t launch_route_bwd(RouteArgs& a, cudaStream_t stream) {
  const int64_t ctas = ((int64_t)a.tokens + kWarps - 1) / kWarps;
  return launch_pdl(route_bwd_kernel<NI, WIDE>, dim3((unsigned)ctas), kThreads, 0, stream, a);
}

// Calls F<NI, WIDE> for a number of experts.
#define NVFP4_ROUTE_CALL(F, experts, wide, ...)                                        \
  ((experts) <= 32    ? ((wide) ? F<1, true>(__VA_ARGS__) : F<1, false>(__VA_ARGS__))  \
   : (experts) <= 64  ? ((wide) ? F<2, true>(__VA_ARGS__) : F<2, false>(__VA_ARGS__))  \
   : (experts) <= 128 ? ((wide) ? F<4, true>(__VA_ARGS__) : F<4, false>(__VA_ARGS__))  \
   : (experts) <= 256 ? ((wide) ? F<8, true>(__VA_ARGS__) : F<8, false>(__VA_ARGS__))  \
                      : ((wide) ? F<16, true>(__VA_ARGS__) : F<16, false>(__VA_ARGS__)))

nvfp4_status check_move(int64_t tokens, int64_t cols, int32_t top, int64_t rows) {
  if (tokens <= 0 || cols <= 0 || cols % 8 || cols > INT32_MAX / 2 || top <= 0 || top > kMaxTop ||
      rows <= 0)
    return NVFP4_ERR_SHAPE;
  if (tokens > INT32_MAX || rows > INT32_MAX || tokens + rows > INT32_MAX) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

// Threads per row: a power of two that leaves each about two vectors of 8.
int move_tpr(int64_t cols) {
  int tpr = 32;
  while (tpr < kMoveThreads && tpr * 16 < cols) tpr *= 2;
  return tpr;
}

// CTAs that look after the padding rows.
unsigned clear_ctas(int64_t rows) {
  constexpr int per = kMoveThreads / 32 * kClearRows;
  return (unsigned)((rows + per - 1) / per);
}

// F<TOP> for the slots of a token.
#define NVFP4_MOVE_KERNEL(F, top) \
  ((top) <= 1 ? F<1> : (top) <= 2 ? F<2> : (top) <= 4 ? F<4> : (top) <= 8 ? F<8> : F<16>)

}  // namespace

int64_t route_rows(int64_t tokens, int64_t experts, int32_t top) {
  const int64_t n = tokens * top;
  return (n + (kGroupAlign - 1) * std::min<int64_t>(experts, n)) / kGroupAlign * kGroupAlign;
}

nvfp4_status route_sizes_impl(int64_t tokens, int64_t experts, int32_t top, int64_t* rows,
                              size_t* workspace_bytes) {
  const nvfp4_status st = check_route(tokens, experts, top);
  if (st != NVFP4_OK) return st;
  if (rows) *rows = route_rows(tokens, experts, top);
  if (workspace_bytes) *workspace_bytes = (size_t)(kMaxSms + 1) * experts * sizeof(int32_t);
  return NVFP4_OK;
}

nvfp4_status route_fwd_impl(const void* logits, int32_t in_dtype, int64_t tokens,
                            int64_t experts, int64_t ld, int32_t top, int32_t mode,
                            int32_t* expert, float* weight, int32_t* sizes, int32_t* offsets,
                            int32_t* row, int32_t* source, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  if (!logits || !expert || !weight || !sizes || !offsets || !row || !source)
    return NVFP4_ERR_INVALID_ARG;
  if (in_dtype != NVFP4_IN_BF16 && in_dtype != NVFP4_IN_FP32) return NVFP4_ERR_INVALID_ARG;
  if (mode != NVFP4_ROUTE_ALL && mode != NVFP4_ROUTE_CHOSEN) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = check_route(tokens, experts, top);
  if (st != NVFP4_OK) return st;
  if (ld < experts) return NVFP4_ERR_SHAPE;
  const bool wide = in_dtype == NVFP4_IN_FP32;
  if ((reinterpret_cast<uintptr_t>(logits) & (wide ? 3u : 1u)) || !a4(expert) || !a4(weight) ||
      !a4(sizes) || !a4(offsets) || !a4(row) || !a4(source))
    return NVFP4_ERR_ALIGN;
  if (!workspace || !a4(workspace) ||
      workspace_bytes < (size_t)(kMaxSms + 1) * experts * sizeof(int32_t))
    return NVFP4_ERR_WORKSPACE;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  RouteArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.tokens = (int)tokens;
  a.experts = (int)experts;
  a.top = top;
  a.mode = mode;
  a.expert = expert;
  a.weight = weight;
  a.sizes = sizes;
  a.offsets = offsets;
  a.row = row;
  a.source = source;
  a.rows = route_rows(tokens, experts, top);
  a.counts = static_cast<int32_t*>(workspace);
  int ctas = route_ctas(tokens, dev.sm_count);
  a.per_cta = (int)((tokens + ctas - 1) / ctas);
  ctas = a.ctas = (int)((tokens + a.per_cta - 1) / a.per_cta);
  return cuda_status(NVFP4_ROUTE_CALL(launch_route, experts, wide, a, ctas, stream));
}

nvfp4_status route_bwd_impl(const void* logits, int32_t in_dtype, int64_t tokens,
                            int64_t experts, int64_t ld, int32_t top, int32_t mode,
                            const int32_t* expert, const float* weight, const float* dweight,
                            void* dlogits, cudaStream_t stream) {
  if (!logits || !expert || !weight || !dweight || !dlogits) return NVFP4_ERR_INVALID_ARG;
  if (in_dtype != NVFP4_IN_BF16 && in_dtype != NVFP4_IN_FP32) return NVFP4_ERR_INVALID_ARG;
  if (mode != NVFP4_ROUTE_ALL && mode != NVFP4_ROUTE_CHOSEN) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = check_route(tokens, experts, top);
  if (st != NVFP4_OK) return st;
  if (ld < experts) return NVFP4_ERR_SHAPE;
  const bool wide = in_dtype == NVFP4_IN_FP32;
  const unsigned el = wide ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(logits) & el) || (reinterpret_cast<uintptr_t>(dlogits) & el) ||
      !a4(expert) || !a4(weight) || !a4(dweight))
    return NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  RouteArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.tokens = (int)tokens;
  a.experts = (int)experts;
  a.top = top;
  a.mode = mode;
  a.expert = const_cast<int32_t*>(expert);
  a.weight = const_cast<float*>(weight);
  a.dweight = dweight;
  a.dlogits = dlogits;
  return cuda_status(NVFP4_ROUTE_CALL(launch_route_bwd, experts, wide, a, stream));
}

nvfp4_status dispatch_impl(const void* x, const int32_t* row, const int32_t* source,
                           int64_t tokens, int64_t cols, int32_t top, int64_t rows, void* xe,
                           cudaStream_t stream) {
  if (!x || !row || !source || !xe) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = check_move(tokens, cols, top, rows);
  if (st != NVFP4_OK) return st;
  if (!a16(x) || !a16(xe) || !a4(row) || !a4(source)) return NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  MoveArgs a = {};
  a.in = static_cast<const uint16_t*>(x);
  a.row = row;
  a.source = source;
  a.out = static_cast<uint16_t*>(xe);
  a.tokens = tokens;
  a.rows = rows;
  a.cols = (int)cols;
  a.top = top;
  a.tpr = move_tpr(cols);
  const int per = kMoveThreads / a.tpr;
  a.clear_ctas = clear_ctas(rows);
  const unsigned token_ctas = (unsigned)((tokens + per - 1) / per);
  return cuda_status(launch_pdl(NVFP4_MOVE_KERNEL(dispatch_kernel, top),
                                a.clear_ctas + token_ctas, kMoveThreads, 0, stream, a));
}

nvfp4_status combine_impl(const void* o, const int32_t* row, const float* weight, int64_t tokens,
                          int64_t cols, int32_t top, int64_t rows, void* y, cudaStream_t stream) {
  if (!o || !row || !y) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = check_move(tokens, cols, top, rows);
  if (st != NVFP4_OK) return st;
  if (!a16(o) || !a16(y) || !a4(row) || !a4(weight)) return NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  MoveArgs a = {};
  a.in = static_cast<const uint16_t*>(o);
  a.row = row;
  a.weight = weight;
  a.out = static_cast<uint16_t*>(y);
  a.tokens = tokens;
  a.rows = rows;
  a.cols = (int)cols;
  a.top = top;
  a.tpr = move_tpr(cols);
  const int per = kMoveThreads / a.tpr;
  return cuda_status(launch_pdl(NVFP4_MOVE_KERNEL(combine_kernel, top),
                                (unsigned)((tokens + per - 1) / per), kMoveThreads, 0, stream, a));
}

nvfp4_status combine_bwd_impl(const void* dy, const void* o, const int32_t* row,
                              const int32_t* source, const float* weight, int64_t tokens,
                              int64_t cols, int32_t top, int64_t rows, void* d_o, float* dweight,
                              cudaStream_t stream) {
  if (!dy || !o || !row || !source || !weight || !d_o || !dweight) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = check_move(tokens, cols, top, rows);
  if (st != NVFP4_OK) return st;
  if (!a16(dy) || !a16(o) || !a16(d_o) || !a4(row) || !a4(source) || !a4(weight) || !a4(dweight))
    return NVFP4_ERR_ALIGN;
  DeviceInfo dev;
  st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  MoveArgs a = {};
  a.in = static_cast<const uint16_t*>(dy);
  a.rows_in = static_cast<const uint16_t*>(o);
  a.row = row;
  a.source = source;
  a.weight = weight;
  a.out = static_cast<uint16_t*>(d_o);
  a.dweight = dweight;
  a.tokens = tokens;
  a.rows = rows;
  a.cols = (int)cols;
  a.top = top;
  a.tpr = move_tpr(cols);
  const int per = kMoveThreads / a.tpr;
  a.clear_ctas = clear_ctas(rows);
  const unsigned token_ctas = (unsigned)((tokens + per - 1) / per);
  return cuda_status(launch_pdl(NVFP4_MOVE_KERNEL(combine_bwd_kernel, top),
                                a.clear_ctas + token_ctas, kMoveThreads, 0, stream, a));
}

}  // namespace nvfp4
