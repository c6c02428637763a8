// route.cu -- routing of a mixture of experts: the choice of each token's k
// experts and their weights, the plan that orders the chosen rows by expert,
// and the rows' way to the experts (dispatch) and back (combine), with the
// gradients.
//
// Choice: the k largest logits of a row, the largest first, the lowest index
// among equals; compared on the bit patterns (mapped so that unsigned order is
// the floats' order), so the choice is exact.  -inf and NaN are never chosen.
// One warp takes a token: lane l holds logits l, l + 32, ..; each of the k
// rounds is a local maximum and two warp reductions (redux).
//
// Plan: expert e owns rows offsets[e] .. offsets[e] + sizes[e] - 1, in the
// order of (token, slot), and the offsets are multiples of 128, the rows of a
// scale atom.  Each CTA counts its tokens' choices per expert; the second
// kernel sums the counts of the CTAs before it (at most one CTA per SM, so
// this is a short read from L2) and ranks its own choices warp by warp.  No
// atomic decides an order: the plan is the same every time.  Few tokens take
// one CTA and one launch for both steps.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxExperts = 512;
constexpr int kMaxTop = 16;
constexpr int kGroupAlign = 128;
constexpr int kSmallTokens = 128;  // up to here one CTA does it all

struct RouteArgs {
  const void* logits;
  int64_t ld;
  int tokens, experts, top;
  int mode;
  int per_cta, per_warp;  // tokens of a CTA, of a warp
  int32_t* expert;
  float* weight;
  int32_t* sizes;
  int32_t* offsets;
  int32_t* row;
  int32_t* source;
  int64_t rows;     // entries of source
  int32_t* counts;  // [CTAs][experts]
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
// equal, and +inf counts as the largest finite value.
NVFP4_DEV uint32_t logit_key(float& v) {
  if (!(v > -INFINITY)) {
    v = -INFINITY;
    return 0u;
  }
  v = fminf(v, 3.402823466e38f) + 0.0f;
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

NVFP4_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The logits of one token in a warp's registers: value and key of experts
// lane + 32 i.
template <int NI, bool WIDE>
NVFP4_DEV void load_token(const RouteArgs& a, int64_t t, int lane, float (&v)[NI],
                          uint32_t (&key)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < a.experts ? load_logit<WIDE>(a.logits, t * a.ld + e) : -INFINITY;
    key[i] = logit_key(v[i]);
  }
}

// Step 1 for the tokens of this CTA: experts and weights to global memory,
// the count of each expert to `hist` (shared).
template <int NI, bool WIDE>
NVFP4_DEV void choose(const RouteArgs& a, int* hist) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < a.experts; e += kThreads) hist[e] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * a.per_cta + warp * a.per_warp;
  const int t1 = min(min(t0 + a.per_warp, (int)(blockIdx.x + 1) * a.per_cta), a.tokens);
  for (int t = t0; t < t1; ++t) {
    float v[NI];
    uint32_t key[NI];
    load_token<NI, WIDE>(a, t, lane, v, key);
    float top_logit = 0.0f, my_logit = 0.0f, all = 0.0f;
    int my_expert = -1;
    for (int j = 0; j < a.top; ++j) {
      uint32_t best = 0u;
      int at = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (key[i] > best) best = key[i], at = i;
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
      if (m == 0u) break;  // nothing left to choose
      const int e = __reduce_min_sync(0xFFFFFFFFu, best == m ? lane + 32 * at : kMaxExperts);
      const float l = __uint_as_float((m & 0x80000000u) ? (m & 0x7FFFFFFFu) : ~m);
      if (j == 0) {
        top_logit = l;
#pragma unroll
        for (int i = 0; i < NI; ++i) all += expf(v[i] - l);  // -inf adds 0
      }
      if (lane == j) my_expert = e, my_logit = l;
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (e == lane + 32 * i) key[i] = 0u;
    }
    const float ex = my_expert >= 0 ? expf(my_logit - top_logit) : 0.0f;
    const float total = warp_sum(a.mode == NVFP4_ROUTE_CHOSEN ? ex : all);
    if (lane < a.top) {
      const int64_t at = (int64_t)t * a.top + lane;
      a.expert[at] = my_expert;
      a.weight[at] = my_expert >= 0 ? ex / total : 0.0f;
      if (my_expert >= 0) atomicAdd(&hist[my_expert], 1);
    }
  }
  __syncthreads();
}

// Step 2: rows of this CTA's choices.  before[e]: choices of e in the CTAs
// before this one; total[e]: in all.  Both in shared memory; base [kWarps]
// [experts] is scratch.
NVFP4_DEV void assign(const RouteArgs& a, const int* before, const int* total, int* offset,
                      int* base) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    if (lane == 0) {
      offset[a.experts] = run;
      if (blockIdx.x == 0) a.offsets[a.experts] = run;
    }
  }
  for (int i = threadIdx.x; i < kWarps * a.experts; i += kThreads) base[i] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * a.per_cta + warp * a.per_warp;
  const int t1 = min(min(t0 + a.per_warp, (int)(blockIdx.x + 1) * a.per_cta), a.tokens);
  int* mine = base + warp * a.experts;
  const int64_t i0 = (int64_t)t0 * a.top, i1 = (int64_t)max(t1, t0) * a.top;
  for (int64_t i = i0 + lane; i < i1; i += 32) {
    const int e = a.expert[i];
    if (e >= 0) atomicAdd(&mine[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kThreads) {
    int run = offset[e] + before[e];
    for (int w = 0; w < kWarps; ++w) {
      const int n = base[w * a.experts + e];
      base[w * a.experts + e] = run;
      run += n;
    }
  }
  __syncthreads();
  // a token's experts differ, so its slots take their places side by side;
  // the warp's tokens follow one another
  for (int t = t0; t < t1; ++t) {
    if (lane < a.top) {
      const int64_t i = (int64_t)t * a.top + lane;
      const int e = a.expert[i];
      int r = -1;
      if (e >= 0) {
        r = mine[e]++;
        if (r < a.rows) a.source[r] = (int32_t)i;
      }
      a.row[i] = r;
    }
    __syncwarp();
  }
  // rows that no choice takes: each expert's padding, and what is behind the last
  for (int e = blockIdx.x; e < a.experts; e += gridDim.x)
    for (int r = offset[e] + total[e] + (int)threadIdx.x; r < offset[e + 1]; r += kThreads)
      if (r < a.rows) a.source[r] = -1;
  for (int64_t r = (int64_t)offset[a.experts] + (int64_t)blockIdx.x * kThreads + threadIdx.x;
       r < a.rows; r += (int64_t)gridDim.x * kThreads)
    a.source[r] = -1;
}

template <int NI, bool WIDE>
__global__ void __launch_bounds__(kThreads) route_choose_kernel(const RouteArgs a) {
  __shared__ int hist[kMaxExperts];
  griddep_wait();
  choose<NI, WIDE>(a, hist);
  for (int e = threadIdx.x; e < a.experts; e += kThreads)
    a.counts[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

struct AssignSmem {
  int before[kMaxExperts], total[kMaxExperts], offset[kMaxExperts + 1];
  int base[kWarps * kMaxExperts];
};

__global__ void __launch_bounds__(kThreads) route_assign_kernel(const RouteArgs a) {
  __shared__ AssignSmem s;
  griddep_wait();
  for (int e = threadIdx.x; e < a.experts; e += kThreads) {
    int before = 0, total = 0;
#pragma unroll 8
    for (int b = 0; b < (int)gridDim.x; ++b) {
      const int n = a.counts[(int64_t)b * a.experts + e];
      total += n;
      if (b < (int)blockIdx.x) before += n;
    }
    s.before[e] = before;
    s.total[e] = total;
  }
  __syncthreads();
  assign(a, s.before, s.total, s.offset, s.base);
}

template <int NI, bool WIDE>
__global__ void __launch_bounds__(kThreads) route_small_kernel(const RouteArgs a) {
  __shared__ AssignSmem s;
  griddep_wait();
  choose<NI, WIDE>(a, s.total);
  for (int e = threadIdx.x; e < a.experts; e += kThreads) s.before[e] = 0;
  __syncthreads();
  assign(a, s.before, s.total, s.offset, s.base);
}

// dl_i = w_i sum_j w_j (dw_i - dw_j) over the chosen (i, j); with the softmax
// over all experts the unchosen, whose weights have no gradient, add their
// share of probability times dw_i, and themselves get -p sum_j w_j dw_j.  The
// differences keep the result exact where one weight is near 1.
template <int NI, bool WIDE>
__global__ void __launch_bounds__(kThreads) route_bwd_kernel(const RouteArgs a) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
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
  float apart = 0.0f, mean = 0.0f;
  for (int j = 0; j < a.top; ++j) {
    const float wj = __shfl_sync(0xFFFFFFFFu, w, j), dj = __shfl_sync(0xFFFFFFFFu, dw, j);
    apart += wj * (dw - dj);
    mean += wj * dj;
  }
  float p[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) p[i] = 0.0f;
  if (a.mode == NVFP4_ROUTE_ALL) {
    uint32_t key[NI], best = 0u;
    load_token<NI, WIDE>(a, t, lane, p, key);
#pragma unroll
    for (int i = 0; i < NI; ++i) best = max(best, key[i]);
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
    const float l = __uint_as_float((m & 0x80000000u) ? (m & 0x7FFFFFFFu) : ~m);
    float all = 0.0f, rest = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      p[i] = key[i] ? expf(p[i] - l) : 0.0f;
      all += p[i];
    }
    all = warp_sum(all);
    const float inv = all > 0.0f ? 1.0f / all : 0.0f;
    for (int j = 0; j < a.top; ++j) {
      const int ej = __shfl_sync(0xFFFFFFFFu, e, j);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (ej == lane + 32 * i) p[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      p[i] *= inv;
      rest += p[i];
      p[i] *= -mean;
    }
    apart += warp_sum(rest) * dw;
  }
  const float mine = w * apart;
  for (int j = 0; j < a.top; ++j) {
    const int ej = __shfl_sync(0xFFFFFFFFu, e, j);
    const float dj = __shfl_sync(0xFFFFFFFFu, mine, j);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (ej == lane + 32 * i) p[i] = dj;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = lane + 32 * i;
    if (c < a.experts) {
      if (WIDE)
        static_cast<float*>(a.dlogits)[t * a.experts + c] = p[i];
      else
        static_cast<__nv_bfloat16*>(a.dlogits)[t * a.experts + c] = __float2bfloat16_rn(p[i]);
    }
  }
}

// ---- rows to the experts and back ------------------------------------------------
// A token (or row) is taken by `tpr` threads of a 256-thread CTA, a power of
// two from 32 on, each 8 columns at a time.
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
  unsigned token_ctas;  // CTAs behind these clear padding rows
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

// The rows of `out` without a source become zero.
NVFP4_DEV void clear_padding(const MoveArgs& a) {
  const int per = kMoveThreads / a.tpr, sub = threadIdx.x / a.tpr, tid = threadIdx.x % a.tpr;
  const int64_t r = (int64_t)(blockIdx.x - a.token_ctas) * per + sub;
  if (r >= a.rows || a.source[r] >= 0) return;
  for (int c = tid * 8; c < a.cols; c += a.tpr * 8)
    *reinterpret_cast<uint4*>(a.out + r * a.cols + c) = make_uint4(0u, 0u, 0u, 0u);
}

// The row of slot j of token t, or -1 (none, or not a row of the tensor).
NVFP4_DEV int64_t slot_row(const MoveArgs& a, int64_t t, int j) {
  const int r = a.row[t * a.top + j];
  return (uint32_t)r < (uint64_t)a.rows ? r : -1;
}

__global__ void __launch_bounds__(kMoveThreads) dispatch_kernel(const MoveArgs a) {
  griddep_wait();
  if (blockIdx.x >= a.token_ctas) return clear_padding(a);
  const int per = kMoveThreads / a.tpr, sub = threadIdx.x / a.tpr, tid = threadIdx.x % a.tpr;
  const int64_t t = (int64_t)blockIdx.x * per + sub;
  if (t >= a.tokens) return;
  for (int c = tid * 8; c < a.cols; c += a.tpr * 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(a.in + t * a.cols + c);
    for (int j = 0; j < a.top; ++j) {
      const int64_t r = slot_row(a, t, j);
      if (r >= 0) *reinterpret_cast<uint4*>(a.out + r * a.cols + c) = v;
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) combine_kernel(const MoveArgs a) {
  griddep_wait();
  const int per = kMoveThreads / a.tpr, sub = threadIdx.x / a.tpr, tid = threadIdx.x % a.tpr;
  const int64_t t = (int64_t)blockIdx.x * per + sub;
  if (t >= a.tokens) return;
  for (int c = tid * 8; c < a.cols; c += a.tpr * 8) {
    float s[8] = {};
#pragma unroll 4
    for (int j = 0; j < a.top; ++j) {
      const int64_t r = slot_row(a, t, j);
      if (r < 0) continue;
      const float w = a.weight ? a.weight[t * a.top + j] : 1.0f;
      float v[8];
      unpack8(*reinterpret_cast<const uint4*>(a.in + r * a.cols + c), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = fmaf(w, v[e], s[e]);
    }
    *reinterpret_cast<uint4*>(a.out + t * a.cols + c) = pack8(s);
  }
}

// do[row] = w dy, dw = <dy, o[row]>: dy is read once for all of a token's
// slots, whose products each thread carries in registers.
template <int TOP>
__global__ void __launch_bounds__(kMoveThreads) combine_bwd_kernel(const MoveArgs a) {
  __shared__ float red[kMoveThreads / 32][TOP];
  griddep_wait();
  if (blockIdx.x >= a.token_ctas) return clear_padding(a);
  const int per = kMoveThreads / a.tpr, sub = threadIdx.x / a.tpr, tid = threadIdx.x % a.tpr;
  const int64_t t = (int64_t)blockIdx.x * per + sub;
  const bool live = t < a.tokens;
  float dot[TOP] = {};
  if (live) {
    for (int c = tid * 8; c < a.cols; c += a.tpr * 8) {
      float d[8];
      unpack8(*reinterpret_cast<const uint4*>(a.in + t * a.cols + c), d);
#pragma unroll
      for (int j = 0; j < TOP; ++j) {
        if (j >= a.top) break;
        const int64_t r = slot_row(a, t, j);
        if (r < 0) continue;
        const float w = a.weight[t * a.top + j];
        float v[8];
        unpack8(*reinterpret_cast<const uint4*>(a.rows_in + r * a.cols + c), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dot[j] = fmaf(d[e], v[e], dot[j]);
          v[e] = w * d[e];
        }
        *reinterpret_cast<uint4*>(a.out + r * a.cols + c) = pack8(v);
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
    for (int w = 0; w < a.tpr / 32; ++w) s += red[sub * (a.tpr / 32) + w][tid];
    a.dweight[t * a.top + tid] = s;  // 0 for a slot without a row
  }
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool a4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// CTAs of the two routing kernels: at most one per SM (the second reads every
// CTA's counts), at least 16 tokens each.
int route_ctas(int64_t tokens, int sms) {
  if (tokens <= kSmallTokens) return 1;
  return (int)std::min<int64_t>(std::min(sms, kMaxSms), (tokens + kWarps - 1) / kWarps);
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
  if (ctas == 1) return launch_pdl(route_small_kernel<NI, WIDE>, 1, kThreads, 0, stream, a);
  const cudaError_t e = launch_pdl(route_choose_kernel<NI, WIDE>, ctas, kThreads, 0, stream, a);
  if (e != cudaSuccess) return e;
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

// Threads per row: the power of two next to the row's vectors.
int move_tpr(int64_t cols) {
  int tpr = 32;
  while (tpr < kMoveThreads && tpr * 8 < cols) tpr *= 2;
  return tpr;
}

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
  if (workspace_bytes) *workspace_bytes = (size_t)kMaxSms * experts * sizeof(int32_t);
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
      workspace_bytes < (size_t)kMaxSms * experts * sizeof(int32_t))
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
  a.per_warp = (a.per_cta + kWarps - 1) / kWarps;
  ctas = (int)((tokens + a.per_cta - 1) / a.per_cta);
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
  a.token_ctas = (unsigned)((tokens + per - 1) / per);
  const unsigned grid = a.token_ctas + (unsigned)((rows + per - 1) / per);
  return cuda_status(launch_pdl(dispatch_kernel, grid, kMoveThreads, 0, stream, a));
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
  a.token_ctas = (unsigned)((tokens + per - 1) / per);
  return cuda_status(launch_pdl(combine_kernel, a.token_ctas, kMoveThreads, 0, stream, a));
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
  a.token_ctas = (unsigned)((tokens + per - 1) / per);
  const unsigned grid = a.token_ctas + (unsigned)((rows + per - 1) / per);
  auto kern = top <= 1   ? combine_bwd_kernel<1>
              : top <= 2 ? combine_bwd_kernel<2>
              : top <= 4 ? combine_bwd_kernel<4>
              : top <= 8 ? combine_bwd_kernel<8>
                         : combine_bwd_kernel<16>;
  return cuda_status(launch_pdl(kern, grid, kMoveThreads, 0, stream, a));
}

}  // namespace nvfp4
