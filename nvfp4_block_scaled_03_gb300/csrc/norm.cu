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
// All arithmetic is FP32; x, y, dx, dy are bf16 or FP32, z, h, dz, dh bf16,
// each rounded once.  The kernels move 2 (x, y) + 2 (z, h) or 3 + 3 streams
// and are bound by memory.  The column sums go to per-CTA partials that a
// second kernel adds in a fixed order: no atomics, so results repeat bit for
// bit.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kVec = 8;            // columns a thread takes at a time
constexpr int kMaxThreads = 512;
constexpr int kMaxVpt = 16;        // 512 threads x 16 x 8 = 65536 columns

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
  // backward
  const void* dy;
  const uint16_t* dh;
  void* dx;
  uint16_t* dz;
  float* drow;      // row gate: its gradient [rows]
  float* partials;  // [grid][2][cols]: S or dw_post, then dw_pre
};

NVFP4_DEV void from_bf16(const uint4 u, float (&v)[kVec]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
NVFP4_DEV void store_bf16(uint16_t* p, const float (&v)[kVec]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
NVFP4_DEV void load_f32(const float* p, float (&v)[kVec]) {
  const float4 lo = *reinterpret_cast<const float4*>(p);
  const float4 hi = *reinterpret_cast<const float4*>(p + 4);
  v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
  v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
}
NVFP4_DEV void store_f32(float* p, const float (&v)[kVec]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Eight columns of the residual stream, kept as loaded.
template <bool WIDE>
struct Stream8;
template <>
struct Stream8<false> {
  uint4 raw = make_uint4(0u, 0u, 0u, 0u);
  NVFP4_DEV void load(const void* p, int64_t at) {
    raw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  }
  NVFP4_DEV void get(float (&v)[kVec]) const { from_bf16(raw, v); }
  NVFP4_DEV static void store(void* p, int64_t at, const float (&v)[kVec]) {
    store_bf16(static_cast<uint16_t*>(p) + at, v);
  }
};
template <>
struct Stream8<true> {
  float raw[kVec] = {};
  NVFP4_DEV void load(const void* p, int64_t at) {
    load_f32(static_cast<const float*>(p) + at, raw);
  }
  NVFP4_DEV void get(float (&v)[kVec]) const {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = raw[e];
  }
  NVFP4_DEV static void store(void* p, int64_t at, const float (&v)[kVec]) {
    store_f32(static_cast<float*>(p) + at, v);
  }
};

// Sums of N values over the threads of the CTA (every thread gets them; the
// order is fixed).  The calls of a CTA alternate between two buffers, so one
// barrier a call suffices: a buffer is written again only after the next
// call's barrier, which every thread reaches after its reads.
struct Reducer {
  float buf[2][5 * 16];
};
template <int N>
NVFP4_DEV void block_sum(float (&v)[N], Reducer& r, int& turn) {
  float* red = r.buf[turn];
  turn ^= 1;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 16 + (threadIdx.x >> 5)] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += red[i * 16 + w];
    v[i] = s;
  }
}

NVFP4_DEV float rstd(float sum_sq, int cols, float eps) {
  return __frsqrt_rn(sum_sq / (float)cols + eps);
}

template <int VPT, bool WIDE>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_kernel(const NormArgs p) {
  __shared__ Reducer red;
  griddep_wait();
  const int tpr = blockDim.x;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at0 = row * p.cols;
    float y[VPT][kVec], n[VPT][kVec], s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * tpr + threadIdx.x) * kVec;
      if (c < p.cols) {
        Stream8<WIDE> x;
        x.load(p.x, at0 + c);
        x.get(y[i]);
        if (p.z) from_bf16(*reinterpret_cast<const uint4*>(p.z + at0 + c), n[i]);
      }
    }
    float rz = 0.0f;
    if (p.z) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if ((i * tpr + threadIdx.x) * kVec < p.cols)
#pragma unroll
          for (int e = 0; e < kVec; ++e) s[0] += n[i][e] * n[i][e];
      block_sum(s, red, turn);
      rz = rstd(s[0], p.cols, p.eps) * p.b;
      if (p.gate_mode == NVFP4_GATE_ROW) rz *= p.gate[row];
    }
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * tpr + threadIdx.x) * kVec;
      if (c < p.cols) {
        if (p.z) {
          float w[kVec];
          load_f32(p.w_post + c, w);
          if (p.gate_mode == NVFP4_GATE_CHANNEL) {
            float g[kVec];
            load_f32(p.gate + c, g);
#pragma unroll
            for (int e = 0; e < kVec; ++e) w[e] *= g[e];
          }
#pragma unroll
          for (int e = 0; e < kVec; ++e) y[i][e] = fmaf(p.a, y[i][e], n[i][e] * rz * w[e]);
        } else {
#pragma unroll
          for (int e = 0; e < kVec; ++e) y[i][e] *= p.a;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) s[0] += y[i][e] * y[i][e];
        if (p.y) Stream8<WIDE>::store(p.y, at0 + c, y[i]);
      }
    }
    if (p.h) {
      block_sum(s, red, turn);
      const float ry = rstd(s[0], p.cols, p.eps);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * tpr + threadIdx.x) * kVec;
        if (c < p.cols) {
          float w[kVec];
          load_f32(p.w_pre + c, w);
#pragma unroll
          for (int e = 0; e < kVec; ++e) w[e] *= y[i][e] * ry;
          store_bf16(p.h + at0 + c, w);
        }
      }
    }
  }
}

template <int VPT, bool WIDE>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormArgs p) {
  __shared__ Reducer red;
  griddep_wait();
  const int tpr = blockDim.x;
  int turn = 0;
  float acc_post[VPT][kVec] = {}, acc_pre[VPT][kVec] = {};
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int64_t at0 = row * p.cols;
    Stream8<WIDE> x[VPT], dy[VPT];
    uint4 z[VPT], dh[VPT];
    float s1[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      z[i] = dh[i] = make_uint4(0u, 0u, 0u, 0u);
      const int c = (i * tpr + threadIdx.x) * kVec;
      if (c < p.cols) {
        if (p.dh || p.z) x[i].load(p.x, at0 + c);
        if (p.dy) dy[i].load(p.dy, at0 + c);
        if (p.z) z[i] = *reinterpret_cast<const uint4*>(p.z + at0 + c);
        if (p.dh) dh[i] = *reinterpret_cast<const uint4*>(p.dh + at0 + c);
      }
    }
    float rz = 0.0f, g_row = 1.0f;
    if (p.z) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float v[kVec];
        from_bf16(z[i], v);
#pragma unroll
        for (int e = 0; e < kVec; ++e) s1[0] += v[e] * v[e];
      }
      block_sum(s1, red, turn);
      rz = rstd(s1[0], p.cols, p.eps);
      if (p.gate_mode == NVFP4_GATE_ROW) g_row = p.gate[row];
    }
    // sums over the row: y^2, u y, and z^ c (c = w_post [g]) times dy, u, y
    float s[5] = {};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * tpr + threadIdx.x) * kVec;
      if (c < p.cols) {
        float xv[kVec], zv[kVec], dyv[kVec], dhv[kVec], cw[kVec] = {}, wp[kVec] = {};
        x[i].get(xv);
        dy[i].get(dyv);
        from_bf16(z[i], zv);
        from_bf16(dh[i], dhv);
        if (p.z) {
          load_f32(p.w_post + c, cw);
          if (p.gate_mode == NVFP4_GATE_CHANNEL) {
            float g[kVec];
            load_f32(p.gate + c, g);
#pragma unroll
            for (int e = 0; e < kVec; ++e) cw[e] *= g[e];
          }
        }
        if (p.dh) load_f32(p.w_pre + c, wp);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float zc = zv[e] * rz * cw[e];
          const float yv = fmaf(p.a, xv[e], p.b * g_row * zc);
          const float u = dhv[e] * wp[e];
          s[0] += yv * yv;
          s[1] += u * yv;
          s[2] += zc * dyv[e];
          s[3] += zc * u;
          s[4] += zc * yv;
        }
      }
    }
    block_sum(s, red, turn);
    const float inv = 1.0f / (float)p.cols;
    float ry = 0.0f, m = 0.0f;  // m = r_y^2 mean(u y): dY = dy + r_y (u - y m)
    if (p.dh) {
      ry = rstd(s[0], p.cols, p.eps);
      m = ry * ry * s[1] * inv;
    }
    // sum over the row of dY z^ c
    const float t = s[2] + ry * (s[3] - m * s[4]);
    const float mz = p.b * g_row * t * inv;
    if (p.drow && threadIdx.x == 0) p.drow[row] = p.b * t;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * tpr + threadIdx.x) * kVec;
      if (c < p.cols) {
        float xv[kVec], zv[kVec], dyv[kVec], dhv[kVec], cw[kVec] = {}, wp[kVec] = {};
        x[i].get(xv);
        dy[i].get(dyv);
        from_bf16(z[i], zv);
        from_bf16(dh[i], dhv);
        if (p.z) {
          load_f32(p.w_post + c, cw);
          if (p.gate_mode == NVFP4_GATE_CHANNEL) {
            float g[kVec];
            load_f32(p.gate + c, g);
#pragma unroll
            for (int e = 0; e < kVec; ++e) cw[e] *= g[e];
          }
        }
        if (p.dh) load_f32(p.w_pre + c, wp);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float zh = zv[e] * rz;
          const float yv = fmaf(p.a, xv[e], p.b * g_row * (zh * cw[e]));
          const float u = dhv[e] * wp[e];
          const float d = dyv[e] + ry * (u - yv * m);
          const float q = p.b * g_row * d;
          acc_pre[i][e] += dhv[e] * (yv * ry);
          acc_post[i][e] += q * zh;
          dyv[e] = p.a * d;
          dhv[e] = rz * (q * cw[e] - zh * mz);
        }
        Stream8<WIDE>::store(p.dx, at0 + c, dyv);
        if (p.z) store_bf16(p.dz + at0 + c, dhv);
      }
    }
  }
  float* out = p.partials + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * tpr + threadIdx.x) * kVec;
    if (c < p.cols) {
      if (p.z) store_f32(out + c, acc_post[i]);
      if (p.dh) store_f32(out + p.cols + c, acc_pre[i]);
    }
  }
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

// Threads of a row's CTA and vectors a thread takes.
struct Shape {
  int threads, vpt;
};
Shape row_shape(int64_t cols) {
  const int64_t vecs = cols / kVec;
  int vpt = 1;
  while (vecs > (int64_t)kMaxThreads * vpt) vpt *= 2;
  const int64_t threads = (vecs + vpt - 1) / vpt;
  return {(int)((threads + 31) / 32 * 32), vpt};
}

// CTAs of `kern` that fit the device at once.
template <auto KERN>
int resident_ctas(int threads, int sms) {
  static std::atomic<int> fit[64][kMaxThreads / 32 + 1];  // one cache per kernel
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  std::atomic<int>& slot = fit[dev][threads / 32];
  int per_sm = slot.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERN, threads, 0) != cudaSuccess ||
        per_sm < 1)
      per_sm = 1;
    slot.store(per_sm, std::memory_order_relaxed);
  }
  return per_sm * sms;
}

template <int VPT, bool WIDE>
cudaError_t launch_fwd(const NormArgs& p, int threads, int sms, cudaStream_t stream) {
  constexpr auto kern = norm_fwd_kernel<VPT, WIDE>;
  const int grid = (int)std::min<int64_t>(p.rows, resident_ctas<kern>(threads, sms));
  return launch_pdl(kern, grid, threads, 0, stream, p);
}

// The backward's grid is capped so that the partials stay small.
constexpr int kBwdCtasPerSm = 2;

template <int VPT, bool WIDE>
cudaError_t launch_bwd(const NormArgs& p, int threads, int sms, cudaStream_t stream, int* grid) {
  constexpr auto kern = norm_bwd_kernel<VPT, WIDE>;
  *grid = (int)std::min<int64_t>(
      p.rows, std::min(resident_ctas<kern>(threads, sms), kBwdCtasPerSm * sms));
  return launch_pdl(kern, *grid, threads, 0, stream, p);
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
  return (size_t)std::min<int64_t>(rows, (int64_t)kBwdCtasPerSm * sms) * 2 * cols * sizeof(float);
}

}  // namespace

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
  const Shape s = row_shape(q->cols);
  const bool wide = q->stream_dtype == NVFP4_IN_FP32;
  const int sms = dev.sm_count;
#define NVFP4_NORM_FWD(V) \
  case V:                 \
    return cuda_status(wide ? launch_fwd<V, true>(p, s.threads, sms, stream) \
                            : launch_fwd<V, false>(p, s.threads, sms, stream));
  switch (s.vpt) {
    NVFP4_NORM_FWD(1)
    NVFP4_NORM_FWD(2)
    NVFP4_NORM_FWD(4)
    NVFP4_NORM_FWD(8)
    NVFP4_NORM_FWD(16)
  }
#undef NVFP4_NORM_FWD
  return NVFP4_ERR_SHAPE;
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
  const Shape s = row_shape(q->cols);
  const bool wide = q->stream_dtype == NVFP4_IN_FP32;
  int grid = 0;
  cudaError_t e = cudaErrorInvalidValue;
#define NVFP4_NORM_BWD(V)                                                   \
  case V:                                                                   \
    e = wide ? launch_bwd<V, true>(p, s.threads, sms, stream, &grid)        \
             : launch_bwd<V, false>(p, s.threads, sms, stream, &grid);      \
    break;
  switch (s.vpt) {
    NVFP4_NORM_BWD(1)
    NVFP4_NORM_BWD(2)
    NVFP4_NORM_BWD(4)
    NVFP4_NORM_BWD(8)
    NVFP4_NORM_BWD(16)
  }
#undef NVFP4_NORM_BWD
  if (e != cudaSuccess) return NVFP4_ERR_CUDA;
  const bool channel = q->gate_mode == NVFP4_GATE_CHANNEL;
  const int first = z ? 0 : 1, sums = (z ? 1 : 0) + (w_pre ? 1 : 0);
  // blockIdx.y 0 is the post sum, 1 the pre sum; without z only the latter
  const dim3 rgrid((unsigned)((q->cols + 31) / 32), (unsigned)(first + sums));
  return cuda_status(launch_pdl(norm_bwd_reduce_kernel, rgrid, dim3(256), 0, stream,
                                (const float*)p.partials, grid, (int)q->cols, w_post,
                                channel ? gate : (const float*)nullptr, dw_post,
                                channel ? dgate : (float*)nullptr, dw_pre));
}

}  // namespace nvfp4
