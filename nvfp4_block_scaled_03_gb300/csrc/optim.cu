// optim.cu -- the optimizer step of an FP32 master weight, fused with the
// amax its next NVFP4 quantisation needs.
//
// "NVFP4 pretraining recipe" page, Figure 1 text: the MLP GEMMs' BF16
// outputs end up folded into FP32 master weights on the optimizer step, and
// each step quantises the weights 16x16 under a per-tensor FP32 scale, which
// is computed from the tensor's amax.  Taking that amax while the update
// writes the weight removes the quantiser's own amax pass (one full read of
// the FP32 weight per step).  The pages name no optimizer; the update is
// plain SGD, elementwise in binary32 with the product rounded first:
//   W[i] <- W[i] - lr * G[i]
//   G[i] <- 0                  (NVFP4_ZERO_GRAD: ready for the next fold)
//   amax  = max_i |W[i]|       over the values written
// Work: persistent grid-stride over 16-byte chunks, four chunks of W and of
// G in flight per thread; one partial maximum per CTA, reduced by a second
// one-CTA launch (deterministic: a maximum does not depend on the order).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

NVFP4_DEV float sgd1(float w, float g, float lr) { return __fsub_rn(w, __fmul_rn(lr, g)); }

template <bool ZERO, bool AMAX>
__global__ void __launch_bounds__(kThreads) sgd_amax_kernel(float* __restrict__ W,
                                                            float* __restrict__ G, int64_t n4,
                                                            float lr, float* partials) {
  __shared__ float red[kThreads / 32];
  float4* w4 = reinterpret_cast<float4*>(W);
  float4* g4 = reinterpret_cast<float4*>(G);
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  float m = 0.0f;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n4; i += kUnroll * stride) {
    float4 w[kUnroll], g[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t q = i + u * stride;
      if (q < n4) {
        w[u] = w4[q];
        g[u] = g4[q];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t q = i + u * stride;
      if (q < n4) {
        const float4 r = make_float4(sgd1(w[u].x, g[u].x, lr), sgd1(w[u].y, g[u].y, lr),
                                     sgd1(w[u].z, g[u].z, lr), sgd1(w[u].w, g[u].w, lr));
        w4[q] = r;
        if (ZERO) g4[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (AMAX)
          m = fmaxf(m, fmaxf(fmaxf(fabsf(r.x), fabsf(r.y)), fmaxf(fabsf(r.z), fabsf(r.w))));
      }
    }
  }
  if (AMAX) {
    m = block_max(m, red);
    if (threadIdx.x == 0) partials[blockIdx.x] = m;
  }
}

__global__ void __launch_bounds__(kThreads) sgd_amax_finalize_kernel(const float* partials, int n,
                                                                     float* amax) {
  __shared__ float red[kThreads / 32];
  float m = 0.0f;
  for (int i = threadIdx.x; i < n; i += kThreads) m = fmaxf(m, partials[i]);
  m = block_max(m, red);
  if (threadIdx.x == 0) *amax = m;
}

// W = keep W - step update (bf16), four chunks of 4 elements a thread in flight, 512
// contiguous bytes of W a warp (14336 x 4096: 98 us, floor 86; chunks of 8 elements, with
// whole 16-byte loads of the update, 106); the elements behind the last chunk are the
// last CTA's.
NVFP4_DEV float apply1(float w, float u, float keep, float step) {
  return fmaf(-step, u, __fmul_rn(keep, w));
}

template <bool AMAX>
NVFP4_DEV float apply_share(float* __restrict__ W, const uint16_t* __restrict__ U, int64_t n,
                            float keep, float step) {
  constexpr int kChunks = 4;
  const int64_t n4 = n / 4, stride = (int64_t)gridDim.x * blockDim.x;
  float m = 0.0f;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n4; i += kChunks * stride) {
    float4 w[kChunks];
    uint2 u[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int64_t q = i + c * stride;
      if (q < n4) {
        w[c] = reinterpret_cast<const float4*>(W)[q];
        u[c] = reinterpret_cast<const uint2*>(U)[q];
      }
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int64_t q = i + c * stride;
      if (q >= n4) continue;
      const float4 v = w[c];
      const float4 r = make_float4(apply1(v.x, __uint_as_float(u[c].x << 16), keep, step),
                                   apply1(v.y, __uint_as_float(u[c].x & 0xFFFF0000u), keep, step),
                                   apply1(v.z, __uint_as_float(u[c].y << 16), keep, step),
                                   apply1(v.w, __uint_as_float(u[c].y & 0xFFFF0000u), keep, step));
      reinterpret_cast<float4*>(W)[q] = r;
      if (AMAX) m = fmaxf(m, fmaxf(fmaxf(fabsf(r.x), fabsf(r.y)), fmaxf(fabsf(r.z), fabsf(r.w))));
    }
  }
  const int64_t t = n4 * 4 + threadIdx.x;
  if (blockIdx.x == gridDim.x - 1 && t < n) {
    const float r = apply1(W[t], __uint_as_float((uint32_t)U[t] << 16), keep, step);
    W[t] = r;
    if (AMAX) m = fmaxf(m, fabsf(r));
  }
  return m;
}

template <bool AMAX>
__global__ void __launch_bounds__(kThreads) muon_apply_kernel(float* __restrict__ W,
                                                              const uint16_t* __restrict__ U,
                                                              int64_t n, float keep, float step,
                                                              float* partials) {
  __shared__ float red[kThreads / 32];
  float m = apply_share<AMAX>(W, U, n, keep, step);
  if (AMAX) {
    m = block_max(m, red);
    if (threadIdx.x == 0) partials[blockIdx.x] = m;
  }
}

// A small weight's step on one cluster, whose first CTA gathers the others' maxima: one
// launch instead of two.
constexpr int kClusterCtas = 16, kClusterThreads = 1024;
__global__ void __launch_bounds__(kClusterThreads)
    muon_apply_small_kernel(float* __restrict__ W, const uint16_t* __restrict__ U, int64_t n,
                            float keep, float step, float* amax) {
  __shared__ float red[kClusterThreads / 32];
  __shared__ float maxima[kClusterCtas];
  // another CTA's shared memory is only there once that CTA runs: this one says so here
  // and looks for the others under the loads' time, before it stores
  cluster_arrive();
  const float m = block_max(apply_share<true>(W, U, n, keep, step), red);
  __syncwarp();
  cluster_wait();
  if (threadIdx.x == 0)
    st_cluster_u32(mapa_shared(smem_u32(&maxima[cluster_ctarank()]), 0), __float_as_uint(m));
  __syncwarp();
  cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    float most = maxima[0];
    for (int c = 1; c < (int)gridDim.x; ++c) most = fmaxf(most, maxima[c]);
    *amax = most;
  }
}
// Measured (us, one launch on a cluster and two on all SMs): calls one behind another 7.7
// and 10.0 for 4096 to 2^18 elements, 8.2 and 10.0 for 2^19; a call waited for 17.5 and
// 19.5, at 2^18 19.0 and 19.8, at 2^19 20.7 and 19.9.  In a replayed graph, where a launch
// costs less, the two are the quicker from 4096 on: 3.3 and 3.1, at 2^18 4.4 and 3.4.
constexpr int64_t kClusterElements = 1 << 18;

// Launches it; false: the device has no room for such a cluster.
bool launch_small(float* W, const uint16_t* U, int64_t n, float keep, float step, float* amax,
                  cudaStream_t s, cudaError_t* err) {
  static std::atomic<int> fits[64];  // 1: yes, -1: no
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kClusterCtas);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kClusterCtas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int known = fits[dev].load(std::memory_order_relaxed);
  if (known == 0) {
    int count = 0;
    known = cudaFuncSetAttribute(muon_apply_small_kernel,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&count, muon_apply_small_kernel, &cfg) ==
                        cudaSuccess &&
                    count > 0
                ? 1
                : -1;
    if (known < 0) cudaGetLastError();
    fits[dev].store(known, std::memory_order_relaxed);
  }
  if (known < 0) return false;
  *err = cudaLaunchKernelEx(&cfg, muon_apply_small_kernel, W, U, n, keep, step, amax);
  return true;
}

// CTAs of a persistent launch: as many as are resident at once (looked up
// once per kernel and device), at most one partial slot each, at most one
// per kThreads chunks.
template <auto KERN>
int sgd_grid(int64_t n4, int sms) {
  static std::atomic<int> fit[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  int per_sm = fit[dev].load(std::memory_order_relaxed);
  if (per_sm == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERN, kThreads, 0) !=
            cudaSuccess ||
        per_sm < 1)
      per_sm = 1;
    fit[dev].store(per_sm, std::memory_order_relaxed);
  }
  const int64_t want = std::max<int64_t>(1, (n4 + kThreads - 1) / kThreads);
  return (int)std::min<int64_t>(std::min<int64_t>(want, (int64_t)sms * per_sm), kMaxPartials);
}

template <bool ZERO, bool AMAX>
nvfp4_status launch_sgd(float* W, float* G, int64_t n4, float lr, float* partials, int sms,
                        int* grid, cudaStream_t s) {
  auto kern = sgd_amax_kernel<ZERO, AMAX>;
  *grid = sgd_grid<sgd_amax_kernel<ZERO, AMAX>>(n4, sms);
  kern<<<*grid, kThreads, 0, s>>>(W, G, n4, lr, partials);
  return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_sgd_step(float* W, float* G, int64_t n, float lr, uint32_t flags,
                                       float* amax, void* workspace, size_t workspace_bytes,
                                       nvfp4_stream stream) {
  if (!W || !G || (flags & ~(uint32_t)NVFP4_ZERO_GRAD) || !std::isfinite(lr))
    return NVFP4_ERR_INVALID_ARG;
  if (n <= 0 || n % 4) return NVFP4_ERR_SHAPE;
  const uintptr_t wb = reinterpret_cast<uintptr_t>(W), gb = reinterpret_cast<uintptr_t>(G);
  const uintptr_t bytes = (uintptr_t)n * sizeof(float);
  if (wb < gb + bytes && gb < wb + bytes) return NVFP4_ERR_INVALID_ARG;  // overlap
  if (!a16(W) || !a16(G) || (reinterpret_cast<uintptr_t>(amax) & 3u)) return NVFP4_ERR_ALIGN;
  if (amax && (!workspace || workspace_bytes < kQuantWorkspaceBytes || !a16(workspace)))
    return NVFP4_ERR_WORKSPACE;
  DeviceInfo dev;
  nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* partials = static_cast<float*>(workspace);
  const int64_t n4 = n / 4;
  const bool zero = flags & NVFP4_ZERO_GRAD;
  int grid = 0;
  if (amax) {
    st = zero ? launch_sgd<true, true>(W, G, n4, lr, partials, dev.sm_count, &grid, s)
              : launch_sgd<false, true>(W, G, n4, lr, partials, dev.sm_count, &grid, s);
    if (st != NVFP4_OK) return st;
    sgd_amax_finalize_kernel<<<1, kThreads, 0, s>>>(partials, grid, amax);
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
  }
  return zero ? launch_sgd<true, false>(W, G, n4, lr, nullptr, dev.sm_count, &grid, s)
              : launch_sgd<false, false>(W, G, n4, lr, nullptr, dev.sm_count, &grid, s);
}

extern "C" nvfp4_status nvfp4_muon_apply(float* W, const void* update, int64_t n, float lr,
                                         float scale, float decay, float* amax, void* workspace,
                                         size_t workspace_bytes, nvfp4_stream stream) {
  if (!W || !update || !std::isfinite(lr) || !std::isfinite(scale) || !std::isfinite(decay))
    return NVFP4_ERR_INVALID_ARG;
  if (n <= 0 || n > INT64_MAX / 16) return NVFP4_ERR_SHAPE;
  const uintptr_t wb = reinterpret_cast<uintptr_t>(W), ub = reinterpret_cast<uintptr_t>(update);
  if (wb < ub + (uintptr_t)n * 2 && ub < wb + (uintptr_t)n * 4) return NVFP4_ERR_INVALID_ARG;
  if (!a16(W) || !a16(update) || (reinterpret_cast<uintptr_t>(amax) & 3u)) return NVFP4_ERR_ALIGN;
  if (amax && (!workspace || workspace_bytes < kQuantWorkspaceBytes || !a16(workspace)))
    return NVFP4_ERR_WORKSPACE;
  DeviceInfo dev;
  const nvfp4_status st = current_device(&dev);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const float keep = (float)(1.0 - (double)lr * decay), step = (float)((double)lr * scale);
  const uint16_t* u = static_cast<const uint16_t*>(update);
  if (!amax) {
    const int grid = sgd_grid<muon_apply_kernel<false>>(n / 4, dev.sm_count);
    muon_apply_kernel<false><<<grid, kThreads, 0, s>>>(W, u, n, keep, step, nullptr);
    return cuda_status(cudaGetLastError());
  }
  cudaError_t err;
  if (n <= kClusterElements && launch_small(W, u, n, keep, step, amax, s, &err))
    return cuda_status(err);
  float* partials = static_cast<float*>(workspace);
  const int grid = sgd_grid<muon_apply_kernel<true>>(n / 4, dev.sm_count);
  muon_apply_kernel<true><<<grid, kThreads, 0, s>>>(W, u, n, keep, step, partials);
  if (cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
  sgd_amax_finalize_kernel<<<1, kThreads, 0, s>>>(partials, grid, amax);
  return cuda_status(cudaGetLastError());
}
