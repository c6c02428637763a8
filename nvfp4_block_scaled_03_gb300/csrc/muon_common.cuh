// muon_common.cuh -- what the kernels of the orthogonalised momentum share: the
// scale of the f16 operands, descriptors and the f16 tcgen05 instruction.
#pragma once

#include <cuda_fp16.h>

#include "gemm_common.cuh"

namespace nvfp4 {

// A call of nvfp4_muon_update behind its checks.
struct MuonCall {
  const nvfp4_muon_params* p;
  void* grad;
  float* momentum;
  __nv_bfloat16* update;
  bool wide, zero;
  void* workspace;
  int sms;
  cudaStream_t stream;
};

// The kernel that keeps matrices of at most 128 rows or columns on chip
// (muon_panel.cu): whether it takes these sizes, its workspace, the call.
bool muon_panel_fits(int64_t rows, int64_t cols);
size_t muon_panel_workspace(int64_t rows, int64_t cols);
nvfp4_status muon_panel(const MuonCall& c);
nvfp4_status muon_panel_read_error(unsigned int* code);
nvfp4_status muon_panel_set_injection(unsigned int stall, unsigned long long wait_ns);

namespace {

constexpr float kScale = 4096.0f, kUnscale = 1.0f / 4096.0f;

// What U is multiplied by to give X with the operands' scale.  Squares in FP32 lose a norm
// below 1e-18, which counts as that: U's entries are smaller then, X's at most about 1, and
// the factor is finite for any eps.
NVFP4_DEV float start_scale(float squares, float eps) {
  return kScale / fmaxf(fmaxf(sqrtf(squares), eps), 1e-18f);
}

// MN-major operand tile: rows of 128 bytes (64 along M or N) for each k with the
// 128-byte swizzle, 8 rows (1024 bytes) a swizzle atom; the next 64 of M or N lie
// `next` bytes further.
NVFP4_DEV uint64_t smem_desc_mn(uint32_t saddr, uint32_t next) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(next >> 4) << 16;  // leading byte offset: the next 64 of M or N
  d |= (uint64_t)(1024 >> 4) << 32;  // stride byte offset: the next 8 of K
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;            // SWIZZLE_128B
  return d;
}

// Instruction descriptor for kind::f16: f16 A and B, FP32 accumulators.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

NVFP4_DEV uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
NVFP4_DEV float2 unpack_f16x2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool WIDE>
NVFP4_DEV float grad_at(const void* g, int64_t i) {
  if (WIDE) return static_cast<const float*>(g)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(g)[i] << 16);
}
template <bool WIDE>
NVFP4_DEV float4 grad4_at(const void* g, int64_t i) {
  if (WIDE) return *reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g) + i);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}

inline size_t up1k(size_t v) { return (v + 1023) / 1024 * 1024; }

}  // namespace
}  // namespace nvfp4
