// Single values of the orthogonalisation and the Muon step: reading what is
// orthogonalised, writing the result.
#pragma once

#include "muon.cuh"

namespace dc {
namespace {

// Eight consecutive values of either type.
__device__ __forceinline__ void load8(const void* p, dc_dtype dt, long long i, float* v) {
  if (dt == DC_BF16) {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(k & 1 ? w[k >> 1] & 0xffff0000u : w[k >> 1] << 16);
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
__device__ __forceinline__ float load_in(const void* p, dc_dtype dt, long long i) {
  return dt == DC_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Whether the step is skipped: its scale is not finite.
__device__ __forceinline__ bool skipped(const MuonGroup& g, float* scale) {
  *scale = g.update && g.grad_scale ? *g.grad_scale : 1.f;
  return !(fabsf(*scale) <= 3.402823466e38f);
}

// What is orthogonalised of an input value and, in a step, its updated m.
__device__ __forceinline__ float direction(const MuonGroup& g, float scale, float v, float m) {
  if (!g.update) return v;
  return g.nesterov ? m * g.momentum + v * scale * g.rest : m;
}

// One value of the result: out, or taken off its parameter's old value p.
__device__ __forceinline__ void write_one(const MuonGroup& g, const MuonMat& t, float lr, long long i, float p, float v) {
  const bool bf16 = t.out_dtype == DC_BF16;
  void* out = t.out;
  if (g.update) {
    v = p * (1.f - lr * t.weight_decay) - v * (lr * t.rate);
    if (t.master) t.master[i] = v;
    out = t.param;
  }
  if (bf16)
    static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(out)[i] = v;
}

}  // namespace
}  // namespace dc
