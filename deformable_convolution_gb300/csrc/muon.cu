// Orthogonalisation by Newton-Schulz products and the Muon step: the passes
// over single elements around the products.
#include "muon.cuh"
#include "muon_values.cuh"

namespace dc {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += part[w];
  return v;
}

__global__ void __launch_bounds__(kThreads) muon_squares(const __grid_constant__ MuonGroup g) {
  // Beside the launch of the small matrices, which waited for what came before:
  // it is waited for only before this grid ends, so that what follows finds both done
  // (and starts no earlier than that wait).
  if (!g.beside) {
    pdl_wait();
    pdl_release();
  }
  const MuonMat& t = g.mat[blockIdx.y];
  float scale;
  if (skipped(g, &scale) || blockIdx.x >= t.parts) {
    if (g.beside) pdl_wait();
    return;
  }
  const long long count = (long long)t.rows * t.cols, step = (long long)t.parts * kThreads;
  float sum = 0.f;
  // eight values a thread where the arrays allow it (the order of a matrix's sum
  // goes by its size and the arrays' alignment)
  if (t.vec) {
    for (long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * 8; i < count; i += step * 8) {
      float v[8], m[8];
      load8(t.in, t.in_dtype, i, v);
      if (g.update) {
        load8(t.m, DC_F32, i, m);
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = m[k] * g.momentum + v[k] * scale * g.rest;
        float4* to = reinterpret_cast<float4*>(t.m + i);
        to[0] = make_float4(m[0], m[1], m[2], m[3]);
        to[1] = make_float4(m[4], m[5], m[6], m[7]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float u = direction(g, scale, v[k], m[k]);
        sum += u * u;
      }
    }
  } else {
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < count; i += step) {
      const float v = load_in(t.in, t.in_dtype, i);
      float m = 0.f;
      if (g.update) t.m[i] = m = t.m[i] * g.momentum + v * scale * g.rest;
      const float u = direction(g, scale, v, m);
      sum += u * u;
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) t.part[blockIdx.x] = sum;
  if (g.beside) pdl_wait();
}

__global__ void __launch_bounds__(kThreads) muon_begin(const __grid_constant__ MuonGroup g) {
  pdl_wait();
  pdl_release();
  const MuonMat& t = g.mat[blockIdx.y];
  float scale;
  if (skipped(g, &scale) || blockIdx.x >= t.parts) return;
  if (blockIdx.x == 0 && threadIdx.x < 4) t.done[threadIdx.x] = 0u;
  float sum = 0.f;
  for (int i = threadIdx.x; i < t.parts; i += kThreads) sum += t.part[i];
  const float norm = sqrtf(block_sum(sum));
  // a norm that is not finite makes every element NaN
  const float f = norm <= 3.402823466e38f ? kOrthoScale / (norm + kOrthoEps) : __uint_as_float(0x7fffffffu);
  const long long count = (long long)t.rows * t.cols, step = (long long)t.parts * kThreads;
  const long long low = muon_x_low(t);
  if (t.vec && t.cols % 8 == 0) {
    const unsigned row8 = (unsigned)t.cols / 8;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < count / 8; i += step) {
      const unsigned long long r = count < (1LL << 34) ? (unsigned)i / row8 : (unsigned long long)i / row8;
      float v[8], m[8];
      load8(t.in, t.in_dtype, i * 8, v);
      if (g.update) load8(t.m, DC_F32, i * 8, m);
      uint32_t h[4], l[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = direction(g, scale, v[2 * k], m[2 * k]) * f, b = direction(g, scale, v[2 * k + 1], m[2 * k + 1]) * f;
        const __half2 hi = __floats2half2_rn(a, b);
        const float2 back = __half22float2(hi);
        const __half2 lo = __floats2half2_rn(a - back.x, b - back.y);
        h[k] = *reinterpret_cast<const uint32_t*>(&hi);
        l[k] = *reinterpret_cast<const uint32_t*>(&lo);
      }
      __half* x = t.x[0] + r * t.ld + (i - r * row8) * 8;
      *reinterpret_cast<uint4*>(x) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(x + low) = make_uint4(l[0], l[1], l[2], l[3]);
    }
    return;
  }
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < count; i += step) {
    const long long r = i / t.cols;
    const float v = direction(g, scale, load_in(t.in, t.in_dtype, i), g.update ? t.m[i] : 0.f) * f;
    const __half h = __float2half_rn(v);
    __half* x = t.x[0] + r * t.ld + (i - r * t.cols);
    x[0] = h;
    x[low] = __float2half_rn(v - __half2float(h));
  }
}

template <typename K, typename... A>
cudaError_t launch(K kern, dim3 grid, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  note_launches(1);
  return e;
}

}  // namespace

void muon_plan(MuonGroup* g) {
  // a matrix's blocks go by its own size: its sums' order, and so its result's
  // last bits, do not depend on the matrices beside it
  g->parts = 0;
  for (int i = 0; i < g->count; ++i) {
    MuonMat& t = g->mat[i];
    const long long count = (long long)t.rows * t.cols, want = ceil_div_ll(count, 8 * kThreads);
    t.parts = (int)(want < kMuonParts ? want : kMuonParts);
    t.vec = count % 8 == 0 && (uintptr_t)t.in % 16 == 0 && (uintptr_t)t.m % 16 == 0;
    if (t.parts > g->parts) g->parts = t.parts;
  }
}

cudaError_t launch_muon_squares(const MuonGroup& g, cudaStream_t s) {
  return launch(muon_squares, dim3((unsigned)g.parts, (unsigned)g.count), s, g);
}
cudaError_t launch_muon_begin(const MuonGroup& g, cudaStream_t s) {
  return launch(muon_begin, dim3((unsigned)g.parts, (unsigned)g.count), s, g);
}
}  // namespace dc
