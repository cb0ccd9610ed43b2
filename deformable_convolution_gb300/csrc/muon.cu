// Orthogonalisation by Newton-Schulz products and the Muon step: the passes
// over single elements around the products.
#include "muon.cuh"

namespace dc {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_in(const void* p, dc_dtype dt, long long i) {
  return dt == DC_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Whether the step is skipped: its scale is not finite.
__device__ __forceinline__ bool skipped(const MuonGroup& g, float* scale) {
  *scale = g.update && g.grad_scale ? *g.grad_scale : 1.f;
  return !(fabsf(*scale) <= 3.402823466e38f);
}

// What is orthogonalised: u of the updated m and the gradient, or `in`.
__device__ __forceinline__ float direction(const MuonGroup& g, const MuonMat& t, float scale, long long i) {
  const float v = load_in(t.in, t.in_dtype, i);
  if (!g.update) return v;
  const float m = t.m[i];
  return g.nesterov ? m * g.momentum + v * scale * g.rest : m;
}

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
  pdl_wait();
  pdl_release();
  const MuonMat& t = g.mat[blockIdx.y];
  float scale;
  if (skipped(g, &scale) || blockIdx.x >= t.parts) return;
  const long long count = (long long)t.rows * t.cols;
  float sum = 0.f;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < count; i += (long long)t.parts * kThreads) {
    if (g.update) {
      const float v = load_in(t.in, t.in_dtype, i) * scale;
      t.m[i] = t.m[i] * g.momentum + v * g.rest;
    }
    const float u = direction(g, t, scale, i);
    sum += u * u;
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) t.part[blockIdx.x] = sum;
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
  const long long count = (long long)t.rows * t.cols;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < count; i += (long long)t.parts * kThreads) {
    const long long r = i / t.cols;
    const float v = direction(g, t, scale, i) * f;
    const __half h = __float2half_rn(v);
    __half* x = t.x[0] + r * t.ld + (i - r * t.cols);
    x[0] = h;
    x[muon_x_low(t)] = __float2half_rn(v - __half2float(h));
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
    const long long want = ceil_div_ll((long long)t.rows * t.cols, 8 * kThreads);
    t.parts = (int)(want < kMuonParts ? want : kMuonParts);
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
