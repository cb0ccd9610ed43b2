// Products of matrices in 8-bit floating point with block scales.
#include <cuda_fp8.h>

#include "fp8.cuh"

namespace dc {
namespace {

constexpr int kTile = 64, kStep = 32;

__device__ __forceinline__ float decode(unsigned char q, dc_fp8 f) {
  const __half_raw h = f == DC_E4M3 ? __nv_cvt_fp8_to_halfraw(q, __NV_E4M3) : __nv_cvt_fp8_to_halfraw(q, __NV_E5M2);
  return __half2float(__half(h));
}

__device__ __forceinline__ float scale_of(const unsigned char* s, long long i, int rows, int k, int r, int c) {
  const long long kr = (rows + 127) / 128, kc = (k + 127) / 128;
  return __uint_as_float(
      (uint32_t)s[((i * kr + r / 128) * ((kc + 3) / 4) + c / 512) * 512 + (r & 31) * 16 + (r % 128) / 32 * 4 + c / 128 % 4]
      << 23);
}

__global__ void __launch_bounds__(256) fp8_matmul(Fp8Product t) {
  __shared__ float sa[kTile][kStep + 1], sb[kTile][kStep + 1];
  pdl_wait();
  pdl_release();
  const dc_fp8_product& p = t.p;
  const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile, ld = (p.k + 127) / 128 * 128;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  const int first = p.sum ? 0 : blockIdx.z, last = p.sum ? p.batch : first + 1;
  for (int i = first; i < last; ++i) {
    const long long ia = p.a_shared ? 0 : i, ib = p.b_shared ? 0 : i;
    const unsigned char* a = static_cast<const unsigned char*>(t.a) + ia * p.m * (long long)ld;
    const unsigned char* b = static_cast<const unsigned char*>(t.b) + ib * p.n * (long long)ld;
    for (int k0 = 0; k0 < p.k; k0 += kStep) {
      for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
        const int r = e / kStep, c = e % kStep;
        sa[r][c] = m0 + r < p.m ? decode(a[(long long)(m0 + r) * ld + k0 + c], p.a_format) *
                                      scale_of(static_cast<const unsigned char*>(t.a_scales), ia, p.m, p.k, m0 + r, k0 + c)
                                : 0.f;
        sb[r][c] = n0 + r < p.n ? decode(b[(long long)(n0 + r) * ld + k0 + c], p.b_format) *
                                      scale_of(static_cast<const unsigned char*>(t.b_scales), ib, p.n, p.k, n0 + r, k0 + c)
                                : 0.f;
      }
      __syncthreads();
      for (int c = 0; c < kStep; ++c)
        for (int u = 0; u < 4; ++u)
          for (int v = 0; v < 4; ++v) acc[u][v] += sa[ty * 4 + u][c] * sb[tx * 4 + v][c];
      __syncthreads();
    }
  }
  for (int u = 0; u < 4; ++u)
    for (int v = 0; v < 4; ++v) {
      const int m = m0 + ty * 4 + u, n = n0 + tx * 4 + v;
      if (m >= p.m || n >= p.n) continue;
      const long long at = ((long long)(p.sum ? 0 : blockIdx.z) * p.m + m) * p.n + n;
      if (p.out == DC_F32)
        static_cast<float*>(t.d)[at] = acc[u][v];
      else
        static_cast<__nv_bfloat16*>(t.d)[at] = __float2bfloat16_rn(acc[u][v]);
    }
}

}  // namespace

size_t fp8_matmul_workspace_bytes(const dc_fp8_product&) { return 0; }

cudaError_t launch_fp8_matmul(const Fp8Product& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ceil_div_ll(a.p.n, kTile), (unsigned)ceil_div_ll(a.p.m, kTile),
                     a.p.sum ? 1u : (unsigned)a.p.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_matmul, a);
  note_launches(1);
  return e;
}

}  // namespace dc
