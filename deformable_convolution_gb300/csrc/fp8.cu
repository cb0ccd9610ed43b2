// Matrices in 8-bit floating point with a power-of-two scale for each block of
// 128 values: quantising both orientations of a matrix from one read, and
// reading the codes back.
#include <cuda_fp8.h>

#include "dc_common.cuh"
#include "fp8.cuh"

namespace dc {
namespace {

constexpr int kThreads = 256;
constexpr int kB = DC_FP8_BLOCK;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale byte of a block whose largest magnitude has these bits: exponent
// e = exponent(top) - high (+ 1 where top's mantissa is above 1.75), so that
// top / 2^e is at most 1.75 * 2^high, the largest code.  Bits order like
// magnitudes, and what is not finite sorts above.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  constexpr int high = FMT == DC_E4M3 ? 8 : 15;
  const int e = (int)(top >> 23) - high + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e);
}

// 2^-(byte - 127): exact for bytes 1 .. 254 (those that blocks have are at
// most 247); NaN for 255, which makes the block's codes NaN.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - byte) << 23);
}

// Two codes of scaled values, rounded to nearest even; `a` in the low byte.
template <int FMT>
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(
      make_float2(a, b), __NV_SATFINITE, FMT == DC_E4M3 ? __NV_E4M3 : __NV_E5M2);
  return (uint32_t)c;
}

// Tile [128 rows][128 columns] per block, from one read to both orientations.
template <typename T, int FMT, bool SQUARE>
__global__ void __launch_bounds__(kThreads) fp8_quantize(Fp8Args a) {
  __shared__ float tile[kB][kB + 1];
  __shared__ uint32_t row_top[kB], col_top[kB];
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x;
  const int r0 = blockIdx.y * kB, c0 = blockIdx.x * kB;
  const T* x = static_cast<const T*>(a.x) + (long long)blockIdx.z * a.rows * a.cols;
  if (tid < kB) row_top[tid] = col_top[tid] = 0u;
  __syncthreads();
  const int lane = tid & 31, warp = tid >> 5;
  uint32_t ct[4] = {0u, 0u, 0u, 0u};
  for (int r = warp; r < kB; r += kThreads / 32) {
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = lane + 32 * j;
      const bool in = r0 + r < a.rows && c0 + c < a.cols;
      const float v = in ? ld_f(x + (long long)(r0 + r) * a.cols + c0 + c) : 0.f;
      tile[r][c] = v;
      const uint32_t m = magnitude(v);
      top = max(top, m);
      ct[j] = max(ct[j], m);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) row_top[r] = top;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) atomicMax(&col_top[lane + 32 * j], ct[j]);
  __syncthreads();
  if (SQUARE) {
    uint32_t top = 0u;
    for (int r = lane; r < kB; r += 32) top = max(top, row_top[r]);
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if (tid < kB) row_top[tid] = col_top[tid] = top;
    __syncthreads();
  }
  const long long kr = ceil_div_ll(a.rows, kB), kc = ceil_div_ll(a.cols, kB);
  if (tid < kB) {
    const int at = (tid & 31) * 16 + (tid >> 5) * 4;
    const uint32_t rb = scale_byte<FMT>(row_top[tid]), cb = scale_byte<FMT>(col_top[tid]);
    if (a.scales)
      a.scales[((blockIdx.z * kr + blockIdx.y) * ((kc + 3) / 4) + blockIdx.x / 4) * 512 + at + blockIdx.x % 4] =
          (unsigned char)rb;
    if (a.scales_t)
      a.scales_t[((blockIdx.z * kc + blockIdx.x) * ((kr + 3) / 4) + blockIdx.y / 4) * 512 + at + blockIdx.y % 4] =
          (unsigned char)cb;
  }
  if (a.codes)
    for (int r = warp; r < kB && r0 + r < a.rows; r += kThreads / 32) {
      const float s = inverse_scale(scale_byte<FMT>(row_top[r]));
      unsigned char* q = a.codes + ((long long)blockIdx.z * a.rows + r0 + r) * (kc * kB) + c0;
      const uint32_t lo = codes2<FMT>(tile[r][4 * lane] * s, tile[r][4 * lane + 1] * s);
      const uint32_t hi = codes2<FMT>(tile[r][4 * lane + 2] * s, tile[r][4 * lane + 3] * s);
      reinterpret_cast<uint32_t*>(q)[lane] = lo | (hi << 16);
    }
  if (a.codes_t)
    for (int c = warp; c < kB && c0 + c < a.cols; c += kThreads / 32) {
      const float s = inverse_scale(scale_byte<FMT>(col_top[c]));
      unsigned char* q = a.codes_t + ((long long)blockIdx.z * a.cols + c0 + c) * (kr * kB) + r0;
      const uint32_t lo = codes2<FMT>(tile[4 * lane][c] * s, tile[4 * lane + 1][c] * s);
      const uint32_t hi = codes2<FMT>(tile[4 * lane + 2][c] * s, tile[4 * lane + 3][c] * s);
      reinterpret_cast<uint32_t*>(q)[lane] = lo | (hi << 16);
    }
}

// rows, cols: of the matrix that the codes are of (transposed or not).
template <int FMT>
__global__ void __launch_bounds__(kThreads)
    fp8_values(int batch, int rows, int cols, const unsigned char* __restrict__ codes,
               const unsigned char* __restrict__ scales, float* __restrict__ out) {
  pdl_wait();
  pdl_release();
  const long long total = (long long)batch * rows * cols;
  const long long kc = ceil_div_ll(cols, kB), kr = ceil_div_ll(rows, kB);
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total; i += (long long)gridDim.x * kThreads) {
    const long long row = i / cols;
    const int c = (int)(i - row * cols);
    const long long b = row / rows;
    const int r = (int)(row - b * rows);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(codes[row * kc * kB + c], FMT == DC_E4M3 ? __NV_E4M3 : __NV_E5M2);
    const uint32_t s = scales[((b * kr + r / kB) * ((kc + 3) / 4) + c / kB / 4) * 512 + (r & 31) * 16 + (r % kB) / 32 * 4 +
                              c / kB % 4];
    // 2^(s - 127), s at least 1; 255: the codes are NaN
    out[i] = __half2float(__half(h)) * __uint_as_float(s << 23);
  }
}

template <typename T, int FMT>
cudaError_t quantize(const Fp8Args& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ceil_div_ll(a.cols, kB), (unsigned)ceil_div_ll(a.rows, kB), (unsigned)a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.square ? cudaLaunchKernelEx(&cfg, fp8_quantize<T, FMT, true>, a)
                                 : cudaLaunchKernelEx(&cfg, fp8_quantize<T, FMT, false>, a);
  note_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8Args& a, cudaStream_t s) {
  if (a.dtype == DC_BF16)
    return a.format == DC_E4M3 ? quantize<__nv_bfloat16, DC_E4M3>(a, s) : quantize<__nv_bfloat16, DC_E5M2>(a, s);
  return a.format == DC_E4M3 ? quantize<float, DC_E4M3>(a, s) : quantize<float, DC_E5M2>(a, s);
}

cudaError_t launch_fp8_values(int batch, int rows, int cols, dc_fp8 format, const void* codes,
                              const void* scales, float* out, cudaStream_t s) {
  const long long blocks = ceil_div_ll((long long)batch * rows * cols, kThreads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto* c = static_cast<const unsigned char*>(codes);
  const auto* sc = static_cast<const unsigned char*>(scales);
  const cudaError_t e = format == DC_E4M3
                            ? cudaLaunchKernelEx(&cfg, fp8_values<DC_E4M3>, batch, rows, cols, c, sc, out)
                            : cudaLaunchKernelEx(&cfg, fp8_values<DC_E5M2>, batch, rows, cols, c, sc, out);
  note_launches(1);
  return e;
}

}  // namespace dc
