// Matrices in 8-bit floating point with a power-of-two scale for each block of
// 128 values: quantising both orientations of a matrix from one read, and
// reading the codes back.
#include <cuda_fp8.h>

#include "dc_common.cuh"
#include "fp8.cuh"
#include "fp8_codes.cuh"

namespace dc {
namespace {

constexpr int kThreads = 256;
constexpr int kB = DC_FP8_BLOCK;

// One block takes a tile of 128 rows and 128 columns, a thread 8 x 8 values of
// it in registers: the half warp h (of 16) has rows 8 h .., its lane l columns
// 8 l ... A row's largest magnitude is a maximum over 16 lanes (of scale bytes,
// which order like the magnitudes, two rows in a word), a column's one over
// half warps through shared memory.  Codes of the rows leave from registers, 16
// lanes writing a line of 128 bytes; those of the columns go through a tile in
// shared memory whose 8-byte units are swizzled by the column group: neither
// its writes nor its reads meet in a bank.
template <typename T, int FMT, bool SQUARE, bool DIRECT, bool TRANSPOSED>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) fp8_quantize(Fp8Args a, int vectors) {
  __shared__ uint32_t part[TRANSPOSED && !SQUARE ? kThreads / 32 : 1][kB];
  __shared__ uint32_t shared_top;
  __shared__ float col_inv[kB];
  __shared__ __align__(16) unsigned char tile[TRANSPOSED ? kB * kB : 16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int l = lane & 15, h = 2 * warp + (lane >> 4);
  const int tiles_c = (a.cols + kB - 1) / kB;
  const int by = blockIdx.x / tiles_c, bx = blockIdx.x - by * tiles_c;  // the tile's row and column
  const int r0 = by * kB, c0 = bx * kB;
  const int row = r0 + 8 * h, col = c0 + 8 * l;
  const T* x = static_cast<const T*>(a.x) + ((long long)blockIdx.z * a.rows + row) * a.cols + col;
  if (SQUARE && tid == 0) shared_top = 0u;
  pdl_wait();
  pdl_release();
  Eight<T> v[8];
  const int left = min(8, a.cols - col);  // columns of this thread's that there are
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int some = row + r < a.rows ? left : 0;
    if (vectors && some > 0)  // then `some` is eight
      v[r].load(x + (long long)r * a.cols);
    else
      v[r].load_some(x + (long long)r * a.cols, some);
  }
  const long long kr = ceil_div_ll(a.rows, kB), kc = ceil_div_ll(a.cols, kB);
  uint32_t byte[8];  // the rows' scales
  if (SQUARE) {
    uint32_t top = 0u;
#pragma unroll
    for (int r = 0; r < 8; ++r) top = max(top, v[r].top());
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if (lane == 0) atomicMax(&shared_top, top);
    __syncthreads();
    const uint32_t b = scale_byte<FMT>(shared_top);
#pragma unroll
    for (int r = 0; r < 8; ++r) byte[r] = b;
  } else {
    if (TRANSPOSED) {
      uint32_t top[8];
      column_tops<T>(v, top);
      if (lane < 16) {
        *reinterpret_cast<uint4*>(&part[warp][8 * l]) = make_uint4(top[0], top[1], top[2], top[3]);
        *reinterpret_cast<uint4*>(&part[warp][8 * l + 4]) = make_uint4(top[4], top[5], top[6], top[7]);
      }
    }
    if (DIRECT) {
#pragma unroll
      for (int r = 0; r < 8; r += 2) {
        uint32_t two = scale_byte<FMT>(v[r].top()) | (scale_byte<FMT>(v[r + 1].top()) << 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, o));
        byte[r] = two & 0xffffu;
        byte[r + 1] = two >> 16;
      }
    }
  }
  if (DIRECT) {
    // the byte of row r of the tile: (r % 32) * 16 + r / 32 * 4, for the run's place among four
    unsigned char* sc = a.scales + ((blockIdx.z * kr + by) * ((kc + 3) / 4) + bx / 4) * 512 +
                        (8 * h & 31) * 16 + h / 4 * 4 + bx % 4;
    unsigned char* q = a.codes + ((long long)blockIdx.z * a.rows + row) * (kc * kB) + col;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float s = inverse_scale(byte[r]);
      uint2 c;
      c.x = codes2<FMT>(v[r].get(0) * s, v[r].get(1) * s) | (codes2<FMT>(v[r].get(2) * s, v[r].get(3) * s) << 16);
      c.y = codes2<FMT>(v[r].get(4) * s, v[r].get(5) * s) | (codes2<FMT>(v[r].get(6) * s, v[r].get(7) * s) << 16);
      if (row + r < a.rows) *reinterpret_cast<uint2*>(q + r * (kc * kB)) = c;
      if (l == r) sc[16 * r] = (unsigned char)byte[r];
    }
  }
  if (!TRANSPOSED) return;
  if (!SQUARE) __syncthreads();
  if (tid < kB) {
    uint32_t b = byte[0];
    if (!SQUARE) {
      uint32_t top = 0u;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) top = max(top, part[w][tid]);
      b = scale_byte<FMT>(top);
    }
    col_inv[tid] = inverse_scale(b);
    a.scales_t[((blockIdx.z * kc + bx) * ((kr + 3) / 4) + by / 4) * 512 + (tid & 31) * 16 +
               (tid >> 5) * 4 + by % 4] = (unsigned char)b;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = col_inv[8 * l + i];
    uint2 c;
    c.x = codes2<FMT>(v[0].get(i) * s, v[1].get(i) * s) | (codes2<FMT>(v[2].get(i) * s, v[3].get(i) * s) << 16);
    c.y = codes2<FMT>(v[4].get(i) * s, v[5].get(i) * s) | (codes2<FMT>(v[6].get(i) * s, v[7].get(i) * s) << 16);
    *reinterpret_cast<uint2*>(tile + (8 * l + i) * kB + ((h ^ l) << 3)) = c;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (tid >> 3) + 32 * k, u = tid & 7, g = c >> 3;  // units 2 u and 2 u + 1 of column c
    uint4 q = *reinterpret_cast<const uint4*>(tile + c * kB + (((2 * u) ^ (g & ~1)) << 3));
    if (g & 1) q = make_uint4(q.z, q.w, q.x, q.y);
    if (c0 + c < a.cols)
      *reinterpret_cast<uint4*>(a.codes_t + ((long long)blockIdx.z * a.cols + c0 + c) * (kr * kB) + r0 + 16 * u) = q;
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
  cfg.gridDim = dim3((unsigned)(ceil_div_ll(a.cols, kB) * ceil_div_ll(a.rows, kB)), 1, (unsigned)a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int vectors = a.cols % 8 == 0 && (uintptr_t)a.x % 16 == 0;
  auto go = [&](auto kern) { return cudaLaunchKernelEx(&cfg, kern, a, vectors); };
  const cudaError_t e =
      !a.codes_t  ? (a.square ? go(fp8_quantize<T, FMT, true, true, false>) : go(fp8_quantize<T, FMT, false, true, false>))
      : !a.codes ? (a.square ? go(fp8_quantize<T, FMT, true, false, true>) : go(fp8_quantize<T, FMT, false, false, true>))
                 : (a.square ? go(fp8_quantize<T, FMT, true, true, true>) : go(fp8_quantize<T, FMT, false, true, true>));
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
