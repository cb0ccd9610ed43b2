// Arguments and launchers of the matrices in 8 bits (fp8.cu, fp8_matmul.cu).
#pragma once

#include "dc_common.cuh"

namespace dc {

struct Fp8Args {
  int batch, rows, cols, square;
  dc_dtype dtype;
  dc_fp8 format;
  const void* x;
  unsigned char* codes;  // either pair may be null
  unsigned char* scales;
  unsigned char* codes_t;
  unsigned char* scales_t;
};
cudaError_t launch_fp8_quantize(const Fp8Args& a, cudaStream_t s);
cudaError_t launch_fp8_values(int batch, int rows, int cols, dc_fp8 format, const void* codes,
                              const void* scales, float* out, cudaStream_t s);

struct Fp8Product {
  dc_fp8_product p;
  const void* a;
  const void* a_scales;
  const void* b;
  const void* b_scales;
  void* d;
  void* ws;
};
struct Fp8Pointwise {
  dc_fp8_layer p;
  const void* x;
  const void* w_codes;
  const void* w_scales;
  void* y;
};
cudaError_t launch_fp8_pointwise(const Fp8Pointwise& t, cudaStream_t s);
size_t fp8_matmul_workspace_bytes(const dc_fp8_product& p);
cudaError_t launch_fp8_matmul(const Fp8Product& a, cudaStream_t s);

}  // namespace dc
