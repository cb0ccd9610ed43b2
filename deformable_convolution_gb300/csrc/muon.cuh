// Work table, storage and launchers of the orthogonalisation and the Muon step
// (muon.cu, muon_products.cu).
#pragma once

#include <cuda_fp16.h>

#include "dc_common.cuh"

namespace dc {

// Matrices of one group of launches.
constexpr int kMuonMats = 40;
constexpr int kMuonParts = 608;  // most blocks of the first launch for one matrix
// Values between the products are kept times 2^12: X and A stay below 2^12 *
// 1.5 and the polynomial of A below 2^12 * 4, inside a 16-bit float's range,
// and a pair's low part keeps its digits down to 2^-36.
constexpr float kOrthoScale = 4096.f;
constexpr float kOrthoA = 3.4445f, kOrthoB = -4.7750f, kOrthoC = 2.0315f, kOrthoEps = 1e-7f;

struct MuonMat {
  // what is orthogonalised: `in` (dc_orthogonalize), or m after its update
  const void* in;
  void* out;
  void* param;
  float* master;
  float* m;
  // pairs of 16-bit floats, the low parts `x_low` (p_low) values after the high ones
  __half* x[2];  // [2][rows][ld]
  __half* gram;  // [2][side][lds], the diagonals apart in float32 [lds]
  __half* poly;
  float* gram_diag;
  float* poly_diag;
  float* part;  // sums of squares of the blocks of the first launch
  float* sums;         // a split gram's (muon_sums_bytes)
  unsigned int* done;  // [4] CTAs' finished tiles of each kind
  int rows, cols, ld, side, lds;
  int parts;    // blocks of the launches over single elements
  int vec;      // whose arrays are whole 16-byte pieces
  bool tall;  // rows > cols: A = X^T X, X = a X + X B
  dc_dtype in_dtype, out_dtype;
  float weight_decay, rate;
};

struct MuonGroup {
  int count, steps, parts;  // parts: the largest of the matrices'
  dc_ortho_precision precision;
  bool update;  // a Muon step
  bool beside;  // launched right behind the small matrices of the same call
  float momentum, rest;
  int nesterov;
  float lr;
  const float* grad_scale;
  const float* lr_device;
  MuonMat mat[kMuonMats];
};

__host__ __device__ inline long long muon_x_low(const MuonMat& t) { return (long long)t.rows * t.ld; }
__host__ __device__ inline long long muon_p_low(const MuonMat& t) { return (long long)t.side * t.lds; }

// What the launches of a group share, from its matrices.
void muon_plan(MuonGroup* g);
// Sums of squares of the matrix (a Muon step: m updated); then X times 2^12 /
// (norm + eps) as pairs into x[0], and the counts at 0.
cudaError_t launch_muon_squares(const MuonGroup& g, cudaStream_t s);
cudaError_t launch_muon_begin(const MuonGroup& g, cudaStream_t s);
// All steps; the result to out, or to the parameters.
cudaError_t launch_muon_steps(const MuonGroup& g, cudaStream_t s);
size_t muon_sums_bytes(const MuonMat& t);
// Matrices with a short side up to 64 go through all of it in one launch.
bool muon_is_small(int rows, int cols);
cudaError_t launch_muon_small(const MuonGroup& g, cudaStream_t s);

}  // namespace dc
