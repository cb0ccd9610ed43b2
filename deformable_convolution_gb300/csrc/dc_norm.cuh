// Group norm with an activation: what its translation units share (tilings,
// vector access, activations, statistics, cluster and launch helpers).
//
// Statistics.  A thread keeps (count, mean, M2) of what it has read, M2 the
// sum of squared distances from its own mean: a batch of vectors is averaged
// first and its squared distances summed second, and two such triples merge
// exactly,
//   d = mb - ma, m = ma + d nb / (na + nb), M2 = M2a + M2b + d^2 na nb / (na + nb),
// so no sum of squares about a far-off origin is ever formed (a large mean
// over a small spread costs no digits).
#pragma once

#include <type_traits>

#include "dc_common.cuh"

namespace dc {


// Two floats in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 ra, rb, rd;\n mov.b64 ra, {%2,%3};\n mov.b64 rb, {%4,%5};\n"
      " mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0,%1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 ra, rb, rd;\n mov.b64 ra, {%2,%3};\n mov.b64 rb, {%4,%5};\n"
      " add.rn.f32x2 rd, ra, rb;\n mov.b64 {%0,%1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2,%3};\n mov.b64 rb, {%4,%5};\n"
      " mov.b64 rc, {%6,%7};\n fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0,%1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// V floats as pairs; V = 1 leaves the second of its pair unused.
template <int V>
struct Pairs {
  static constexpr int n = (V + 1) / 2;
  float2 p[n];
  __device__ __forceinline__ float& operator[](int e) { return e & 1 ? p[e >> 1].y : p[e >> 1].x; }
  __device__ __forceinline__ float operator[](int e) const {
    return e & 1 ? p[e >> 1].y : p[e >> 1].x;
  }
};

template <typename T>
struct VecOf {
  static constexpr int n = 16 / sizeof(T);
};

// V floats to p (aligned to V * sizeof(T) bytes).
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float* f) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) p[e] = f[e];
    }
  } else if constexpr (V == 1) {
    p[0] = __float2bfloat16_rn(f[0]);
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
      w[e] = *reinterpret_cast<uint32_t*>(&b);
    }
    if constexpr (V == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// V packed elements to pairs.
template <typename T, int V>
__device__ __forceinline__ void unpack(const uint32_t* u, Pairs<V>& f) {
#pragma unroll
  for (int e = 0; e < Pairs<V>::n; ++e) {
    if (sizeof(T) == 4)
      f.p[e] = make_float2(__uint_as_float(u[V == 1 ? 0 : 2 * e]),
                           V == 1 ? 0.f : __uint_as_float(u[V == 1 ? 0 : 2 * e + 1]));
    else
      f.p[e] = make_float2(__uint_as_float(u[e] << 16),
                           V == 1 ? 0.f : __uint_as_float(u[e] & 0xffff0000u));
  }
}

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, Pairs<V>& f) {
  constexpr int kBytes = V * sizeof(T);
  uint32_t u[(kBytes + 3) / 4];
  if constexpr (kBytes >= 16) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      u[4 * i] = v.x, u[4 * i + 1] = v.y, u[4 * i + 2] = v.z, u[4 * i + 3] = v.w;
    }
  } else if constexpr (kBytes == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    u[0] = v.x, u[1] = v.y;
  } else if constexpr (kBytes == 4) {
    u[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    u[0] = *reinterpret_cast<const unsigned short*>(p);
  }
  unpack<T, V>(u, f);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Pairs<V>& f) {
  store_vec<T, V>(p, reinterpret_cast<const float*>(f.p));
}

// The elements [lo, hi) of a vector whose ends lie outside the row.
template <typename T, int V>
__device__ __forceinline__ void load_part(const T* p, int lo, int hi, float* f) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = e >= lo && e < hi ? to_f(p[e]) : 0.f;
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T* p, int lo, int hi, const float* f) {
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e >= lo && e < hi) p[e] = from_f<T>(f[e]);
}

// One instruction each, subnormal numbers as 0.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// sum / n by the approximate reciprocal w of n and the remainder: exact where
// the quotient is a float (a constant's mean is the constant).
__device__ __forceinline__ float quotient(float sum, float n, float w) {
  const float m = sum * w;
  return fmaf(fmaf(-m, n, sum), w, m);
}
__device__ __forceinline__ float2 quotient2(float2 sum, float n, float w) {
  const float2 m = mul2(sum, both(w));
  return fma2(fma2(make_float2(-m.x, -m.y), both(n), sum), both(w), m);
}

// 1 / (1 + exp(-z))
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  const float2 t = mul2(z, both(-1.4426950408889634f));
  const float2 u = add2(make_float2(exp2_approx(t.x), exp2_approx(t.y)), both(1.f));
  return make_float2(rcp_approx(u.x), rcp_approx(u.y));
}

// The normal distribution's Phi(z), and e = exp(-z^2 / 2): Abramowitz and
// Stegun's rational approximation 7.1.26 of erf (absolute error 1.5e-7) at
// |z| / sqrt 2; it needs e anyway, as the slope does.  z Phi(z) measured on
// 2^19 values in [-9, 9], largest error over a range of z against that of
// 0.5 z (1 + erf) in float32: [-5, -4] 5.9e-8 / 1.2e-7, [-4, -2] 2.1e-7 /
// 2.6e-7, [-2, -1] 1.5e-7 / 1.8e-7, [-1, 1] 1.5e-7 / 1.4e-7, [2, 9] 4.2e-7 /
// 4.7e-7; the slope 3e-7 anywhere.
__device__ __forceinline__ float2 normal_cdf2(float2 z, float2* e) {
  const float2 a = make_float2(fabsf(z.x), fabsf(z.y));
  const float2 u = fma2(a, both(0.3275911f * 0.70710678118654752f), both(1.f));
  const float2 t = make_float2(rcp_approx(u.x), rcp_approx(u.y));
  const float2 s = mul2(mul2(z, z), both(-0.72134752044448170f));
  *e = make_float2(exp2_approx(s.x), exp2_approx(s.y));
  float2 q = fma2(both(0.5f * 1.061405429f), t, both(0.5f * -1.453152027f));
  q = fma2(q, t, both(0.5f * 1.421413741f));
  q = fma2(q, t, both(0.5f * -0.284496736f));
  q = fma2(q, t, both(0.5f * 0.254829592f));
  q = mul2(mul2(q, t), *e);  // Phi(-|z|)
  const float2 c = add2(both(1.f), make_float2(-q.x, -q.y));
  return make_float2(z.x < 0.f ? q.x : c.x, z.y < 0.f ? q.y : c.y);
}

// Activations by kind: 0 max(z, floor), the floor 0 for the ReLU and -inf for
// none (NaN is kept); 1 SiLU; 2 GELU.
template <int ACT>
__device__ __forceinline__ float2 act_fwd2(float2 z, float floor) {
  if (ACT == 1) return mul2(z, sigmoid2(z));
  if (ACT == 2) {
    float2 e;
    const float2 c = normal_cdf2(z, &e);
    return mul2(z, c);
  }
  float2 y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y.x) : "f"(z.x), "f"(floor));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y.y) : "f"(z.y), "f"(floor));
  return y;
}

// d * act'(z); the ReLU's closed side passes nothing, whatever d is.
template <int ACT>
__device__ __forceinline__ float2 act_bwd2(float2 z, float2 d, float floor) {
  if (ACT == 1) {
    const float2 sg = sigmoid2(z);
    const float2 r = add2(both(1.f), make_float2(-sg.x, -sg.y));
    return mul2(d, fma2(mul2(z, sg), r, sg));
  }
  if (ACT == 2) {
    float2 e;
    const float2 cdf = normal_cdf2(z, &e);
    return mul2(d, fma2(mul2(z, both(0.39894228040143268f)), e, cdf));
  }
  const bool none = floor < 0.f;  // (every z is open then, NaN and -inf too)
  return make_float2(z.x > floor || none ? d.x : 0.f, z.y > floor || none ? d.y : 0.f);
}

// ---------------------------------------------------------------- the tiling
// NCHW: a row is one channel of one image, hw consecutive elements; `lpr`
// lanes of a warp walk a row's 16-byte vectors (the first and last may hang
// over the row's ends), a warp takes 32 / lpr rows, and a long row is cut into
// `parts` segments of `seg` vectors.
struct Shape {
  int n, c, groups, cpg, hw;
  float floor;  // of activation kind 0
  float eps;
  int v;                // NHWC: channels of a thread's vector
  int parts, seg, lpr;  // NCHW
  // reciprocals: of a unit's values, cpg, parts and the columns of a block
  // (a block runs its few hundred instructions of preparation once: a
  // division in full is one part in twenty of them)
  float inv_total, inv_cpg, inv_parts, inv_cb;
};

// a / b for 0 <= a < 2^20 by the rounded reciprocal of b: (a + 1/2) / b is at
// least 1 / (2 b) from a whole number, the product's error below a / b * 2^-22.
__device__ __forceinline__ int quick_div(int a, float inv) {
  return (int)(((float)a + 0.5f) * inv);
}

// The mean of a unit from its sum.
__device__ __forceinline__ float unit_mean(const Shape& s, float sum) {
  return quotient(sum, (float)s.hw * (float)s.cpg, s.inv_total);
}

// How the blocks share the work.  A unit has `blocks` of them: a cluster that
// holds the unit in shared memory from its statistics to its results (one
// launch for a pass), or blocks that leave their statistics in memory for a
// second launch, which reads the unit again (from L2, where it fits there).
// NCHW: a unit is a group of an image; its rows are cut into tasks as above,
// dealt over the warps of the unit's blocks in `rounds`.
struct RowTeam {
  int blocks, warps, units;  // of a unit, of a unit in a block, units of a block
  int tasks, rounds;         // of a unit, of a warp
  // whole-vector rows, forward: the unit's vectors in one run, `span` of them
  // to a block (0: by tasks)
  int span, step_c, step_v;  // threads of a unit in a block, as channels and vectors
};
// NHWC: a unit is a slice of channels, `cb` vectors wide, of an image (whole
// groups, in a cluster); a thread keeps one of its columns and walks pixels,
// `rl` threads to a column.
struct ColTeam {
  int blocks, slices, width;  // blocks of a unit, units of an image, channels of a unit
  int cb, rl, ng;             // ng: groups of a unit (cluster)
  int span;                   // pixels of a block
  int held;                   // pixels of a thread kept in shared memory
  int rows;                   // of the backward's table of channel sums
  int shares;                 // most slices that share a group (two launches)
};
constexpr int kTeam = 512;       // most threads of a cluster's block
constexpr int kTwo = 256;        // threads of a block of two launches
constexpr int kMaxCluster = 16;
constexpr int kMaxGroups = 64;   // of a unit (NHWC, in a cluster)

// Whether the backward keeps dz, in float32, where it held grad_y: where the
// slope costs more than a wider slot (SiLU, GELU), or the slot is that wide.
constexpr bool keep_dz(bool grad_f32, int act_kind) { return grad_f32 || act_kind != 0; }

struct NormPlan {
  Shape s;
  bool cluster;  // one launch; else two
  RowTeam row;
  ColTeam col;
  unsigned blocks;  // of a launch (two launches: of `images` images)
  int threads;
  size_t smem;
  int parts;   // rows of channel sums that an image leaves (backward)
  int images;  // two launches: at a time, so that the second finds them in L2
};
// The forward, or the backward up to the channels' sums.  Two launches: the
// first (second = false) or the second of images [img0, img0 + count).
cudaError_t launch_nchw(const NormPlan& p, const NormArgs& a, bool backward, cudaStream_t s);
cudaError_t launch_nhwc(const NormPlan& p, const NormArgs& a, bool backward, cudaStream_t s);
cudaError_t launch_two_nchw(const NormPlan& p, const NormArgs& a, bool backward, bool second,
                            int img0, int count, cudaStream_t s);
cudaError_t launch_two_nhwc(const NormPlan& p, const NormArgs& a, bool backward, bool second,
                            int img0, int count, cudaStream_t s);
// Workspace of the two launches: the channels' sums (backward), then an entry
// for each group of an image, block of it and slice that shares it.
inline size_t norm_part_bytes(const NormPlan& p, const NormArgs& a, bool backward) {
  return backward ? ((size_t)p.parts * a.n * a.c * sizeof(float2) + 255) / 256 * 256 : 0;
}

__host__ __device__ inline int row_vectors(int hw, int mis, int vec) {
  return (mis + hw + vec - 1) / vec;
}

// Two launches over whole-vector rows: the `count` vectors from `begin` on that
// block `rank` takes of its unit, `span` to a block.  (A block has 2^30 at most,
// a unit 2^31 and more: a group of 32 GB.)
struct BlockRun {
  long long begin;
  int count;
  __host__ __device__ BlockRun(int cpg, int row_vectors, int span, int rank)
      : begin((long long)rank * span) {
    const long long left = (long long)cpg * row_vectors - begin;
    count = left < 0 ? 0 : left < span ? (int)left : span;
  }
};

__device__ __forceinline__ void merge(float& n, float& mean, float& m2, float nb, float mb,
                                      float m2b) {
  if (nb == 0.f) return;
  const float t = n + nb, d = mb - mean, w = n > 0.f ? nb * rcp_approx(t) : 1.f;
  mean += d * w;
  m2 += m2b + d * d * n * w;
  n = t;
}

// Sum over the lpr lanes that share a row (lpr a power of two), in every lane.
__device__ __forceinline__ float row_sum(float v, int lpr) {
  if (lpr == 32) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  for (int o = lpr >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_sum(float v) { return row_sum(v, 32); }

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// This block's place in its cluster, and the cluster's in the grid (a launch
// without clusters counts as clusters of one).
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_id() {
  int r;
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
// *p of the cluster's block `rank` = v
__device__ __forceinline__ void store_cluster(float* p, int rank, float v) {
  uint32_t to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(to)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}

// Asynchronous copy of BYTES (4, 8 or 16) to shared memory; of 16, only the
// first `bytes` are read and the rest becomes zero.
// TWICE: the other half of a 32-byte sector is copied too, so the sector stays
// in L1 (past it, the sector comes from L2 for each half).
template <int BYTES, bool TWICE = false>
__device__ __forceinline__ void copy_async(void* to, const void* from, int bytes = BYTES) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
  if (BYTES == 16 && TWICE)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(bytes)
                 : "memory");
  else if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(bytes)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(from), "n"(BYTES)
                 : "memory");
}
// Copies are grouped as they are started, and a thread waits until no more
// than `open` of its groups are (or 7), so that it works on the first of its
// vectors while the others arrive.
__device__ __forceinline__ void copy_group() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copy_wait(int open) {
  switch (open < 7 ? open : 7) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}

// A thread's stream of `count` items through slots of its own: start(i, slot)
// starts the copies of item i, work(i, most, slot) works on items [i, i + most)
// in the slots from `slot` on.  kRing batches of B items: two arrive while one
// is worked on, and the copies go to the batch whose work is done.
constexpr int kRing = 3;
template <int B, typename START, typename WORK>
__device__ __forceinline__ void through_ring(int count, START&& start, WORK&& work) {
  int next = 0, put = 0, at = 0;
  auto batch = [&] {
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (next + b < count) start(next + b, put + b);
    copy_group();
    next += B;
    put = put == (kRing - 1) * B ? 0 : put + B;
  };
#pragma unroll
  for (int r = 0; r < kRing - 1; ++r) batch();
  for (int i = 0; i < count; i += B) {
    batch();
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    work(i, min(count - i, B), at);
    at = at == (kRing - 1) * B ? 0 : at + B;
  }
}

// Dynamic shared memory that a kernel may be launched with: more than any plan
// asks for, and one value for all of them.  The limit is the kernel's, not the
// call's: a host thread that set it to its own launch's need would have the
// launch of another one, in between, refused.
constexpr int kSmemLimit = 160 * 1024;
template <typename K>
cudaError_t allow_smem(K kern, size_t smem) {
  if (smem <= 40 * 1024) return cudaSuccess;  // (beside up to 6 KB of static arrays)
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
}

template <typename K, typename... A>
cudaError_t launch_team(K kern, const NormPlan& p, int cluster, cudaStream_t s, A... args) {
  cudaError_t e = cudaSuccess;
  if (cluster > 8)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = allow_smem(kern, p.smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.blocks);
  cfg.blockDim = dim3((unsigned)p.threads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, args...);
  note_launches(1);
  return e;
}

// A launch without a cluster (programmatic, as all of this library's).
template <typename K, typename... A>
cudaError_t launch_smem(K kern, unsigned blocks, int threads, size_t smem, cudaStream_t s,
                        A... args) {
  cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, args...);
  note_launches(1);
  return e;
}
template <typename K, typename... A>
cudaError_t launch_plain(K kern, unsigned blocks, int threads, cudaStream_t s, A... args) {
  return launch_smem(kern, blocks, threads, 0, s, args...);
}

template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename F>
cudaError_t by_dtype(dc_dtype dt, F&& f) {
  return dt == DC_BF16 ? f(__nv_bfloat16{}) : f(float{});
}
// f(x's type, grad_y's type)
template <typename F>
cudaError_t by_dtypes(const NormArgs& a, F&& f) {
  if (a.dt == DC_F32) return f(float{}, float{});
  return a.gdt == DC_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}
template <typename F>
cudaError_t by_act(int act, F&& f) {
  return act == DC_ACT_SILU ? f(Int<1>{}) : act == DC_ACT_GELU ? f(Int<2>{}) : f(Int<0>{});
}
template <typename T, typename F>
cudaError_t by_width(int v, F&& f) {
  if (v == VecOf<T>::n) return f(Int<VecOf<T>::n>{});
  if (sizeof(T) == 2 && v == 4) return f(Int<4>{});
  return f(Int<1>{});
}

}  // namespace dc
