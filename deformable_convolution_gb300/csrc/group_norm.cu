// Group norm with an activation, forward and backward, between deformable
// layers (no counterpart on the explainer page; the definitions are in the
// ABI header): how a call runs, and the three-launch form (statistics or sums
// of parts, their merging, the results) for units too large for a cluster and
// too few for the rest of the GPU.
#include <math.h>

#include "dc_norm.cuh"

namespace dc {
namespace {

constexpr int kThreads = 256;

Tiling make_tiling(const NormArgs& a) {
  Tiling t{};
  const int vec = a.dt == DC_BF16 ? 8 : 4;
  if (!a.nhwc) {
    const int vr = row_vectors(a.hw, a.hw % vec ? vec - 1 : 0, vec);
    t.lpr = 1;
    while (t.lpr < 32 && t.lpr < vr) t.lpr *= 2;
    t.parts = (int)ceil_div_ll(vr, 64 * t.lpr);
    t.seg = (int)ceil_div_ll(vr, t.parts);
    t.parts = (int)ceil_div_ll(vr, t.seg);
  } else {
    // 16 bytes, or 8 where only that much is of one group (or divides c)
    t.v = a.c % vec == 0 && (vec == 4 || a.cpg % 8 != 4) ? vec : a.c % 4 == 0 ? 4 : 1;
    t.cols = a.c / t.v;
    t.cb = t.cols < 32 ? t.cols : 32;
    t.rl = kThreads / t.cb;
    t.seg = 16 * t.rl;
    t.parts = (int)ceil_div_ll(a.hw, t.seg);
  }
  return t;
}

Shape make_shape(const NormArgs& a) {
  return Shape{a.n, a.c, a.groups, a.cpg, a.hw, a.act == DC_ACT_RELU ? 0.f : -INFINITY, a.eps, make_tiling(a)};
}

// Elements of row `row` in segment `part` (NCHW), pixels of part (NHWC).
template <bool NHWC, int VEC>
__device__ __forceinline__ int part_count(const Shape& s, long long row, int part) {
  if (NHWC) {
    const int left = s.hw - part * s.t.seg;
    return left < s.t.seg ? left : s.t.seg;
  }
  const int mis = (int)((row * s.hw) % VEC);
  long long lo = (long long)part * s.t.seg * VEC - mis, hi = lo + (long long)s.t.seg * VEC;
  if (lo < 0) lo = 0;
  if (hi > s.hw) hi = s.hw;
  return hi > lo ? (int)(hi - lo) : 0;
}

// One row segment of a warp's task: this lane's vectors v0 + k * lpr < v1.
template <int VEC>
struct RowTask {
  long long row, off;  // off: the row's first vector in elements (aligned)
  int mis, v0, v1, sub;
  bool live;
  __device__ RowTask(const Shape& s, long long task) {
    const int lane = threadIdx.x & 31, per = 32 / s.t.lpr;
    const long long blk = task / s.t.parts;
    const int part = (int)(task - blk * s.t.parts);
    row = blk * per + lane / s.t.lpr;
    sub = lane & (s.t.lpr - 1);
    live = row < (long long)s.n * s.c;
    const long long first = row * s.hw;
    mis = (int)(first % VEC);
    off = first - mis;
    v0 = part * s.t.seg;
    const int vr = row_vectors(s.hw, mis, VEC);
    v1 = live ? (v0 + s.t.seg < vr ? v0 + s.t.seg : vr) : v0;
  }
  // element range of vector v that lies in the row
  __device__ __forceinline__ void range(const Shape& s, int v, int* lo, int* hi) const {
    const long long e0 = (long long)v * VEC - mis, left = s.hw - e0;
    *lo = e0 < 0 ? (int)-e0 : 0;
    *hi = left < VEC ? (int)left : VEC;
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void load_row(const T* p, int lo, int hi, float* f) {
  if (lo == 0 && hi == VEC)
    load_vec<T, VEC>(p, f);
  else
    load_part<T, VEC>(p, lo, hi, f);
}

// ---------------------------------------------------------------- NCHW

template <typename T>
__global__ void __launch_bounds__(kThreads)
    stats_nchw(Shape s, const T* x, float2* part, long long tasks) {
  pdl_wait();
  constexpr int VEC = VecOf<T>::n;
  const long long task = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (task < tasks) {
    const RowTask<VEC> r(s, task);
    float n = 0.f, mean = 0.f, m2 = 0.f;
    for (int v = r.v0 + r.sub; v < r.v1; v += s.t.lpr) {
      int lo, hi;
      r.range(s, v, &lo, &hi);
      float f[VEC];
      load_row<T, VEC>(x + r.off + (long long)v * VEC, lo, hi, f);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum += f[e];
      const float cnt = (float)(hi - lo), mb = sum / cnt;
      float q = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e >= lo && e < hi) q += (f[e] - mb) * (f[e] - mb);
      merge(n, mean, m2, cnt, mb, q);
    }
    const float tot = row_sum(n, s.t.lpr);
    const float m = row_sum(n * mean, s.t.lpr) / fmaxf(tot, 1.f);
    const float q = row_sum(m2 + n * (mean - m) * (mean - m), s.t.lpr);
    if (r.live && r.sub == 0)
      part[(task % s.t.parts) * ((long long)s.n * s.c) + r.row] = make_float2(m, q);
  }
  pdl_release();
}

template <typename T, int ACT>
__global__ void __launch_bounds__(kThreads)
    apply_nchw(Shape s, const T* x, const float* gamma, const float* beta, const float* mean,
               const float* rstd, T* y, long long tasks) {
  pdl_wait();
  constexpr int VEC = VecOf<T>::n;
  const long long task = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (task < tasks) {
    const RowTask<VEC> r(s, task);
    if (r.live) {
      const int ch = (int)(r.row % s.c);
      const float mu = mean[r.row / s.cpg];
      const float a = rstd[r.row / s.cpg] * (gamma ? gamma[ch] : 1.f), b = beta ? beta[ch] : 0.f;
      for (int v = r.v0 + r.sub; v < r.v1; v += s.t.lpr) {
        int lo, hi;
        r.range(s, v, &lo, &hi);
        float f[VEC];
        load_row<T, VEC>(x + r.off + (long long)v * VEC, lo, hi, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = act_fwd<ACT>(fmaf(f[e] - mu, a, b), s.floor);
        if (lo == 0 && hi == VEC)
          store_vec<T, VEC>(y + r.off + (long long)v * VEC, f);
        else
          store_part<T, VEC>(y + r.off + (long long)v * VEC, lo, hi, f);
      }
    }
  }
  pdl_release();
}

template <typename T, typename TG, int ACT>
__global__ void __launch_bounds__(kThreads)
    sums_nchw(Shape s, const T* x, const TG* gy, const float* gamma, const float* beta,
              const float* mean, const float* rstd, float2* part, long long tasks) {
  pdl_wait();
  constexpr int VEC = VecOf<T>::n;
  const long long task = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (task < tasks) {
    const RowTask<VEC> r(s, task);
    float sa = 0.f, sb = 0.f;
    if (r.live) {
      const int ch = (int)(r.row % s.c);
      const float mu = mean[r.row / s.cpg], rs = rstd[r.row / s.cpg];
      const float g = gamma ? gamma[ch] : 1.f, b = beta ? beta[ch] : 0.f;
      for (int v = r.v0 + r.sub; v < r.v1; v += s.t.lpr) {
        int lo, hi;
        r.range(s, v, &lo, &hi);
        float f[VEC], d[VEC];
        load_row<T, VEC>(x + r.off + (long long)v * VEC, lo, hi, f);
        load_row<TG, VEC>(gy + r.off + (long long)v * VEC, lo, hi, d);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (e >= lo && e < hi) {
            const float xh = (f[e] - mu) * rs;
            const float dz = act_bwd<ACT>(fmaf(xh, g, b), d[e], s.floor);
            sa += dz;
            sb = fmaf(dz, xh, sb);
          }
      }
    }
    sa = row_sum(sa, s.t.lpr);
    sb = row_sum(sb, s.t.lpr);
    if (r.live && r.sub == 0)
      part[(task % s.t.parts) * ((long long)s.n * s.c) + r.row] = make_float2(sa, sb);
  }
  pdl_release();
}

template <typename T, typename TG, int ACT>
__global__ void __launch_bounds__(kThreads)
    apply_bwd_nchw(Shape s, const T* x, const TG* gy, const float* gamma, const float* beta,
                   const float* mean, const float* rstd, const float2* coef, T* gx,
                   long long tasks) {
  pdl_wait();
  constexpr int VEC = VecOf<T>::n;
  const long long task = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (task < tasks) {
    const RowTask<VEC> r(s, task);
    if (r.live) {
      const int ch = (int)(r.row % s.c);
      const float mu = mean[r.row / s.cpg], rs = rstd[r.row / s.cpg];
      const float g = gamma ? gamma[ch] : 1.f, b = beta ? beta[ch] : 0.f;
      const float2 k = coef[r.row / s.cpg];
      for (int v = r.v0 + r.sub; v < r.v1; v += s.t.lpr) {
        int lo, hi;
        r.range(s, v, &lo, &hi);
        float f[VEC], d[VEC];
        load_row<T, VEC>(x + r.off + (long long)v * VEC, lo, hi, f);
        load_row<TG, VEC>(gy + r.off + (long long)v * VEC, lo, hi, d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (f[e] - mu) * rs;
          const float dz = act_bwd<ACT>(fmaf(xh, g, b), d[e], s.floor);
          f[e] = rs * (fmaf(g, dz, -k.x) - xh * k.y);
        }
        if (lo == 0 && hi == VEC)
          store_vec<T, VEC>(gx + r.off + (long long)v * VEC, f);
        else
          store_part<T, VEC>(gx + r.off + (long long)v * VEC, lo, hi, f);
      }
    }
  }
  pdl_release();
}

// ---------------------------------------------------------------- NHWC

// This thread's column of a block and its pixels p0 + k * rl < p1.
template <int V>
struct ColTask {
  long long base;  // of the image's first pixel, plus the column's channel
  int img, part, ch, p0, p1, lane;
  bool live;
  __device__ explicit ColTask(const Shape& s) {
    img = blockIdx.x / s.t.parts;
    part = blockIdx.x % s.t.parts;
    const int col = blockIdx.y * s.t.cb + threadIdx.x % s.t.cb;
    lane = threadIdx.x / s.t.cb;
    live = lane < s.t.rl && col < s.t.cols;
    ch = col * V;
    base = (long long)img * s.hw * s.c + ch;
    p0 = part * s.t.seg + lane;
    const int end = part * s.t.seg + s.t.seg;
    p1 = live ? (end < s.hw ? end : s.hw) : p0;
  }
};

// val[e] summed over the block's pixel lanes, in every thread of the column.
template <int V>
__device__ __forceinline__ void col_sum(const Shape& s, bool live, float* val, float* sm) {
  const int width = s.t.cb * V;
  __syncthreads();
  if (threadIdx.x < s.t.cb * s.t.rl) {
    const int at = threadIdx.x / s.t.cb * width + threadIdx.x % s.t.cb * V;
#pragma unroll
    for (int e = 0; e < V; ++e) sm[at + e] = live ? val[e] : 0.f;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += kThreads) {
    float t = 0.f;
    for (int l = 0; l < s.t.rl; ++l) t += sm[l * width + i];
    sm[i] = t;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < V; ++e) val[e] = sm[threadIdx.x % s.t.cb * V + e];
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) stats_nhwc(Shape s, const T* x, float2* part) {
  pdl_wait();
  __shared__ float sm[kThreads * V];
  const ColTask<V> r(s);
  float n = 0.f, mean[V] = {}, m2[V] = {};
  constexpr int kBatch = 4;
  for (int p = r.p0; p < r.p1; p += kBatch * s.t.rl) {
    float f[kBatch][V];
    float cnt = 0.f;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int q = p + k * s.t.rl;
      if (q < r.p1) {
        load_vec<T, V>(x + r.base + (long long)q * s.c, f[k]);
        cnt += 1.f;
      }
    }
    const float w = 1.f / cnt, t = n + cnt, wn = cnt / t;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float sum = 0.f, q2 = 0.f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k < (int)cnt) sum += f[k][e];
      const float mb = sum * w;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k < (int)cnt) q2 += (f[k][e] - mb) * (f[k][e] - mb);
      const float d = mb - mean[e];
      mean[e] += d * wn;
      m2[e] += q2 + d * d * n * wn;
    }
    n = t;
  }
  const float total = (float)part_count<true, 1>(s, 0, r.part);
  float m[V];
#pragma unroll
  for (int e = 0; e < V; ++e) m[e] = n * mean[e];
  col_sum<V>(s, r.live, m, sm);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    m[e] /= total;
    m2[e] += n * (mean[e] - m[e]) * (mean[e] - m[e]);
  }
  col_sum<V>(s, r.live, m2, sm);
  if (r.live && r.lane == 0) {
    float2* to = part + ((long long)r.part * s.n + r.img) * s.c + r.ch;
#pragma unroll
    for (int e = 0; e < V; ++e) to[e] = make_float2(m[e], m2[e]);
  }
  pdl_release();
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads)
    apply_nhwc(Shape s, const T* x, const float* gamma, const float* beta, const float* mean,
               const float* rstd, T* y) {
  pdl_wait();
  const ColTask<V> r(s);
  if (r.live) {
    float mu[V], a[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const long long g = (long long)r.img * s.groups + (r.ch + e) / s.cpg;
      mu[e] = mean[g];
      a[e] = rstd[g] * (gamma ? gamma[r.ch + e] : 1.f);
      b[e] = beta ? beta[r.ch + e] : 0.f;
    }
    for (int p = r.p0; p < r.p1; p += s.t.rl) {
      float f[V];
      load_vec<T, V>(x + r.base + (long long)p * s.c, f);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = act_fwd<ACT>(fmaf(f[e] - mu[e], a[e], b[e]), s.floor);
      store_vec<T, V>(y + r.base + (long long)p * s.c, f);
    }
  }
  pdl_release();
}

template <typename T, typename TG, int V, int ACT>
__global__ void __launch_bounds__(kThreads)
    sums_nhwc(Shape s, const T* x, const TG* gy, const float* gamma, const float* beta,
              const float* mean, const float* rstd, float2* part) {
  pdl_wait();
  __shared__ float sm[kThreads * V];
  const ColTask<V> r(s);
  float sa[V] = {}, sb[V] = {};
  if (r.live) {
    float mu[V], rs[V], g[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const long long at = (long long)r.img * s.groups + (r.ch + e) / s.cpg;
      mu[e] = mean[at];
      rs[e] = rstd[at];
      g[e] = gamma ? gamma[r.ch + e] : 1.f;
      b[e] = beta ? beta[r.ch + e] : 0.f;
    }
    for (int p = r.p0; p < r.p1; p += s.t.rl) {
      float f[V], d[V];
      load_vec<T, V>(x + r.base + (long long)p * s.c, f);
      load_vec<TG, V>(gy + r.base + (long long)p * s.c, d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xh = (f[e] - mu[e]) * rs[e];
        const float dz = act_bwd<ACT>(fmaf(xh, g[e], b[e]), d[e], s.floor);
        sa[e] += dz;
        sb[e] = fmaf(dz, xh, sb[e]);
      }
    }
  }
  col_sum<V>(s, r.live, sa, sm);
  col_sum<V>(s, r.live, sb, sm);
  if (r.live && r.lane == 0) {
    float2* to = part + ((long long)r.part * s.n + r.img) * s.c + r.ch;
#pragma unroll
    for (int e = 0; e < V; ++e) to[e] = make_float2(sa[e], sb[e]);
  }
  pdl_release();
}

template <typename T, typename TG, int V, int ACT>
__global__ void __launch_bounds__(kThreads)
    apply_bwd_nhwc(Shape s, const T* x, const TG* gy, const float* gamma, const float* beta,
                   const float* mean, const float* rstd, const float2* coef, T* gx) {
  pdl_wait();
  const ColTask<V> r(s);
  if (r.live) {
    float mu[V], rs[V], g[V], b[V];
    float2 k[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const long long at = (long long)r.img * s.groups + (r.ch + e) / s.cpg;
      mu[e] = mean[at];
      rs[e] = rstd[at];
      k[e] = coef[at];
      g[e] = gamma ? gamma[r.ch + e] : 1.f;
      b[e] = beta ? beta[r.ch + e] : 0.f;
    }
    for (int p = r.p0; p < r.p1; p += s.t.rl) {
      float f[V], d[V];
      load_vec<T, V>(x + r.base + (long long)p * s.c, f);
      load_vec<TG, V>(gy + r.base + (long long)p * s.c, d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xh = (f[e] - mu[e]) * rs[e];
        const float dz = act_bwd<ACT>(fmaf(xh, g[e], b[e]), d[e], s.floor);
        f[e] = rs[e] * (fmaf(g[e], dz, -k[e].x) - xh * k[e].y);
      }
      store_vec<T, V>(gx + r.base + (long long)p * s.c, f);
    }
  }
  pdl_release();
}

// ---------------------------------------------------------------- merging
// part[p][image * c + channel], both layouts.

// One warp for each group of each image.
template <bool NHWC, int VEC>
__global__ void __launch_bounds__(kThreads)
    merge_stats(Shape s, const float2* part, float* mean, float* rstd) {
  pdl_wait();
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit < (long long)s.n * s.groups) {
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)s.n * s.c, row0 = unit * s.cpg;
    const long long entries = (long long)s.cpg * s.t.parts;
    const float total = (float)s.hw * (float)s.cpg;
    float sum = 0.f;
    for (long long i = lane; i < entries; i += 32) {
      const int p = (int)(i / s.cpg);
      const long long row = row0 + i % s.cpg;
      sum += (float)part_count<NHWC, VEC>(s, row, p) * part[p * rows + row].x;
    }
    const float m = warp_sum(sum) / total;
    float q = 0.f;
    for (long long i = lane; i < entries; i += 32) {
      const int p = (int)(i / s.cpg);
      const long long row = row0 + i % s.cpg;
      const float2 e = part[p * rows + row];
      const float d = e.x - m;
      q += e.y + (float)part_count<NHWC, VEC>(s, row, p) * d * d;
    }
    q = warp_sum(q);
    if (lane == 0) {
      mean[unit] = m;
      rstd[unit] = 1.f / sqrtf(q / total + s.eps);
    }
  }
  pdl_release();
}

// One warp for each group of each image: chan = the sums of each channel of
// each image, coef = (s1, s2).
__global__ void __launch_bounds__(kThreads)
    merge_sums(Shape s, const float2* part, const float* gamma, float2* chan, float2* coef) {
  pdl_wait();
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit < (long long)s.n * s.groups) {
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)s.n * s.c, row0 = unit * s.cpg;
    float a = 0.f, b = 0.f;
    for (int i = lane; i < s.cpg; i += 32) {
      float ca = 0.f, cb = 0.f;
      for (int p = 0; p < s.t.parts; ++p) {
        const float2 e = part[p * rows + row0 + i];
        ca += e.x;
        cb += e.y;
      }
      chan[row0 + i] = make_float2(ca, cb);
      const float g = gamma ? gamma[(row0 + i) % s.c] : 1.f;
      a = fmaf(g, ca, a);
      b = fmaf(g, cb, b);
    }
    a = warp_sum(a);
    b = warp_sum(b);
    const float total = (float)s.hw * (float)s.cpg;
    if (lane == 0) coef[unit] = make_float2(a / total, b / total);
  }
  pdl_release();
}

// grad_gamma and grad_beta from `rows` rows of c channel sums: 32 channels a
// block, 32 lanes of rows each, added in a fixed order.
__global__ void __launch_bounds__(1024)
    sum_images(long long rows, int c, const float2* chan, float* ggamma, float* gbeta) {
  pdl_wait();
  pdl_release();
  __shared__ float2 sm[32][33];
  const int ch = blockIdx.x * 32 + (threadIdx.x & 31), lane = threadIdx.x >> 5;
  float a = 0.f, b = 0.f;
  if (ch < c)
#pragma unroll 4
    for (long long i = lane; i < rows; i += 32) {
      const float2 e = chan[i * c + ch];
      a += e.x;
      b += e.y;
    }
  sm[lane][threadIdx.x & 31] = make_float2(a, b);
  __syncthreads();
  // warp w sums channel w over the lanes
  const float2 e = sm[threadIdx.x & 31][lane];
  a = warp_sum(e.x);
  b = warp_sum(e.y);
  const int to = blockIdx.x * 32 + lane;
  if ((threadIdx.x & 31) == 0 && to < c) {
    if (gbeta) gbeta[to] = a;
    if (ggamma) ggamma[to] = b;
  }
}

// ---------------------------------------------------------------- launching

template <typename K, typename... A>
cudaError_t launch(K kern, dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
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

constexpr int kSms = 152;

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

constexpr int kBlockBytes = 92 * 1024;  // most of a unit in a block: two blocks to an SM
constexpr int kFourBytes = 50 * 1024;   // four blocks to an SM
constexpr int kLeastBytes = 16 * 1024;  // not split further to make more blocks

// Blocks of a unit of `bytes`: enough that it fits, and that every SM gets two,
// as long as a block keeps work worth its launch.  The backward, whose blocks
// compute for longer, overlaps better as four to an SM where the cluster stays
// small (stack's 256 units of 150 KB: 15.6 us as three blocks of 50 KB, 18.6
// as two of 75).
int cluster_of(double bytes, long long units, bool backward) {
  long long k = (long long)ceil(bytes / kBlockBytes), most = (long long)(bytes / kLeastBytes);
  const long long four = (long long)ceil(bytes / kFourBytes);
  if (backward && four <= 8) k = four;
  long long spread = ceil_div_ll(2 * kSms, units);
  if (spread > most) spread = most;
  if (k < spread) k = spread;
  return (int)(k < 1 ? 1 : k > kMaxCluster ? kMaxCluster : k);
}
// Threads of a block for so many vectors: eight each.
int threads_of(double vectors) {
  const double t = vectors / 8;
  return t >= kTeam ? kTeam : t <= 64 ? 64 : (int)ceil(t / 32) * 32;
}

NormPlan make_plan(const NormArgs& a, bool backward) {
  NormPlan p{};
  p.s = make_shape(a);
  p.parts = 1;
  if (a.n == 0) return p;
  const int vec = a.dt == DC_BF16 ? 8 : 4, elt = a.dt == DC_BF16 ? 2 : 4;
  const bool keep = keep_dz(a.gdt == DC_F32, a.act == DC_ACT_SILU || a.act == DC_ACT_GELU);
  // 16-byte pieces of a held vector of x, and of one of grad_y
  const int planes = 1 + (backward ? (keep && a.dt == DC_BF16 ? 2 : 1) : 0);
  const long long groups = (long long)a.n * a.groups;
  if (!a.nhwc) {
    Tiling t{};
    const int vr = row_vectors(a.hw, a.hw % vec ? vec - 1 : 0, vec);
    t.lpr = 1;
    while (t.lpr < 32 && t.lpr < vr) t.lpr *= 2;
    const long long blks = ceil_div_ll(a.cpg, 32 / t.lpr);
    const double bytes = (double)a.cpg * vr * 16 * planes;
    RowTeam& r = p.row;
    r.cluster = cluster_of(bytes, groups, backward);
    const long long run = (long long)a.cpg * vr;
    if (!backward && a.hw % vec == 0 && run < 1 << 30) {
      r.span = (int)ceil_div_ll(run, r.cluster);
      r.warps = threads_of(r.span) / 32;
      if (r.warps * 32 > r.span) r.warps = (int)ceil_div_ll(r.span, 32);
      r.units = 1;
      if (r.cluster == 1)
        while (r.units * r.warps < 4 && groups / (2 * r.units) >= 4 * kSms) r.units *= 2;
      const int threads = 32 * r.warps;
      r.step_c = threads / vr;
      r.step_v = threads % vr;
      r.slots = (int)ceil_div_ll(r.span, threads);
      const long long slot = 16LL * threads * r.units;
      r.held = slot * r.slots <= kBlockBytes ? r.slots : (int)(kBlockBytes / slot);
      if (r.held < r.slots && groups * r.cluster < kSms) return p;
      p.threads = threads * r.units;
      p.smem = (size_t)(slot * r.held);
      p.team = true;
      p.blocks = (unsigned)(ceil_div_ll(groups, r.units) * r.cluster);
      return p;
    }
    // segments of a row: until every SM has 16 warps, or four vectors a lane are left
    t.parts = 1;
    while (groups * blks * t.parts < 16 * kSms && ceil_div_ll(vr, t.parts + 1) >= 4 * t.lpr)
      ++t.parts;
    long long tasks = blks * t.parts;
    int warps = (int)ceil_div_ll(tasks, r.cluster);
    if (warps > 16) warps = 16;
    // no more of a row in a task than a block can hold
    const int slots = kBlockBytes / (warps * 32 * 16 * planes);
    if (ceil_div_ll(vr, t.parts) > (long long)slots * t.lpr)
      t.parts = (int)ceil_div_ll(vr, (long long)slots * t.lpr);
    t.seg = (int)ceil_div_ll(vr, t.parts);
    t.parts = (int)ceil_div_ll(vr, t.seg);
    tasks = blks * t.parts;
    if (tasks > 1 << 20) return p;
    if (r.cluster > tasks) r.cluster = (int)tasks;
    r.tasks = (int)tasks;
    r.rounds = (int)ceil_div_ll(tasks, r.cluster * warps);
    r.warps = (int)ceil_div_ll(tasks, (long long)r.cluster * r.rounds);
    r.units = 1;
    if (r.cluster == 1)
      while (r.units * r.warps < 4 && groups / (2 * r.units) >= 4 * kSms) r.units *= 2;
    p.threads = 32 * r.warps * r.units;
    r.slots = (int)ceil_div_ll(t.seg, t.lpr);
    const long long slot = (long long)p.threads * 16 * planes * r.slots;
    r.held = slot * r.rounds <= kBlockBytes ? r.rounds : (int)(kBlockBytes / slot);
    // a unit that must be read twice, by too few blocks: the form with more
    if (r.held < r.rounds && groups * r.cluster < kSms) return p;
    p.smem = (size_t)(slot * r.held);
    p.team = true;
    p.s.t = t;
    p.blocks = (unsigned)(ceil_div_ll(groups, r.units) * r.cluster);
    p.parts = t.parts;
    return p;
  }
  const int v = p.s.t.v;
  const long long base = (long long)a.cpg / gcd(a.cpg, v) * v;
  if (base / v > 256) return p;
  const int slices_most = (int)(a.c / base);
  const int held_bytes = v * (elt + (backward ? (keep ? 4 : 2) : 0));  // of a pixel's column
  ColTeam& c = p.col;
  // the narrowest slice of 128 bytes a pixel, or of 64 where that leaves few
  // blocks or does not fit in a cluster
  for (int bytes = 128; bytes >= 64; bytes /= 2) {
    int m = 1;
    while (m < slices_most && (m * base * elt < bytes || slices_most % m)) ++m;
    while (m > 1 && (m * base / v > 256 || m * base / a.cpg > kMaxGroups || slices_most % m)) --m;
    c.width = (int)(m * base);
    c.slices = a.c / c.width;
    c.cb = c.width / v;
    c.ng = c.width / a.cpg;
    c.cluster = cluster_of((double)a.hw * c.cb * held_bytes, (long long)a.n * c.slices, backward);
    if ((long long)a.n * c.slices * c.cluster >= 2 * kSms &&
        (double)a.hw * c.cb * held_bytes <= (double)kMaxCluster * kBlockBytes)
      break;
  }
  if (c.ng > kMaxGroups) return p;
  const long long units = (long long)a.n * c.slices;
  if (units * c.cluster > INT_MAX) return p;
  c.span = (int)ceil_div_ll(a.hw, c.cluster);
  const int most = threads_of((double)c.span * c.cb);
  c.rl = most / c.cb;
  if (c.rl < 1) c.rl = 1;
  if (c.rl > c.span) c.rl = c.span;
  c.slots = (int)ceil_div_ll(c.span, c.rl);
  p.threads = (int)ceil_div_ll((long long)c.rl * c.cb, 32) * 32;
  const long long slot = (long long)p.threads * held_bytes;
  const bool copies = v * elt >= 4;  // (an asynchronous copy moves 4 bytes at least)
  c.held = !copies ? 0 : slot * c.slots <= kBlockBytes ? c.slots : (int)(kBlockBytes / slot);
  if (c.held < c.slots && units * c.cluster < kSms) return p;
  c.rows = 32 % c.cb ? c.rl : p.threads / 32;
  p.smem = (size_t)(slot * c.held) + (size_t)c.cluster * c.ng * (backward ? 2 : 3) * sizeof(float);
  if (backward) p.smem += (size_t)c.rows * c.width * sizeof(float2);
  p.team = true;
  p.blocks = (unsigned)(units * c.cluster);
  p.parts = c.cluster;
  return p;
}

long long row_tasks(const Shape& s) {
  return ceil_div_ll((long long)s.n * s.c, 32 / s.t.lpr) * s.t.parts;
}
dim3 row_grid(const Shape& s) { return dim3((unsigned)ceil_div_ll(row_tasks(s), kThreads / 32)); }
dim3 col_grid(const Shape& s) {
  return dim3((unsigned)s.t.parts * (unsigned)s.n, (unsigned)ceil_div_ll(s.t.cols, s.t.cb));
}
dim3 unit_grid(const Shape& s) {
  return dim3((unsigned)ceil_div_ll((long long)s.n * s.groups, kThreads / 32));
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// The workspace: parts, then mean and rstd (forward) or the channels' sums
// and the groups' coefficients (backward).
size_t part_bytes(const Shape& s) {
  return round256((size_t)s.t.parts * s.n * s.c * sizeof(float2));
}

}  // namespace

bool norm_supported(const NormArgs& a) {
  constexpr long long kGrid = (1LL << 31) - 1;
  if (a.c > 1 << 20 || (long long)a.n * a.c > kGrid) return false;
  const Shape s = make_shape(a);
  return a.nhwc ? (long long)s.t.parts * a.n <= kGrid : row_tasks(s) <= kGrid;
}

size_t norm_workspace_bytes(const NormArgs& a, bool backward) {
  if (a.n == 0) return 0;
  const NormPlan p = make_plan(a, backward);
  if (p.team)
    return backward ? round256((size_t)p.parts * a.n * a.c * sizeof(float2)) : 0;
  const Shape& s = p.s;
  const size_t units = (size_t)a.n * a.groups;
  if (!backward) return part_bytes(s) + round256(units * sizeof(float2));
  return part_bytes(s) + round256((size_t)a.n * a.c * sizeof(float2)) +
         round256(units * sizeof(float2));
}

bool norm_one_launch(const NormArgs& a, bool backward) { return make_plan(a, backward).team; }

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
  const NormPlan p = make_plan(a, false);
  return a.nhwc ? launch_team_nhwc(p, a, false, st) : launch_team_nchw(p, a, false, st);
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st) {
  const NormPlan p = make_plan(a, true);
  return a.nhwc ? launch_team_nhwc(p, a, true, st) : launch_team_nchw(p, a, true, st);
}

namespace {
float* ws_mean(const NormArgs& a, const Shape& s) {
  return a.mean ? a.mean : reinterpret_cast<float*>(a.ws + part_bytes(s));
}
float* ws_rstd(const NormArgs& a, const Shape& s) {
  return a.rstd ? a.rstd
                : reinterpret_cast<float*>(a.ws + part_bytes(s)) + (size_t)a.n * a.groups;
}
float2* ws_chan(const NormArgs& a, const Shape& s) {
  return reinterpret_cast<float2*>(a.ws + part_bytes(s));
}
float2* ws_coef(const NormArgs& a, const Shape& s) {
  return reinterpret_cast<float2*>(a.ws + part_bytes(s) +
                                   round256((size_t)a.n * a.c * sizeof(float2)));
}
}  // namespace

cudaError_t launch_norm_stats(const NormArgs& a, cudaStream_t st) {
  const Shape s = make_shape(a);
  float2* part = reinterpret_cast<float2*>(a.ws);
  return by_dtype(a.dt, [&](auto t) {
    using T = decltype(t);
    const T* x = static_cast<const T*>(a.x);
    if (!a.nhwc) return launch(stats_nchw<T>, row_grid(s), kThreads, st, s, x, part, row_tasks(s));
    return by_width<T>(s.t.v, [&](auto w) {
      return launch(stats_nhwc<T, decltype(w)::value>, col_grid(s), kThreads, st, s, x, part);
    });
  });
}

cudaError_t launch_norm_merge(const NormArgs& a, cudaStream_t st) {
  const Shape s = make_shape(a);
  const float2* part = reinterpret_cast<const float2*>(a.ws);
  float *m = ws_mean(a, s), *r = ws_rstd(a, s);
  if (a.nhwc) return launch(merge_stats<true, 1>, unit_grid(s), kThreads, st, s, part, m, r);
  if (a.dt == DC_BF16)
    return launch(merge_stats<false, 8>, unit_grid(s), kThreads, st, s, part, m, r);
  return launch(merge_stats<false, 4>, unit_grid(s), kThreads, st, s, part, m, r);
}

cudaError_t launch_norm_apply(const NormArgs& a, cudaStream_t st) {
  const Shape s = make_shape(a);
  const float *m = ws_mean(a, s), *r = ws_rstd(a, s);
  return by_dtype(a.dt, [&](auto t) {
    using T = decltype(t);
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.y);
    return by_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      if (!a.nhwc)
        return launch(apply_nchw<T, ACT>, row_grid(s), kThreads, st, s, x, a.gamma, a.beta, m, r,
                      y, row_tasks(s));
      return by_width<T>(s.t.v, [&](auto w) {
        return launch(apply_nhwc<T, decltype(w)::value, ACT>, col_grid(s), kThreads, st, s, x,
                      a.gamma, a.beta, m, r, y);
      });
    });
  });
}

cudaError_t launch_norm_sums(const NormArgs& a, cudaStream_t st) {
  const Shape s = make_shape(a);
  float2* part = reinterpret_cast<float2*>(a.ws);
  const float *m = a.mean, *r = a.rstd;
  return by_dtypes(a, [&](auto t, auto g) {
    using T = decltype(t);
    using TG = decltype(g);
    const T* x = static_cast<const T*>(a.x);
    const TG* gy = static_cast<const TG*>(a.gy);
    return by_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      if (!a.nhwc)
        return launch(sums_nchw<T, TG, ACT>, row_grid(s), kThreads, st, s, x, gy, a.gamma, a.beta,
                      m, r, part, row_tasks(s));
      return by_width<T>(s.t.v, [&](auto w) {
        return launch(sums_nhwc<T, TG, decltype(w)::value, ACT>, col_grid(s), kThreads, st, s, x,
                      gy, a.gamma, a.beta, m, r, part);
      });
    });
  });
}

cudaError_t launch_norm_merge_bwd(const NormArgs& a, cudaStream_t st) {
  const Shape s = make_shape(a);
  return launch(merge_sums, unit_grid(s), kThreads, st, s, reinterpret_cast<const float2*>(a.ws),
                a.gamma, ws_chan(a, s), ws_coef(a, s));
}

cudaError_t launch_norm_apply_bwd(const NormArgs& a, cudaStream_t st) {
  const Shape s = make_shape(a);
  const float2* coef = ws_coef(a, s);
  const float *m = a.mean, *r = a.rstd;
  return by_dtypes(a, [&](auto t, auto g) {
    using T = decltype(t);
    using TG = decltype(g);
    const T* x = static_cast<const T*>(a.x);
    const TG* gy = static_cast<const TG*>(a.gy);
    T* gx = static_cast<T*>(a.gx);
    return by_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      if (!a.nhwc)
        return launch(apply_bwd_nchw<T, TG, ACT>, row_grid(s), kThreads, st, s, x, gy, a.gamma,
                      a.beta, m, r, coef, gx, row_tasks(s));
      return by_width<T>(s.t.v, [&](auto w) {
        return launch(apply_bwd_nhwc<T, TG, decltype(w)::value, ACT>, col_grid(s), kThreads, st, s,
                      x, gy, a.gamma, a.beta, m, r, coef, gx);
      });
    });
  });
}

cudaError_t launch_norm_params(const NormArgs& a, cudaStream_t st) {
  const NormPlan p = make_plan(a, true);
  const float2* chan = !a.n     ? nullptr
                       : p.team ? reinterpret_cast<const float2*>(a.ws)
                                : ws_chan(a, p.s);
  return launch(sum_images, dim3((unsigned)ceil_div_ll(a.c, 32)), 1024, st,
                (long long)p.parts * a.n, a.c, chan, a.ggamma, a.gbeta);
}

}  // namespace dc
