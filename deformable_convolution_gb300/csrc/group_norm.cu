// Group norm with an activation, forward and backward, between deformable
// layers (no counterpart on the explainer page; the definitions are in the
// ABI header).
//
// Statistics.  A thread keeps (count, mean, M2) of what it has read, M2 the
// sum of squared distances from its own mean: a batch of vectors in registers
// is averaged first and its squared distances summed second, and two such
// triples merge exactly,
//   d = mb - ma, m = ma + d nb / (na + nb), M2 = M2a + M2b + d^2 na nb / (na + nb),
// so no sum of squares about a far-off origin is ever formed (a large mean
// over a small spread costs no digits).
#include "dc_common.cuh"

namespace dc {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct VecOf {
  static constexpr int n = 16 / sizeof(T);
};

// V elements at p (aligned to V * sizeof(T) bytes) as floats.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
  if constexpr (V * sizeof(T) == 32) {
    load_vec<T, V / 2>(p, f);
    load_vec<T, V / 2>(p + V / 2, f + V / 2);
  } else if constexpr (sizeof(T) == 4) {
    if constexpr (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = p[e];
    }
  } else if constexpr (V == 1) {
    f[0] = to_f(p[0]);
  } else {
    uint32_t w[V / 2];
    if constexpr (V == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      static_assert(V == 4);
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}

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

__device__ __forceinline__ float act_fwd(float z, int act) {
  switch (act) {
    case DC_ACT_RELU: return z <= 0.f ? 0.f : z;
    case DC_ACT_SILU: return __fdividef(z, 1.f + __expf(-z));
    case DC_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  }
  return z;
}

// act'(z)
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case DC_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case DC_ACT_SILU: {
      const float sg = __fdividef(1.f, 1.f + __expf(-z));
      return sg * (1.f + z * (1.f - sg));
    }
    case DC_ACT_GELU:
      return 0.5f * (1.f + erff(z * 0.70710678118654752f)) +
             z * __expf(-0.5f * z * z) * 0.39894228040143268f;
  }
  return 1.f;
}

// ---------------------------------------------------------------- the tiling
// NCHW: a row is one channel of one image, hw consecutive elements; `lpr`
// lanes of a warp walk a row's 16-byte vectors (the first and last may hang
// over the row's ends), a warp takes 32 / lpr rows, and a long row is cut into
// `parts` segments of `seg` vectors.
// NHWC: a thread keeps one vector of v channels and walks pixels; a block
// takes cb such columns and `seg` pixels of an image.
struct Tiling {
  int parts, seg;
  int lpr;             // NCHW
  int v, cols, cb, rl;  // NHWC: vector width, vectors of a pixel, of a block, pixel lanes
};

struct Shape {
  int n, c, groups, cpg, hw, act;
  float eps;
  Tiling t;
};

__host__ __device__ inline int row_vectors(int hw, int mis, int vec) {
  return (mis + hw + vec - 1) / vec;
}

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
    t.v = a.c % vec == 0 ? vec : a.dt == DC_BF16 && a.c % 4 == 0 ? 4 : 1;
    t.cols = a.c / t.v;
    t.cb = t.cols < 32 ? t.cols : 32;
    t.rl = kThreads / t.cb;
    t.seg = 16 * t.rl;
    t.parts = (int)ceil_div_ll(a.hw, t.seg);
  }
  return t;
}

Shape make_shape(const NormArgs& a) {
  return Shape{a.n, a.c, a.groups, a.cpg, a.hw, a.act, a.eps, make_tiling(a)};
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

__device__ __forceinline__ void merge(float& n, float& mean, float& m2, float nb, float mb,
                                      float m2b) {
  if (nb == 0.f) return;
  const float t = n + nb, d = mb - mean, w = nb / t;
  mean += d * w;
  m2 += m2b + d * d * n * w;
  n = t;
}

// Sum over the lpr lanes that share a row (lpr a power of two), in every lane.
__device__ __forceinline__ float row_sum(float v, int lpr) {
  for (int o = lpr >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float warp_sum(float v) { return row_sum(v, 32); }

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

template <typename T>
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
        for (int e = 0; e < VEC; ++e) f[e] = act_fwd(fmaf(f[e] - mu, a, b), s.act);
        if (lo == 0 && hi == VEC)
          store_vec<T, VEC>(y + r.off + (long long)v * VEC, f);
        else
          store_part<T, VEC>(y + r.off + (long long)v * VEC, lo, hi, f);
      }
    }
  }
  pdl_release();
}

template <typename T, typename TG>
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
            const float dz = d[e] * act_slope(fmaf(xh, g, b), s.act);
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

template <typename T, typename TG>
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
          const float dz = d[e] * act_slope(fmaf(xh, g, b), s.act);
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

template <typename T, int V>
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
      for (int e = 0; e < V; ++e) f[e] = act_fwd(fmaf(f[e] - mu[e], a[e], b[e]), s.act);
      store_vec<T, V>(y + r.base + (long long)p * s.c, f);
    }
  }
  pdl_release();
}

template <typename T, typename TG, int V>
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
        const float dz = d[e] * act_slope(fmaf(xh, g[e], b[e]), s.act);
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

template <typename T, typename TG, int V>
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
        const float dz = d[e] * act_slope(fmaf(xh, g[e], b[e]), s.act);
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

// ---------------------------------------------------------------- one launch
// A cluster of K blocks holds a unit (a group of an image; NHWC: a slice of
// whole groups) in registers from its statistics to its results: x (and
// grad_y) come from memory once.  What does not fit is read in `rounds`: the
// first passes over it leave it in L2, where the second finds it.  The blocks
// exchange their statistics by stores into each other's shared memory, one
// cluster barrier behind the loads.

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *p of the cluster's block `rank` = v
__device__ __forceinline__ void store_cluster(float* p, int rank, float v) {
  uint32_t to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(to)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
}

constexpr int kTeam = 512;        // most threads of a block
constexpr int kMaxCluster = 16;

// A vector as it lies in memory.
template <typename T, int V>
struct Raw {
  uint4 w[(V * sizeof(T) + 15) / 16];
};
template <typename T, int V>
__device__ __forceinline__ void load_raw(const T* p, Raw<T, V>* r) {
  constexpr int kBytes = V * sizeof(T);
  if constexpr (kBytes >= 16) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) r->w[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (kBytes == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r->w[0].x = v.x, r->w[0].y = v.y;
  } else if constexpr (sizeof(T) == 4) {
    r->w[0].x = __float_as_uint(p[0]);
  } else {
    r->w[0].x = *reinterpret_cast<const unsigned short*>(p);
  }
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, float* f) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.w);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = __uint_as_float(w[e]);
  } else if constexpr (V == 1) {
    f[0] = __uint_as_float(w[0] << 16);
  } else {
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}
// The elements [lo, hi) of a vector, zeros for the others.
template <typename T, int V>
__device__ __forceinline__ void load_raw_part(const T* p, int lo, int hi, Raw<T, V>* r) {
  float f[V];
  load_part<T, V>(p, lo, hi, f);
  uint32_t* w = reinterpret_cast<uint32_t*>(r->w);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = __float_as_uint(f[e]);
  } else {
#pragma unroll
    for (int e = 0; e < V / 2; ++e)
      w[e] = __float_as_uint(f[2 * e]) >> 16 | (__float_as_uint(f[2 * e + 1]) & 0xffff0000u);
  }
}

// The activation of a vector's values, one branch for all of them.
template <int V>
__device__ __forceinline__ void act_vec(float* f, int act) {
  switch (act) {
    case DC_ACT_RELU:
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = act_fwd(f[e], DC_ACT_RELU);
      break;
    case DC_ACT_SILU:
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = act_fwd(f[e], DC_ACT_SILU);
      break;
    case DC_ACT_GELU:
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = act_fwd(f[e], DC_ACT_GELU);
      break;
  }
}
// d *= act'(z)
template <int V>
__device__ __forceinline__ void slope_vec(const float* z, float* d, int act) {
  switch (act) {
    case DC_ACT_RELU:
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] = z[e] > 0.f ? d[e] : d[e] * 0.f;
      break;
    case DC_ACT_SILU:
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] *= act_slope(z[e], DC_ACT_SILU);
      break;
    case DC_ACT_GELU:
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] *= act_slope(z[e], DC_ACT_GELU);
      break;
  }
}

// NCHW: a unit's rows are cut into tasks as above, one to a warp and round.
struct RowTeam {
  int cluster, warps, units;  // blocks of a unit, warps of a unit in a block, units of a block
  int tasks, rounds;          // of a unit
};

// The task of a warp in round r: tasks are dealt over the cluster's warps.
template <int VEC, bool EVEN>
struct UnitTask {
  long long row, off;
  int ch, part, mis, v0, v1, sub;
  bool live;
  __device__ UnitTask(const Shape& s, unsigned unit, int t, int tasks) {
    const int lane = threadIdx.x & 31, per = 32 / s.t.lpr;
    const int blk = t / s.t.parts;
    part = t - blk * s.t.parts;
    const int local = blk * per + lane / s.t.lpr;
    sub = lane & (s.t.lpr - 1);
    live = t < tasks && local < s.cpg;
    row = (long long)unit * s.cpg + (live ? local : 0);
    ch = (int)(unit % (unsigned)s.groups) * s.cpg + (live ? local : 0);
    const long long first = row * s.hw;
    mis = EVEN ? 0 : (int)(first % VEC);
    off = first - mis;
    v0 = part * s.t.seg;
    const int vr = row_vectors(s.hw, mis, VEC);
    v1 = live ? (v0 + s.t.seg < vr ? v0 + s.t.seg : vr) : v0;
  }
  __device__ __forceinline__ void range(const Shape& s, int v, int* lo, int* hi) const {
    *lo = 0;
    *hi = VEC;
    if (!EVEN) {
      const long long e0 = (long long)v * VEC - mis, left = s.hw - e0;
      if (e0 < 0) *lo = (int)-e0;
      if (left < VEC) *hi = (int)left;
    }
  }
};

template <typename T, int VEC, bool EVEN, int NV, typename TASK>
__device__ __forceinline__ void load_task(const Shape& s, const TASK& k, const T* x,
                                          Raw<T, VEC>* raw) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = k.v0 + k.sub + i * s.t.lpr;
    if (v >= k.v1) continue;
    const T* p = x + k.off + (long long)v * VEC;
    int lo, hi;
    k.range(s, v, &lo, &hi);
    if (EVEN || (lo == 0 && hi == VEC))
      load_raw<T, VEC>(p, &raw[i]);
    else
      load_raw_part<T, VEC>(p, lo, hi, &raw[i]);
  }
}

// (n, mean, m2) merged with the warp's task: its mean first, then the squared
// distances from it.
template <typename T, int VEC, bool EVEN, int NV, typename TASK>
__device__ __forceinline__ void task_stats(const Shape& s, const TASK& k, const Raw<T, VEC>* raw,
                                           float& n, float& mean, float& m2) {
  float cnt = 0.f, sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = k.v0 + k.sub + i * s.t.lpr;
    if (v >= k.v1) continue;
    float f[VEC];
    unpack<T, VEC>(raw[i], f);
    int lo, hi;
    k.range(s, v, &lo, &hi);
    cnt += (float)(hi - lo);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum += f[e];
  }
  cnt = warp_sum(cnt);
  const float m = warp_sum(sum) / fmaxf(cnt, 1.f);
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = k.v0 + k.sub + i * s.t.lpr;
    if (v >= k.v1) continue;
    float f[VEC];
    unpack<T, VEC>(raw[i], f);
    int lo, hi;
    k.range(s, v, &lo, &hi);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (EVEN || (e >= lo && e < hi)) q = fmaf(f[e] - m, f[e] - m, q);
  }
  merge(n, mean, m2, cnt, m, warp_sum(q));
}

template <typename T, bool EVEN, int NV>
__global__ void __launch_bounds__(kTeam, 2)
    fwd_nchw(Shape s, RowTeam tm, const T* x, const float* gamma, const float* beta, T* y,
             float* mean_out, float* rstd_out) {
  constexpr int VEC = VecOf<T>::n;
  __shared__ float sn[256], sm[256], sq[256];
  const bool many = tm.cluster > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % tm.cluster, u = warp / tm.warps, w = warp - u * tm.warps;
  const unsigned unit = blockIdx.x / tm.cluster * tm.units + u;  // (n * c is below 2^31)
  const bool here = unit < (unsigned)s.n * s.groups;
  const int team = tm.cluster * tm.warps, tasks = here ? tm.tasks : 0;
  float n = 0.f, mean = 0.f, m2 = 0.f;
  Raw<T, VEC> raw[NV];
  // the rounds that stay in L2, then the one that stays in registers
  for (int r = tm.rounds - 1; r >= 0; --r) {
    const UnitTask<VEC, EVEN> k(s, here ? unit : 0, rank * tm.warps + w + r * team, tasks);
    load_task<T, VEC, EVEN, NV>(s, k, x, raw);
    task_stats<T, VEC, EVEN, NV>(s, k, raw, n, mean, m2);
  }
  // the unit's (count, mean, M2): one triple from each of its warps
  if (many) {
    cluster_wait();
    if (lane < tm.cluster) {
      const int at = rank * tm.warps + w;
      store_cluster(&sn[at], lane, n);
      store_cluster(&sm[at], lane, mean);
      store_cluster(&sq[at], lane, m2);
    }
    cluster_arrive();
    cluster_wait();
  } else {
    if (lane == 0) sn[warp] = n, sm[warp] = mean, sq[warp] = m2;
    __syncthreads();
  }
  const int first = many ? 0 : u * tm.warps;
  float sum = 0.f;
  for (int i = lane; i < team; i += 32) sum = fmaf(sn[first + i], sm[first + i], sum);
  const float total = (float)s.hw * (float)s.cpg;
  const float mu = warp_sum(sum) / total;
  float q = 0.f;
  for (int i = lane; i < team; i += 32) {
    const float d = sm[first + i] - mu;
    q += fmaf(sn[first + i] * d, d, sq[first + i]);
  }
  const float rs = 1.f / sqrtf(warp_sum(q) / total + s.eps);
  if (!here) return;
  if (rank == 0 && w == 0 && lane == 0) {
    if (mean_out) mean_out[unit] = mu;
    if (rstd_out) rstd_out[unit] = rs;
  }
  for (int r = 0; r < tm.rounds; ++r) {
    const UnitTask<VEC, EVEN> k(s, unit, rank * tm.warps + w + r * team, tasks);
    if (r) load_task<T, VEC, EVEN, NV>(s, k, x, raw);
    const float a = rs * (gamma ? gamma[k.ch] : 1.f), b = beta ? beta[k.ch] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = k.v0 + k.sub + i * s.t.lpr;
      if (v >= k.v1) continue;
      float f[VEC];
      unpack<T, VEC>(raw[i], f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = fmaf(f[e] - mu, a, b);
      act_vec<VEC>(f, s.act);
      int lo, hi;
      k.range(s, v, &lo, &hi);
      T* to = y + k.off + (long long)v * VEC;
      if (EVEN || (lo == 0 && hi == VEC))
        store_vec<T, VEC>(to, f);
      else
        store_part<T, VEC>(to, lo, hi, f);
    }
  }
}

template <typename T, typename TG, bool EVEN, int NV>
__global__ void __launch_bounds__(kTeam, 1)
    bwd_nchw(Shape s, RowTeam tm, const T* x, const TG* gy, const float* gamma, const float* beta,
             const float* mean, const float* rstd, T* gx, float2* part) {
  constexpr int VEC = VecOf<T>::n;
  __shared__ float sa[256], sb[256];
  const bool many = tm.cluster > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % tm.cluster, u = warp / tm.warps, w = warp - u * tm.warps;
  const unsigned unit = blockIdx.x / tm.cluster * tm.units + u;  // (n * c is below 2^31)
  const bool here = unit < (unsigned)s.n * s.groups;
  const int team = tm.cluster * tm.warps, tasks = here ? tm.tasks : 0;
  const float mu = here ? mean[unit] : 0.f, rs = here ? rstd[unit] : 0.f;
  Raw<T, VEC> raw[NV];
  Raw<TG, VEC> graw[NV];
  float ga = 0.f, gb = 0.f;
  for (int r = tm.rounds - 1; r >= 0; --r) {
    const UnitTask<VEC, EVEN> k(s, here ? unit : 0, rank * tm.warps + w + r * team, tasks);
    load_task<T, VEC, EVEN, NV>(s, k, x, raw);
    load_task<TG, VEC, EVEN, NV>(s, k, gy, graw);
    const float g = gamma ? gamma[k.ch] : 1.f, b = beta ? beta[k.ch] : 0.f;
    float a1 = 0.f, b1 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = k.v0 + k.sub + i * s.t.lpr;
      if (v >= k.v1) continue;
      float f[VEC], z[VEC], d[VEC];
      unpack<T, VEC>(raw[i], f);
      unpack<TG, VEC>(graw[i], d);
      int lo, hi;
      k.range(s, v, &lo, &hi);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        f[e] = (f[e] - mu) * rs;
        z[e] = fmaf(f[e], g, b);
      }
      slope_vec<VEC>(z, d, s.act);
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (EVEN || (e >= lo && e < hi)) {
          a1 += d[e];
          b1 = fmaf(d[e], f[e], b1);
        }
    }
    a1 = row_sum(a1, s.t.lpr);
    b1 = row_sum(b1, s.t.lpr);
    if (k.live && k.sub == 0) {
      part[(long long)k.part * s.n * s.c + k.row] = make_float2(a1, b1);
      ga = fmaf(g, a1, ga);
      gb = fmaf(g, b1, gb);
    }
  }
  ga = warp_sum(ga);
  gb = warp_sum(gb);
  if (many) {
    cluster_wait();
    if (lane < tm.cluster) {
      store_cluster(&sa[rank * tm.warps + w], lane, ga);
      store_cluster(&sb[rank * tm.warps + w], lane, gb);
    }
    cluster_arrive();
    cluster_wait();
  } else {
    if (lane == 0) sa[warp] = ga, sb[warp] = gb;
    __syncthreads();
  }
  const int first = many ? 0 : u * tm.warps;
  ga = gb = 0.f;
  for (int i = lane; i < team; i += 32) {
    ga += sa[first + i];
    gb += sb[first + i];
  }
  const float total = (float)s.hw * (float)s.cpg;
  const float s1 = warp_sum(ga) / total, s2 = warp_sum(gb) / total;
  if (!here) return;
  for (int r = 0; r < tm.rounds; ++r) {
    const UnitTask<VEC, EVEN> k(s, unit, rank * tm.warps + w + r * team, tasks);
    if (r) {
      load_task<T, VEC, EVEN, NV>(s, k, x, raw);
      load_task<TG, VEC, EVEN, NV>(s, k, gy, graw);
    }
    const float g = gamma ? gamma[k.ch] : 1.f, b = beta ? beta[k.ch] : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = k.v0 + k.sub + i * s.t.lpr;
      if (v >= k.v1) continue;
      float f[VEC], z[VEC], d[VEC];
      unpack<T, VEC>(raw[i], f);
      unpack<TG, VEC>(graw[i], d);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        f[e] = (f[e] - mu) * rs;
        z[e] = fmaf(f[e], g, b);
      }
      slope_vec<VEC>(z, d, s.act);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = rs * (fmaf(g, d[e], -s1) - f[e] * s2);
      int lo, hi;
      k.range(s, v, &lo, &hi);
      T* to = gx + k.off + (long long)v * VEC;
      if (EVEN || (lo == 0 && hi == VEC))
        store_vec<T, VEC>(to, f);
      else
        store_part<T, VEC>(to, lo, hi, f);
    }
  }
}

// NHWC: a unit is a slice of whole groups, `cb` vectors wide, of an image; a
// thread keeps one of its columns and walks pixels, `rl` threads to a column.
struct ColTeam {
  int cluster, slices, width;  // blocks of a unit, units of an image, channels of a unit
  int cb, rl, ng;              // ng: groups of a unit
  int rounds, nv;              // nv: pixels of a thread in a round
};
constexpr int kMaxGroups = 64;  // of a unit

template <int V>
struct UnitCol {
  long long base;
  int img, ch, col, lane, rank;
  bool live;
  __device__ UnitCol(const Shape& s, const ColTeam& tm) {
    const int id = blockIdx.x / tm.cluster;
    rank = blockIdx.x % tm.cluster;
    img = id / tm.slices;
    lane = threadIdx.x / tm.cb;
    col = threadIdx.x - lane * tm.cb;
    live = lane < tm.rl;
    ch = (id - img * tm.slices) * tm.width + col * V;
    base = (long long)img * s.hw * s.c + ch;
  }
  // pixel of vector i in round r, hw for none
  __device__ __forceinline__ int pixel(const Shape& s, const ColTeam& tm, int r, int i) const {
    const int p = (r * tm.cluster + rank) * (tm.rl * tm.nv) + i * tm.rl + lane;
    return i < tm.nv && live ? p : s.hw;
  }
};

template <typename T, int V, int NV>
__device__ __forceinline__ void load_col(const Shape& s, const ColTeam& tm, const UnitCol<V>& k,
                                         int r, const T* x, Raw<T, V>* raw) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = k.pixel(s, tm, r, i);
    if (p < s.hw) load_raw<T, V>(x + k.base + (long long)p * s.c, &raw[i]);
  }
}

// ONE: a vector's channels are all of one group; else channels are kept apart
// until the block's are merged.
template <typename T, int V, int NV, bool ONE>
__global__ void __launch_bounds__(kTeam, 2)
    fwd_nhwc(Shape s, ColTeam tm, const T* x, const float* gamma, const float* beta, T* y,
             float* mean_out, float* rstd_out) {
  constexpr int E = ONE ? 1 : V;
  __shared__ float2 ent[kTeam * E];
  __shared__ float cnts[kTeam];
  __shared__ float sn[kMaxCluster * kMaxGroups], sm[kMaxCluster * kMaxGroups],
      sq[kMaxCluster * kMaxGroups];
  const bool many = tm.cluster > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const UnitCol<V> k(s, tm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  Raw<T, V> raw[NV];
  float n = 0.f, mean[E] = {}, m2[E] = {};
  for (int r = tm.rounds - 1; r >= 0; --r) {
    load_col<T, V, NV>(s, tm, k, r, x, raw);
    float cnt = 0.f, sum[E] = {}, q[E] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (k.pixel(s, tm, r, i) >= s.hw) continue;
      float f[V];
      unpack<T, V>(raw[i], f);
      cnt += 1.f;
#pragma unroll
      for (int e = 0; e < V; ++e) sum[ONE ? 0 : e] += f[e];
    }
    if (cnt == 0.f) continue;
    const float w = 1.f / (ONE ? cnt * V : cnt);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[e] *= w;  // the means
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (k.pixel(s, tm, r, i) >= s.hw) continue;
      float f[V];
      unpack<T, V>(raw[i], f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = f[e] - sum[ONE ? 0 : e];
        q[ONE ? 0 : e] = fmaf(d, d, q[ONE ? 0 : e]);
      }
    }
    const float c = ONE ? cnt * V : cnt, t = n + c, wn = c / t;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float d = sum[e] - mean[e];
      mean[e] += d * wn;
      m2[e] += q[e] + d * d * n * wn;
    }
    n = t;
  }
  // the block's groups, a warp each
#pragma unroll
  for (int e = 0; e < E; ++e) ent[threadIdx.x * E + e] = make_float2(mean[e], m2[e]);
  cnts[threadIdx.x] = n;
  __syncthreads();
  if (many) cluster_wait();
  const int per = ONE ? s.cpg / V : s.cpg;  // entries of a group in a pixel lane
  for (int g = warp; g < tm.ng; g += warps) {
    float c = 0.f, sum = 0.f;
    for (int i = lane; i < per * tm.rl; i += 32) {
      const int l = i / per, j = g * per + i - l * per;
      const int th = l * tm.cb + (ONE ? j : j / V);
      c += cnts[th];
      sum = fmaf(cnts[th], ent[th * E + (ONE ? 0 : j % V)].x, sum);
    }
    c = warp_sum(c);
    const float m = warp_sum(sum) / fmaxf(c, 1.f);
    float q = 0.f;
    for (int i = lane; i < per * tm.rl; i += 32) {
      const int l = i / per, j = g * per + i - l * per;
      const int th = l * tm.cb + (ONE ? j : j / V);
      const float2 v = ent[th * E + (ONE ? 0 : j % V)];
      const float d = v.x - m;
      q += cnts[th] > 0.f ? fmaf(cnts[th] * d, d, v.y) : 0.f;
    }
    q = warp_sum(q);
    const int at = k.rank * tm.ng + g;
    if (many) {
      if (lane < tm.cluster) {
        store_cluster(&sn[at], lane, c);
        store_cluster(&sm[at], lane, m);
        store_cluster(&sq[at], lane, q);
      }
    } else if (lane == 0) {
      sn[at] = c, sm[at] = m, sq[at] = q;
    }
  }
  if (many) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  for (int g = threadIdx.x; g < tm.ng; g += blockDim.x) {
    const float total = (float)s.hw * (float)s.cpg;
    float sum = 0.f, q = 0.f;
    for (int j = 0; j < tm.cluster; ++j) sum = fmaf(sn[j * tm.ng + g], sm[j * tm.ng + g], sum);
    const float mu = sum / total;
    for (int j = 0; j < tm.cluster; ++j) {
      const float d = sm[j * tm.ng + g] - mu;
      q += fmaf(sn[j * tm.ng + g] * d, d, sq[j * tm.ng + g]);
    }
    const float rs = 1.f / sqrtf(q / total + s.eps);
    ent[g] = make_float2(mu, rs);
    if (k.rank == 0) {
      const int id = blockIdx.x / tm.cluster;
      const long long at = (long long)k.img * s.groups + (id - k.img * tm.slices) * tm.ng + g;
      if (mean_out) mean_out[at] = mu;
      if (rstd_out) rstd_out[at] = rs;
    }
  }
  __syncthreads();
  if (!k.live) return;
  float mu[E], a[V], b[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float2 st = ent[(k.col * V + e) / s.cpg];
    mu[ONE ? 0 : e] = st.x;
    a[e] = st.y * (gamma ? gamma[k.ch + e] : 1.f);
    b[e] = beta ? beta[k.ch + e] : 0.f;
  }
  for (int r = 0; r < tm.rounds; ++r) {
    if (r) load_col<T, V, NV>(s, tm, k, r, x, raw);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = k.pixel(s, tm, r, i);
      if (p >= s.hw) continue;
      float f[V];
      unpack<T, V>(raw[i], f);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = fmaf(f[e] - mu[ONE ? 0 : e], a[e], b[e]);
      act_vec<V>(f, s.act);
      store_vec<T, V>(y + k.base + (long long)p * s.c, f);
    }
  }
}

// smem: float2 [rl][width] of the threads' channel sums.
template <typename T, typename TG, int V, int NV>
__global__ void __launch_bounds__(kTeam, 1)
    bwd_nhwc(Shape s, ColTeam tm, const T* x, const TG* gy, const float* gamma, const float* beta,
             const float* mean, const float* rstd, T* gx, float2* part) {
  extern __shared__ float2 tab[];
  __shared__ float2 ps[kTeam];
  __shared__ float sa[kMaxCluster * kMaxGroups], sb[kMaxCluster * kMaxGroups];
  const bool many = tm.cluster > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const UnitCol<V> k(s, tm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  Raw<T, V> raw[NV];
  Raw<TG, V> graw[NV];
  const int id = blockIdx.x / tm.cluster;
  const long long g0 = (long long)k.img * s.groups + (id - k.img * tm.slices) * tm.ng;
  float mu[V], rs[V], g[V], b[V];
  float s1[V] = {}, s2[V] = {};
  if (k.live) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const long long at = g0 + (k.col * V + e) / s.cpg;
      mu[e] = mean[at];
      rs[e] = rstd[at];
      g[e] = gamma ? gamma[k.ch + e] : 1.f;
      b[e] = beta ? beta[k.ch + e] : 0.f;
    }
  }
  for (int r = tm.rounds - 1; r >= 0; --r) {
    load_col<T, V, NV>(s, tm, k, r, x, raw);
    load_col<TG, V, NV>(s, tm, k, r, gy, graw);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (k.pixel(s, tm, r, i) >= s.hw) continue;
      float f[V], z[V], d[V];
      unpack<T, V>(raw[i], f);
      unpack<TG, V>(graw[i], d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = (f[e] - mu[e]) * rs[e];
        z[e] = fmaf(f[e], g[e], b[e]);
      }
      slope_vec<V>(z, d, s.act);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s1[e] += d[e];
        s2[e] = fmaf(d[e], f[e], s2[e]);
      }
    }
  }
  // the block's sum of each channel: `lanes` threads a channel, then one
  if (k.live) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      tab[k.lane * tm.width + k.col * V + e] = make_float2(s1[e], s2[e]);
  }
  __syncthreads();
  const int lanes = (int)blockDim.x > tm.width ? (int)blockDim.x / tm.width : 1;
  for (int i = threadIdx.x; i < lanes * tm.width; i += blockDim.x) {
    const int l0 = i / tm.width, c = i - l0 * tm.width;
    float2 t = make_float2(0.f, 0.f);
    for (int l = l0; l < tm.rl; l += lanes) {
      const float2 v = tab[l * tm.width + c];
      t.x += v.x;
      t.y += v.y;
    }
    if (lanes > 1)
      ps[i] = t;
    else
      tab[c] = t;  // (lane 0's own entry: read above by this thread alone)
  }
  __syncthreads();
  for (int c = threadIdx.x; c < tm.width; c += blockDim.x) {
    float2 t = lanes > 1 ? ps[c] : tab[c];
    if (lanes > 1) {
      for (int l = 1; l < lanes; ++l) {
        const float2 v = ps[l * tm.width + c];
        t.x += v.x;
        t.y += v.y;
      }
    }
    const int ch = (id - k.img * tm.slices) * tm.width + c;
    part[((long long)k.rank * s.n + k.img) * s.c + ch] = t;
    const float gm = gamma ? gamma[ch] : 1.f;
    tab[c] = make_float2(gm * t.x, gm * t.y);
  }
  __syncthreads();
  if (many) cluster_wait();
  for (int q = warp; q < tm.ng; q += warps) {
    float a1 = 0.f, b1 = 0.f;
    for (int i = lane; i < s.cpg; i += 32) {
      a1 += tab[q * s.cpg + i].x;
      b1 += tab[q * s.cpg + i].y;
    }
    a1 = warp_sum(a1);
    b1 = warp_sum(b1);
    const int at = k.rank * tm.ng + q;
    if (many) {
      if (lane < tm.cluster) {
        store_cluster(&sa[at], lane, a1);
        store_cluster(&sb[at], lane, b1);
      }
    } else if (lane == 0) {
      sa[at] = a1, sb[at] = b1;
    }
  }
  if (many) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  for (int q = threadIdx.x; q < tm.ng; q += blockDim.x) {
    const float total = (float)s.hw * (float)s.cpg;
    float a1 = 0.f, b1 = 0.f;
    for (int j = 0; j < tm.cluster; ++j) {
      a1 += sa[j * tm.ng + q];
      b1 += sb[j * tm.ng + q];
    }
    ps[q] = make_float2(a1 / total, b1 / total);
  }
  __syncthreads();
  if (!k.live) return;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float2 v = ps[(k.col * V + e) / s.cpg];
    s1[e] = v.x;
    s2[e] = v.y;
  }
  for (int r = 0; r < tm.rounds; ++r) {
    if (r) {
      load_col<T, V, NV>(s, tm, k, r, x, raw);
      load_col<TG, V, NV>(s, tm, k, r, gy, graw);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = k.pixel(s, tm, r, i);
      if (p >= s.hw) continue;
      float f[V], z[V], d[V];
      unpack<T, V>(raw[i], f);
      unpack<TG, V>(graw[i], d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = (f[e] - mu[e]) * rs[e];
        z[e] = fmaf(f[e], g[e], b[e]);
      }
      slope_vec<V>(z, d, s.act);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = rs[e] * (fmaf(g[e], d[e], -s1[e]) - f[e] * s2[e]);
      store_vec<T, V>(gx + k.base + (long long)p * s.c, f);
    }
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

template <typename K, typename... A>
cudaError_t launch_team(K kern, unsigned blocks, int threads, int cluster, size_t smem,
                        cudaStream_t s, A... args) {
  if (cluster > 8) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  note_launches(1);
  return e;
}

// How a call runs: as one launch of teams, or in the three-launch form.
struct Plan {
  Shape s;
  bool team;
  RowTeam row;
  ColTeam col;
  unsigned blocks;
  int threads, nv;
  int parts;  // rows of channel sums an image leaves (backward)
};

constexpr int kSms = 152;

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

Plan make_plan(const NormArgs& a, bool backward) {
  Plan p{};
  p.s = make_shape(a);
  p.parts = 1;
  if (a.n == 0) return p;
  const int vec = a.dt == DC_BF16 ? 8 : 4, most = backward ? 4 : 8;
  const long long groups = (long long)a.n * a.groups;
  if (!a.nhwc) {
    Tiling t{};
    const int vr = row_vectors(a.hw, a.hw % vec ? vec - 1 : 0, vec);
    t.lpr = 1;
    while (t.lpr < 32 && t.lpr < vr) t.lpr *= 2;
    const long long blks = ceil_div_ll(a.cpg, 32 / t.lpr);
    long long tasks = 0;
    // vectors of a lane: as many as leave a block for every SM
    for (p.nv = most; p.nv >= 1; p.nv /= 2) {
      t.parts = (int)ceil_div_ll(vr, p.nv * t.lpr);
      tasks = blks * t.parts;
      if (p.nv == 1 || groups * ceil_div_ll(tasks, 16) >= kSms) break;
    }
    t.seg = (int)ceil_div_ll(vr, t.parts);
    t.parts = (int)ceil_div_ll(vr, t.seg);
    tasks = blks * t.parts;
    if (tasks > 1 << 20) return p;
    RowTeam& r = p.row;
    r.tasks = (int)tasks;
    r.cluster = (int)ceil_div_ll(tasks, 16);
    if (r.cluster > kMaxCluster) r.cluster = kMaxCluster;
    r.rounds = (int)ceil_div_ll(tasks, r.cluster * 16);
    r.warps = (int)ceil_div_ll(tasks, r.cluster * r.rounds);
    r.units = 1;
    if (r.rounds > 1 && groups * r.cluster < kSms) return p;
    if (r.cluster == 1)
      while (r.units * r.warps < 8 && groups / (2 * r.units) >= 4 * kSms) r.units *= 2;
    p.team = true;
    p.s.t = t;
    p.threads = 32 * r.warps * r.units;
    p.blocks = (unsigned)(ceil_div_ll(groups, r.units) * r.cluster);
    p.parts = t.parts;
    return p;
  }
  const int v = p.s.t.v, elt = a.dt == DC_BF16 ? 2 : 4;
  const long long base = (long long)a.cpg / gcd(a.cpg, v) * v;
  if (base / v > 256) return p;
  const int slices_most = (int)(a.c / base);
  ColTeam& c = p.col;
  // the narrowest slice of 64 bytes a pixel, or of 128 where there are blocks enough
  for (int bytes = 128; bytes >= 64; bytes /= 2) {
    int m = 1;
    while (m < slices_most && (m * base * elt < bytes || slices_most % m)) ++m;
    while (m > 1 && (m * base / v > 256 || m * base / a.cpg > kMaxGroups || slices_most % m)) --m;
    c.width = (int)(m * base);
    c.slices = a.c / c.width;
    c.cb = c.width / v;
    c.ng = c.width / a.cpg;
    p.nv = most;
    const int rows = kTeam / c.cb * p.nv;
    c.cluster = (int)ceil_div_ll(a.hw, rows);
    if ((long long)a.n * c.slices * c.cluster >= 2 * kSms) break;
  }
  if (c.ng > kMaxGroups) return p;
  const long long units = (long long)a.n * c.slices;
  // few blocks: spread a unit over more, down to 64 pixels each
  while (c.cluster < 8 && units * c.cluster < kSms && a.hw / (c.cluster + 1) >= 64) ++c.cluster;
  if (c.cluster > kMaxCluster) c.cluster = kMaxCluster;
  c.rounds = (int)ceil_div_ll(a.hw, (long long)c.cluster * (kTeam / c.cb) * p.nv);
  if (c.rounds > 1 && units * c.cluster < kSms) return p;
  c.rl = (int)ceil_div_ll(a.hw, (long long)c.cluster * c.rounds * p.nv);
  // a small unit: more threads rather than more pixels a thread
  while (c.rounds == 1 && p.nv > 1 && 2 * c.rl * c.cb <= 256) {
    p.nv /= 2;
    c.rl = (int)ceil_div_ll(a.hw, (long long)c.cluster * p.nv);
  }
  c.nv = p.nv;
  p.threads = (int)ceil_div_ll((long long)c.rl * c.cb, 32) * 32;
  if (units * c.cluster > INT_MAX) return p;
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
template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename T, typename F>
cudaError_t by_width(int v, F&& f) {
  if (v == VecOf<T>::n) return f(Int<VecOf<T>::n>{});
  if (sizeof(T) == 2 && v == 4) return f(Int<4>{});
  return f(Int<1>{});
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
  const Plan p = make_plan(a, backward);
  if (p.team)
    return backward ? round256((size_t)p.parts * a.n * a.c * sizeof(float2)) : 0;
  const Shape& s = p.s;
  const size_t units = (size_t)a.n * a.groups;
  if (!backward) return part_bytes(s) + round256(units * sizeof(float2));
  return part_bytes(s) + round256((size_t)a.n * a.c * sizeof(float2)) +
         round256(units * sizeof(float2));
}

bool norm_one_launch(const NormArgs& a, bool backward) { return make_plan(a, backward).team; }

namespace {
template <int MOST, typename F>
cudaError_t by_count(int nv, F&& f) {
  if (MOST > 4 && nv > 4) return f(Int<MOST>{});
  return f(Int<4>{});
}
}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
  const Plan p = make_plan(a, false);
  const Shape& s = p.s;
  return by_dtype(a.dt, [&](auto t) {
    using T = decltype(t);
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.y);
    return by_count<8>(p.nv, [&](auto nv) {
      constexpr int NV = decltype(nv)::value;
      if (!a.nhwc) {
        auto go = [&](auto kern) {
          return launch_team(kern, p.blocks, p.threads, p.row.cluster, 0, st, s, p.row, x, a.gamma,
                             a.beta, y, a.mean, a.rstd);
        };
        return a.hw % VecOf<T>::n ? go(fwd_nchw<T, false, NV>) : go(fwd_nchw<T, true, NV>);
      }
      return by_width<T>(s.t.v, [&](auto w) {
        constexpr int V = decltype(w)::value;
        auto go = [&](auto kern) {
          return launch_team(kern, p.blocks, p.threads, p.col.cluster, 0, st, s, p.col, x, a.gamma,
                             a.beta, y, a.mean, a.rstd);
        };
        return s.cpg % V ? go(fwd_nhwc<T, V, NV, false>) : go(fwd_nhwc<T, V, NV, true>);
      });
    });
  });
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st) {
  const Plan p = make_plan(a, true);
  const Shape& s = p.s;
  float2* part = reinterpret_cast<float2*>(a.ws);
  return by_dtypes(a, [&](auto t, auto g) {
    using T = decltype(t);
    using TG = decltype(g);
    const T* x = static_cast<const T*>(a.x);
    const TG* gy = static_cast<const TG*>(a.gy);
    T* gx = static_cast<T*>(a.gx);
    constexpr int NV = 4;
    if (!a.nhwc) {
      auto go = [&](auto kern) {
        return launch_team(kern, p.blocks, p.threads, p.row.cluster, 0, st, s, p.row, x, gy,
                           a.gamma, a.beta, a.mean, a.rstd, gx, part);
      };
      return a.hw % VecOf<T>::n ? go(bwd_nchw<T, TG, false, NV>) : go(bwd_nchw<T, TG, true, NV>);
    }
    return by_width<T>(s.t.v, [&](auto w) {
      constexpr int V = decltype(w)::value;
      return launch_team(bwd_nhwc<T, TG, V, NV>, p.blocks, p.threads, p.col.cluster,
                         (size_t)p.col.rl * p.col.width * sizeof(float2), st, s, p.col, x, gy,
                         a.gamma, a.beta, a.mean, a.rstd, gx, part);
    });
  });
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
    if (!a.nhwc)
      return launch(apply_nchw<T>, row_grid(s), kThreads, st, s, x, a.gamma, a.beta, m, r, y,
                    row_tasks(s));
    return by_width<T>(s.t.v, [&](auto w) {
      return launch(apply_nhwc<T, decltype(w)::value>, col_grid(s), kThreads, st, s, x, a.gamma,
                    a.beta, m, r, y);
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
    if (!a.nhwc)
      return launch(sums_nchw<T, TG>, row_grid(s), kThreads, st, s, x, gy, a.gamma, a.beta, m, r,
                    part, row_tasks(s));
    return by_width<T>(s.t.v, [&](auto w) {
      return launch(sums_nhwc<T, TG, decltype(w)::value>, col_grid(s), kThreads, st, s, x, gy,
                    a.gamma, a.beta, m, r, part);
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
    if (!a.nhwc)
      return launch(apply_bwd_nchw<T, TG>, row_grid(s), kThreads, st, s, x, gy, a.gamma, a.beta, m,
                    r, coef, gx, row_tasks(s));
    return by_width<T>(s.t.v, [&](auto w) {
      return launch(apply_bwd_nhwc<T, TG, decltype(w)::value>, col_grid(s), kThreads, st, s, x, gy,
                    a.gamma, a.beta, m, r, coef, gx);
    });
  });
}

cudaError_t launch_norm_params(const NormArgs& a, cudaStream_t st) {
  const Plan p = make_plan(a, true);
  const float2* chan = !a.n     ? nullptr
                       : p.team ? reinterpret_cast<const float2*>(a.ws)
                                : ws_chan(a, p.s);
  return launch(sum_images, dim3((unsigned)ceil_div_ll(a.c, 32)), 1024, st,
                (long long)p.parts * a.n, a.c, chan, a.ggamma, a.gbeta);
}

}  // namespace dc
