// Group norm with an activation on [n][h][w][c] tensors, one launch.
//
// A slice of whole groups of an image, 64 or 128 bytes of every pixel, is a
// unit, held in the shared memory of a cluster's blocks from the statistics to
// the results (as on [n][c][h][w] tensors).  A thread keeps one vector of
// channels and walks pixels, so that gamma, beta and the sums of its channels
// stay in registers; the threads of a channel are added in a fixed order.
#include "dc_norm.cuh"

namespace dc {
namespace {

template <int V>
struct UnitCol {
  long long base;
  int id, img, slice, ch, col, lane, rank, p0, p1;
  bool live;
  __device__ __forceinline__ UnitCol(const Shape& s, const ColTeam& tm) {
    id = cluster_id();
    rank = cluster_rank();
    img = id / tm.slices;
    slice = id - img * tm.slices;
    lane = threadIdx.x / tm.cb;
    col = threadIdx.x - lane * tm.cb;
    live = lane < tm.rl;
    ch = slice * tm.width + col * V;
    base = (long long)img * s.hw * s.c + ch;
    // this thread's pixels p0 + i * rl < p1
    const long long first = (long long)rank * tm.span, end = first + tm.span;
    p0 = (int)min(first + lane, (long long)s.hw);
    p1 = live ? (int)min(end, (long long)s.hw) : p0;
  }
};

// A thread's held pixels: slot i at i * blockDim.x.
template <typename T, int V>
struct __align__(V * sizeof(T) >= 16 ? 16 : V * sizeof(T)) Cell {
  T e[V];
};

template <typename T, int V>
__device__ __forceinline__ void hold_col(const Shape& s, const ColTeam& tm, const UnitCol<V>& k,
                                         const T* x, Cell<T, V>* slot) {
  constexpr int kBytes = V * sizeof(T);
  if constexpr (kBytes >= 4) {
    int p = k.p0;
    for (int i = 0; i < tm.held && p < k.p1; ++i, p += tm.rl, slot += blockDim.x) {
      const T* from = x + k.base + (long long)p * s.c;
      if constexpr (kBytes > 16) {
        copy_async<16>(slot, from);
        copy_async<16>(reinterpret_cast<char*>(slot) + 16, from + V / 2);
      } else {
        copy_async<kBytes>(slot, from);
      }
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void fetch(const Shape& s, const ColTeam& tm, const UnitCol<V>& k, int i,
                                      int p, const T* x, const Cell<T, V>* slot, Pairs<V>& f) {
  if (i < tm.held)
    load_vec<T, V>(slot[(size_t)i * blockDim.x].e, f);
  else
    load_vec<T, V>(x + k.base + (long long)p * s.c, f);
}

// ONE: a vector's channels are all of one group; else channels are kept apart
// until the block's are merged.
template <typename T, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(kTeam, 2)
    fwd_nhwc(Shape s, ColTeam tm, const T* x, const float* gamma, const float* beta, T* y,
             float* mean_out, float* rstd_out) {
  constexpr int E = ONE ? 1 : V;
  constexpr int kBatch = 4;
  extern __shared__ uint4 hold[];
  __shared__ float2 ent[kTeam];
  __shared__ float cnts[kTeam];
  __shared__ float sn[kMaxCluster * kMaxGroups], sm[kMaxCluster * kMaxGroups],
      sq[kMaxCluster * kMaxGroups];
  const bool many = tm.cluster > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const UnitCol<V> k(s, tm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  Cell<T, V>* mine = reinterpret_cast<Cell<T, V>*>(hold) + threadIdx.x;
  hold_col<T, V>(s, tm, k, x, mine);
  constexpr int P = Pairs<V>::n;
  constexpr int EP = ONE ? 1 : P;  // pairs of sums
  float n = 0.f;
  Pairs<2 * EP> mean, m2;  // ONE: the first of a pair alone
#pragma unroll
  for (int e = 0; e < EP; ++e) mean.p[e] = m2.p[e] = both(0.f);
  auto batches = [&](int i0, int i1) {
    for (int i = i0; i < i1; i += kBatch) {
      const int p = k.p0 + i * tm.rl;
      if (p >= k.p1) break;
      Pairs<V> f[kBatch];
      float2 sum[EP], q[EP];
#pragma unroll
      for (int e = 0; e < EP; ++e) sum[e] = q[e] = both(0.f);
      float cnt = 0.f;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (i + b >= i1 || p + b * tm.rl >= k.p1) continue;
        fetch<T, V>(s, tm, k, i + b, p + b * tm.rl, x, mine, f[b]);
        cnt += ONE ? (float)V : 1.f;
#pragma unroll
        for (int e = 0; e < P; ++e) sum[ONE ? 0 : e] = add2(sum[ONE ? 0 : e], f[b].p[e]);
      }
      const float w = rcp_approx(cnt), t = n + cnt, wn = cnt * rcp_approx(t), c = n * wn;
#pragma unroll
      for (int e = 0; e < EP; ++e)  // the means
        sum[e] = ONE ? both((sum[e].x + sum[e].y) * w) : mul2(sum[e], both(w));
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (i + b >= i1 || p + b * tm.rl >= k.p1) continue;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 m = sum[ONE ? 0 : e];
          float2 d = add2(f[b].p[e], make_float2(-m.x, -m.y));
          if (V == 1) d.y = 0.f;
          q[ONE ? 0 : e] = fma2(d, d, q[ONE ? 0 : e]);
        }
      }
#pragma unroll
      for (int e = 0; e < EP; ++e) {
        if (ONE) q[e].x += q[e].y;
        const float2 d = add2(sum[e], make_float2(-mean.p[e].x, -mean.p[e].y));
        mean.p[e] = fma2(d, both(wn), mean.p[e]);
        m2.p[e] = add2(m2.p[e], fma2(mul2(d, d), both(c), q[e]));
      }
      n = t;
    }
  };
  // what is not held first: its loads go on behind the copies
  batches(tm.held, tm.slots);
  copy_wait();
  batches(0, tm.held);
  // the block's groups, a warp each: entries of every pixel lane, channel by
  // channel of the vector where those are apart
  const int cols = ONE ? s.cpg / V : tm.cb;  // columns of a group (all, where they mix)
  float gn = 0.f, gm = 0.f, gq = 0.f;        // of group `warp`, then warp + warps, ...: see below
  cnts[threadIdx.x] = n;
  if (many) cluster_wait();
  for (int g0 = 0; g0 < tm.ng; g0 += warps) {
    const int g = g0 + warp;
    gn = gm = gq = 0.f;
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
      __syncthreads();
      float a = mean[0], b = m2[0];
#pragma unroll
      for (int j = 1; j < E; ++j)
        if (j == e) a = mean[j], b = m2[j];
      ent[threadIdx.x] = make_float2(a, b);
      __syncthreads();
      if (g >= tm.ng) continue;
      const int entries = cols * tm.rl;
      float ln = 0.f, lm = 0.f, lq = 0.f;
      for (int i = lane; i < entries; i += 32) {
        const int l = i / cols, j = i - l * cols;
        const int th = l * tm.cb + (ONE ? g * cols + j : j);
        if (!ONE && (j * V + e) / s.cpg != g) continue;
        const float2 v = ent[th];
        merge(ln, lm, lq, cnts[th], v.x, v.y);
      }
      const float c = warp_sum(ln);
      const float m = warp_sum(ln * lm) / fmaxf(c, 1.f);
      const float q = warp_sum(ln > 0.f ? fmaf(ln * (lm - m), lm - m, lq) : 0.f);
      merge(gn, gm, gq, c, m, q);
    }
    if (g >= tm.ng) continue;
    const int at = k.rank * tm.ng + g;
    if (many) {
      if (lane < tm.cluster) {
        store_cluster(&sn[at], lane, gn);
        store_cluster(&sm[at], lane, gm);
        store_cluster(&sq[at], lane, gq);
      }
    } else if (lane == 0) {
      sn[at] = gn, sm[at] = gm, sq[at] = gq;
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
      if (sn[j * tm.ng + g] > 0.f) q += fmaf(sn[j * tm.ng + g] * d, d, sq[j * tm.ng + g]);
    }
    const float rs = 1.f / sqrtf(q / total + s.eps);
    ent[g] = make_float2(mu, rs);
    if (k.rank == 0) {
      const long long at = (long long)k.img * s.groups + k.slice * tm.ng + g;
      if (mean_out) mean_out[at] = mu;
      if (rstd_out) rstd_out[at] = rs;
    }
  }
  __syncthreads();
  if (!k.live) return;
  Pairs<ONE ? 1 : V> mu;  // minus the mean
  Pairs<V> a, b;
  if (V == 1) a.p[0] = b.p[0] = mu.p[0] = both(0.f);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float2 st = ent[(k.col * V + e) / s.cpg];
    mu[ONE ? 0 : e] = -st.x;
    a[e] = st.y * (gamma ? gamma[k.ch + e] : 1.f);
    b[e] = beta ? beta[k.ch + e] : 0.f;
  }
#pragma unroll 2
  for (int i = 0, p = k.p0; p < k.p1; ++i, p += tm.rl) {
    Pairs<V> f;
    fetch<T, V>(s, tm, k, i, p, x, mine, f);
#pragma unroll
    for (int e = 0; e < P; ++e)
      f.p[e] = fma2(add2(f.p[e], ONE ? both(mu[0]) : mu.p[ONE ? 0 : e]), a.p[e], b.p[e]);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = act_fwd<ACT>(f[e], s.floor);
    store_vec<T, V>(y + k.base + (long long)p * s.c, f);
  }
}

// part[rank][image * c + channel]: the sums of dz and dz * xh over a block's
// pixels.
template <typename T, typename TG, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(kTeam, 2)
    bwd_nhwc(Shape s, ColTeam tm, const T* x, const TG* gy, const float* gamma, const float* beta,
             const float* mean, const float* rstd, T* gx, float2* part) {
  extern __shared__ uint4 hold[];
  __shared__ float2 ps[kTeam];
  __shared__ float sa[kMaxCluster * kMaxGroups], sb[kMaxCluster * kMaxGroups];
  const bool many = tm.cluster > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const UnitCol<V> k(s, tm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  Cell<T, V>* mine = reinterpret_cast<Cell<T, V>*>(hold) + threadIdx.x;
  Cell<TG, V>* mine_g =
      reinterpret_cast<Cell<TG, V>*>(reinterpret_cast<Cell<T, V>*>(hold) +
                                     (size_t)tm.held * blockDim.x) + threadIdx.x;
  float2* tab = reinterpret_cast<float2*>(reinterpret_cast<char*>(hold) +
                                          (size_t)tm.held * blockDim.x * V *
                                              (sizeof(T) + sizeof(TG)));
  hold_col<T, V>(s, tm, k, x, mine);
  hold_col<TG, V>(s, tm, k, gy, mine_g);
  const long long g0 = (long long)k.img * s.groups + k.slice * tm.ng;
  constexpr int P = Pairs<V>::n;
  Pairs<ONE ? 1 : V> mu, rs;  // minus the mean
  Pairs<V> g, b, s1, s2;
#pragma unroll
  for (int e = 0; e < P; ++e) g.p[e] = b.p[e] = s1.p[e] = s2.p[e] = both(0.f);
#pragma unroll
  for (int e = 0; e < (ONE ? 1 : P); ++e) mu.p[e] = rs.p[e] = both(0.f);
  if (k.live) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const long long at = g0 + (k.col * V + e) / s.cpg;
      if (!ONE || e == 0) mu[ONE ? 0 : e] = -mean[at], rs[ONE ? 0 : e] = rstd[at];
      g[e] = gamma ? gamma[k.ch + e] : 1.f;
      b[e] = beta ? beta[k.ch + e] : 0.f;
    }
  }
  // the pair e of xh, and of dz in place of grad_y
  auto grads = [&](const Pairs<V>& f, Pairs<V>& d, int e) {
    const float2 m = ONE ? both(mu[0]) : mu.p[ONE ? 0 : e], r = ONE ? both(rs[0]) : rs.p[ONE ? 0 : e];
    const float2 xh = mul2(add2(f.p[e], m), r);
    const float2 z = fma2(xh, g.p[e], b.p[e]);
    d.p[e] = make_float2(act_bwd<ACT>(z.x, d.p[e].x, s.floor),
                         V == 1 ? 0.f : act_bwd<ACT>(z.y, d.p[e].y, s.floor));
    return xh;
  };
  auto sums = [&](int i0, int i1) {
#pragma unroll 2
    for (int i = i0; i < i1; ++i) {
      const int p = k.p0 + i * tm.rl;
      if (p >= k.p1) break;
      Pairs<V> f, d;
      fetch<T, V>(s, tm, k, i, p, x, mine, f);
      fetch<TG, V>(s, tm, k, i, p, gy, mine_g, d);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 xh = grads(f, d, e);
        s1.p[e] = add2(s1.p[e], d.p[e]);
        s2.p[e] = fma2(d.p[e], xh, s2.p[e]);
      }
    }
  };
  sums(tm.held, tm.slots);
  copy_wait();
  sums(0, tm.held);
  // the block's sum of each channel: pixel lanes of a warp first (where a warp
  // holds whole pixels), then `rows` rows of the table by `lanes` threads a
  // channel, then by one
  int rows = tm.rl, row = k.lane;
  bool put = k.live;
  if (32 % tm.cb == 0) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      for (int o = 16; o >= tm.cb; o >>= 1) {
        s1[e] += __shfl_xor_sync(0xffffffffu, s1[e], o);
        s2[e] += __shfl_xor_sync(0xffffffffu, s2[e], o);
      }
    rows = warps;
    row = warp;
    put = lane < tm.cb;
  }
  if (put) {
#pragma unroll
    for (int e = 0; e < V; ++e) tab[row * tm.width + k.col * V + e] = make_float2(s1[e], s2[e]);
  }
  __syncthreads();
  const int lanes = (int)blockDim.x > tm.width ? (int)blockDim.x / tm.width : 1;
  for (int i = threadIdx.x; i < lanes * tm.width; i += blockDim.x) {
    const int l0 = i / tm.width, c = i - l0 * tm.width;
    float2 t = make_float2(0.f, 0.f);
    for (int l = l0; l < rows; l += lanes) {
      const float2 v = tab[l * tm.width + c];
      t.x += v.x;
      t.y += v.y;
    }
    if (lanes > 1)
      ps[i] = t;
    else
      tab[c] = t;  // (row 0's own entry: read above by this thread alone)
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
    const int ch = k.slice * tm.width + c;
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
  // grad_x = dz * (gamma * rstd) - rstd * s1 - xh * (rstd * s2)
  Pairs<ONE ? 1 : V> k1, k2;
  if (V == 1) k1.p[0] = k2.p[0] = both(0.f);
#pragma unroll
  for (int e = 0; e < (ONE ? 1 : V); ++e) {
    const float2 v = ps[(k.col * V + e) / s.cpg];
    k1[e] = -rs[e] * v.x;
    k2[e] = -rs[e] * v.y;
  }
#pragma unroll 2
  for (int i = 0, p = k.p0; p < k.p1; ++i, p += tm.rl) {
    Pairs<V> f, d;
    fetch<T, V>(s, tm, k, i, p, x, mine, f);
    fetch<TG, V>(s, tm, k, i, p, gy, mine_g, d);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float2 xh = grads(f, d, e);
      const float2 r = ONE ? both(rs[0]) : rs.p[ONE ? 0 : e];
      const float2 c1 = ONE ? both(k1[0]) : k1.p[ONE ? 0 : e];
      const float2 c2 = ONE ? both(k2[0]) : k2.p[ONE ? 0 : e];
      f.p[e] = fma2(xh, c2, fma2(d.p[e], mul2(g.p[e], r), c1));
    }
    store_vec<T, V>(gx + k.base + (long long)p * s.c, f);
  }
}

}  // namespace

cudaError_t launch_team_nhwc(const NormPlan& p, const NormArgs& a, bool backward,
                             cudaStream_t st) {
  const int cpg = p.s.cpg;
  if (!backward)
    return by_dtype(a.dt, [&](auto t) {
      using T = decltype(t);
      return by_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        return by_width<T>(p.s.t.v, [&](auto w) {
          constexpr int V = decltype(w)::value;
          auto go = [&](auto kern) {
            return launch_team(kern, p, p.col.cluster, st, p.s, p.col, static_cast<const T*>(a.x),
                               a.gamma, a.beta, static_cast<T*>(a.y), a.mean, a.rstd);
          };
          return cpg % V ? go(fwd_nhwc<T, V, false, ACT>) : go(fwd_nhwc<T, V, true, ACT>);
        });
      });
    });
  return by_dtypes(a, [&](auto t, auto g) {
    using T = decltype(t);
    using TG = decltype(g);
    return by_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      return by_width<T>(p.s.t.v, [&](auto w) {
        constexpr int V = decltype(w)::value;
        auto go = [&](auto kern) {
          return launch_team(kern, p, p.col.cluster, st, p.s, p.col, static_cast<const T*>(a.x),
                             static_cast<const TG*>(a.gy), a.gamma, a.beta,
                             static_cast<const float*>(a.mean), static_cast<const float*>(a.rstd),
                             static_cast<T*>(a.gx), reinterpret_cast<float2*>(a.ws));
        };
        return cpg % V ? go(bwd_nhwc<T, TG, V, false, ACT>) : go(bwd_nhwc<T, TG, V, true, ACT>);
      });
    });
  });
}

}  // namespace dc
