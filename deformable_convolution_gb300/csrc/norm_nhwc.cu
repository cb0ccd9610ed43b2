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

// Held vectors: slot i of a thread is P pieces of kUnit bytes, blockDim.x
// pieces apart; V elements of T take the first of them.
template <typename T, int V>
constexpr int kUnit = V * sizeof(T) >= 16 ? 16 : V * sizeof(T);
template <typename T, int V>
constexpr int kPieces = V * sizeof(T) / kUnit<T, V>;

template <typename T, int V>
__device__ __forceinline__ void take(const char* slot, Pairs<V>& f) {
  constexpr int kBytes = V * sizeof(T);
  if constexpr (kBytes <= 16) {
    load_vec<T, V>(reinterpret_cast<const T*>(slot), f);
  } else {
    uint32_t u[kBytes / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(slot + i * 16 * blockDim.x);
      u[4 * i] = v.x, u[4 * i + 1] = v.y, u[4 * i + 2] = v.z, u[4 * i + 3] = v.w;
    }
    unpack<T, V>(u, f);
  }
}
// f in float32 over a slot of as many bytes
template <int V>
__device__ __forceinline__ void leave(char* slot, const Pairs<V>& f) {
  const float* e = reinterpret_cast<const float*>(f.p);
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      *reinterpret_cast<float4*>(slot + i * 16 * blockDim.x) =
          make_float4(e[4 * i], e[4 * i + 1], e[4 * i + 2], e[4 * i + 3]);
  } else {
    *reinterpret_cast<float*>(slot) = e[0];
  }
}

// Starts the copies of a thread's first `count` pixels to its slots.
template <typename T, int V>
__device__ __forceinline__ void hold_col(const T* p, long long step, int count, char* slot,
                                         int stride) {
  constexpr int kBytes = V * sizeof(T);
  if constexpr (kBytes >= 4) {  // (an asynchronous copy moves 4 bytes at least)
    for (int i = 0; i < count; ++i, p += step, slot += stride) {
      copy_async<kUnit<T, V>>(slot, p);
      if constexpr (kBytes > 16) copy_async<16>(slot + 16 * blockDim.x, p + V / 2);
    }
  }
}

constexpr int kBatch = 4;

// A thread's (n, mean, m2), a triple for each channel of its vector or (ONE)
// for all of them, merged with those of `most` <= kBatch pixels; get(b, f)
// fetches pixel b.
template <int V, bool ONE, typename M, typename GET>
__device__ __forceinline__ void add_batch(int most, float& n, M& mean, M& m2, GET&& get) {
  constexpr int P = Pairs<V>::n, EP = ONE ? 1 : P;
  Pairs<V> f[kBatch];
  float2 sum[EP], q[EP];
#pragma unroll
  for (int e = 0; e < EP; ++e) sum[e] = q[e] = both(0.f);
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    if (b >= most) continue;
    get(b, f[b]);
#pragma unroll
    for (int e = 0; e < P; ++e) sum[ONE ? 0 : e] = add2(sum[ONE ? 0 : e], f[b].p[e]);
  }
  const float cnt = (float)(ONE ? most * V : most), t = n + cnt;
  const float w = rcp_approx(cnt), wn = cnt * rcp_approx(t), c = n * wn;
#pragma unroll
  for (int e = 0; e < EP; ++e)  // the means
    sum[e] = ONE ? both((sum[e].x + sum[e].y) * w) : mul2(sum[e], both(w));
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    if (b >= most) continue;
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

// ONE: a vector's channels are all of one group; else channels are kept apart
// until the block's are merged.  Dynamic shared memory: the slots, then the
// blocks' triples of the unit's groups, [3][cluster][ng].
template <typename T, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(kTeam, ONE || V < 8 ? 2 : 1)
    fwd_nhwc(Shape s, ColTeam tm, const T* x, const float* gamma, const float* beta, T* y,
             float* mean_out, float* rstd_out) {
  constexpr int P = Pairs<V>::n, E = ONE ? 1 : V, EP = ONE ? 1 : P;
  extern __shared__ uint4 hold[];
  __shared__ float2 ent[kTeam];
  __shared__ float cnts[kTeam];
  const bool many = tm.cluster > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const UnitCol<V> k(s, tm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int stride = kPieces<T, V> * kUnit<T, V> * blockDim.x;
  char* mine = reinterpret_cast<char*>(hold) + threadIdx.x * kUnit<T, V>;
  float* sn = reinterpret_cast<float*>(reinterpret_cast<char*>(hold) + (size_t)tm.held * stride);
  float* sm = sn + tm.cluster * tm.ng;
  float* sq = sm + tm.cluster * tm.ng;
  const int count = k.p1 > k.p0 ? (k.p1 - k.p0 + tm.rl - 1) / tm.rl : 0;  // this thread's pixels
  const int held = count < tm.held ? count : tm.held;
  const long long step = (long long)tm.rl * s.c;
  const T* px = x + k.base + (long long)k.p0 * s.c;
  hold_col<T, V>(px, step, held, mine, stride);
  float n = 0.f;
  Pairs<2 * EP> mean, m2;  // ONE: the first of a pair alone
#pragma unroll
  for (int e = 0; e < EP; ++e) mean.p[e] = m2.p[e] = both(0.f);
  // what is not held first: its loads go on behind the copies
  for (int i = held; i < count; i += kBatch)
    add_batch<V, ONE>(min(count - i, kBatch), n, mean, m2,
                      [&](int b, Pairs<V>& f) { load_vec<T, V>(px + (i + b) * step, f); });
  copy_wait();
  {
    const char* slot = mine;
    auto get = [&](int b, Pairs<V>& f) { take<T, V>(slot + b * stride, f); };
    int i = 0;
    for (; i + kBatch <= held; i += kBatch, slot += kBatch * stride)
      add_batch<V, ONE>(kBatch, n, mean, m2, get);
    if (i < held) add_batch<V, ONE>(held - i, n, mean, m2, get);
  }
  // the block's groups, a warp each: entries of every pixel lane, channel by
  // channel of the vector where those are apart
  const int cols = ONE ? s.cpg / V : tm.cb;  // columns of a group (all, where they mix)
  cnts[threadIdx.x] = n;
  if (many) cluster_wait();
  for (int g0 = 0; g0 < tm.ng; g0 += warps) {
    const int g = g0 + warp;
    float gn = 0.f, gm = 0.f, gq = 0.f;
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
      __syncthreads();
      float a = mean.p[0].x, b = m2.p[0].x;
#pragma unroll
      for (int j = 1; j < E; ++j)
        if (j == e) a = mean[j], b = m2[j];
      ent[threadIdx.x] = make_float2(a, b);
      __syncthreads();
      if (g >= tm.ng) continue;
      const int entries = cols * tm.rl;
      float ln = 0.f, lm = 0.f, lq = 0.f;
      for (int i = lane; i < entries; i += 32) {
        const int l = cols == 1 ? i : i / cols, j = i - l * cols;
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
  // a group's blocks, a lane each
  for (int g = warp; g < tm.ng; g += warps) {
    const float total = (float)s.hw * (float)s.cpg;
    const int at = lane * tm.ng + g;
    const bool in = lane < tm.cluster && sn[at] > 0.f;
    const float mu = warp_sum(in ? sn[at] * sm[at] : 0.f) / total;
    const float d = in ? sm[at] - mu : 0.f;
    const float var = warp_sum(in ? fmaf(sn[at] * d, d, sq[at]) : 0.f) / total;
    const float rs = 1.f / sqrtf(var + s.eps);
    if (lane == 0) {
      ent[g] = make_float2(mu, rs);
      if (k.rank == 0) {
        const long long to = (long long)k.img * s.groups + k.slice * tm.ng + g;
        if (mean_out) mean_out[to] = mu;
        if (rstd_out) rstd_out[to] = rs;
      }
    }
  }
  __syncthreads();
  if (!k.live) return;
  Pairs<ONE ? 1 : V> mu;  // minus the mean
  Pairs<V> a, b;
  if (V == 1) a.p[0] = b.p[0] = mu.p[0] = both(0.f);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float2 st = ent[(k.col * V + (ONE ? 0 : e)) / s.cpg];
    mu[ONE ? 0 : e] = -st.x;
    a[e] = st.y * (gamma ? gamma[k.ch + e] : 1.f);
    b[e] = beta ? beta[k.ch + e] : 0.f;
  }
  T* to = y + k.base + (long long)k.p0 * s.c;
  auto apply = [&](Pairs<V>& f) {
#pragma unroll
    for (int e = 0; e < P; ++e)
      f.p[e] = act_fwd2<ACT>(fma2(add2(f.p[e], ONE ? both(mu[0]) : mu.p[ONE ? 0 : e]), a.p[e],
                                  b.p[e]), s.floor);
    store_vec<T, V>(to, f);
    to += step;
  };
  const char* slot = mine;
#pragma unroll 2
  for (int i = 0; i < held; ++i, slot += stride) {
    Pairs<V> f;
    take<T, V>(slot, f);
    apply(f);
  }
  px += held * step;
  for (int i = held; i < count; ++i, px += step) {
    Pairs<V> f;
    load_vec<T, V>(px, f);
    apply(f);
  }
}

// part[rank][image * c + channel]: the sums of dz and dz * xh over a block's
// pixels.  Dynamic shared memory: the slots of x, of grad_y, a table of channel
// sums, then the blocks' sums of the unit's groups, [2][cluster][ng].
template <typename T, typename TG, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(kTeam, ONE || V < 8 ? 2 : 1)
    bwd_nhwc(Shape s, ColTeam tm, const T* x, const TG* gy, const float* gamma, const float* beta,
             const float* mean, const float* rstd, T* gx, float2* part) {
  constexpr int P = Pairs<V>::n;
  constexpr bool KEEP = keep_dz(sizeof(TG) == 4, ACT);
  using SG = std::conditional_t<KEEP, float, TG>;  // what a slot of grad_y has room for
  extern __shared__ uint4 hold[];
  __shared__ float2 ps[kTeam];
  const bool many = tm.cluster > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const UnitCol<V> k(s, tm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int stride = V * sizeof(T) * blockDim.x, stride_g = V * sizeof(SG) * blockDim.x;
  char* mine = reinterpret_cast<char*>(hold) + threadIdx.x * kUnit<T, V>;
  char* held_g = reinterpret_cast<char*>(hold) + (size_t)tm.held * stride;
  char* mine_g = held_g + threadIdx.x * kUnit<SG, V>;
  float2* tab = reinterpret_cast<float2*>(held_g + (size_t)tm.held * stride_g);
  float* sa = reinterpret_cast<float*>(tab + tm.rows * tm.width);
  float* sb = sa + tm.cluster * tm.ng;
  const int count = k.p1 > k.p0 ? (k.p1 - k.p0 + tm.rl - 1) / tm.rl : 0;
  const int held = count < tm.held ? count : tm.held;
  const long long step = (long long)tm.rl * s.c, off = k.base + (long long)k.p0 * s.c;
  hold_col<T, V>(x + off, step, held, mine, stride);
  hold_col<TG, V>(gy + off, step, held, mine_g, stride_g);
  const long long g0 = (long long)k.img * s.groups + k.slice * tm.ng;
  Pairs<ONE ? 1 : V> mu, rs;  // minus the mean
  Pairs<V> g, b, s1, s2;
#pragma unroll
  for (int e = 0; e < P; ++e) g.p[e] = b.p[e] = s1.p[e] = s2.p[e] = both(0.f);
#pragma unroll
  for (int e = 0; e < (ONE ? 1 : P); ++e) mu.p[e] = rs.p[e] = both(0.f);
  if (k.live) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (!ONE || e == 0) {
        const long long at = g0 + (k.col * V + e) / s.cpg;
        mu[ONE ? 0 : e] = -mean[at], rs[ONE ? 0 : e] = rstd[at];
      }
      g[e] = gamma ? gamma[k.ch + e] : 1.f;
      b[e] = beta ? beta[k.ch + e] : 0.f;
    }
  }
  auto xhat = [&](const Pairs<V>& f, int e) {
    const float2 m = ONE ? both(mu[0]) : mu.p[ONE ? 0 : e];
    return mul2(add2(f.p[e], m), ONE ? both(rs[0]) : rs.p[ONE ? 0 : e]);
  };
  // dz in place of grad_y
  auto slope = [&](const float2 xh, Pairs<V>& d, int e) {
    d.p[e] = act_bwd2<ACT>(fma2(xh, g.p[e], b.p[e]), d.p[e], s.floor);
    if (V == 1) d.p[e].y = 0.f;
  };
  auto sums = [&](const Pairs<V>& f, Pairs<V>& d) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float2 xh = xhat(f, e);
      slope(xh, d, e);
      s1.p[e] = add2(s1.p[e], d.p[e]);
      s2.p[e] = fma2(d.p[e], xh, s2.p[e]);
    }
  };
  // what is not held first: its loads go on behind the copies
#pragma unroll 2
  for (int i = held; i < count; ++i) {
    Pairs<V> f, d;
    load_vec<T, V>(x + off + i * step, f);
    load_vec<TG, V>(gy + off + i * step, d);
    sums(f, d);
  }
  copy_wait();
  {
    const char* slot = mine;
    char* slot_g = mine_g;
#pragma unroll 2
    for (int i = 0; i < held; ++i, slot += stride, slot_g += stride_g) {
      Pairs<V> f, d;
      take<T, V>(slot, f);
      take<TG, V>(slot_g, d);
      sums(f, d);
      if (KEEP) leave<V>(slot_g, d);
    }
  }
  // the block's sum of each channel: pixel lanes of a warp first (where a warp
  // holds whole pixels), then the table's rows by `lanes` threads a channel,
  // then by one
  int row = k.lane;
  bool put = k.live;
  if (32 % tm.cb == 0) {
    for (int o = 16; o >= tm.cb; o >>= 1) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s1[e] += __shfl_xor_sync(0xffffffffu, s1[e], o);
        s2[e] += __shfl_xor_sync(0xffffffffu, s2[e], o);
      }
    }
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
    for (int l = l0; l < tm.rows; l += lanes) {
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
  for (int q = warp; q < tm.ng; q += warps) {  // a group's blocks, a lane each
    const float total = (float)s.hw * (float)s.cpg;
    const bool in = lane < tm.cluster;
    const float a1 = warp_sum(in ? sa[lane * tm.ng + q] : 0.f);
    const float b1 = warp_sum(in ? sb[lane * tm.ng + q] : 0.f);
    if (lane == 0) ps[q] = make_float2(a1 / total, b1 / total);
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
  T* to = gx + off;
  auto result = [&](Pairs<V>& f, Pairs<V>& d, bool is_dz) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float2 xh = xhat(f, e);
      if (!is_dz) slope(xh, d, e);
      const float2 gr = mul2(g.p[e], ONE ? both(rs[0]) : rs.p[ONE ? 0 : e]);
      f.p[e] = fma2(xh, ONE ? both(k2[0]) : k2.p[ONE ? 0 : e],
                    fma2(d.p[e], gr, ONE ? both(k1[0]) : k1.p[ONE ? 0 : e]));
    }
    store_vec<T, V>(to, f);
    to += step;
  };
  const char* slot = mine;
  const char* slot_g = mine_g;
#pragma unroll 2
  for (int i = 0; i < held; ++i, slot += stride, slot_g += stride_g) {
    Pairs<V> f, d;
    take<T, V>(slot, f);
    take<SG, V>(slot_g, d);
    result(f, d, KEEP);
  }
  for (int i = held; i < count; ++i) {
    Pairs<V> f, d;
    load_vec<T, V>(x + off + i * step, f);
    load_vec<TG, V>(gy + off + i * step, d);
    result(f, d, false);
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
