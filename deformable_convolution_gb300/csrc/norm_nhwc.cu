// Group norm with an activation on [n][h][w][c] tensors (mathematics as on
// [n][c][h][w]).
//
// A slice of whole groups of an image, 64 or 128 bytes of every pixel, is a
// unit, held in the shared memory of a cluster's blocks from the statistics to
// the results (as on [n][c][h][w] tensors).  A thread keeps one vector of
// channels and walks pixels, so that gamma, beta and the sums of its channels
// stay in registers; the threads of a channel are added in a fixed order.
//
// Measured (launches alone): forward on 16 x 100 x 168 x 256 bf16 with SiLU
// 69 us, 4.0 TB/s, bytes' time 40.5; backward on 2 x 50 x 84 x 256 bf16 with
// SiLU 10.4 us, most of it the latency of its two launches.  The forward is
// bound by instruction issue and the barriers between a block's phases (17.6
// instructions an element at 2.0 of 4 a cycle, 28 warps an SM): two launches
// for it took 75 us, three 156.
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
    lane = quick_div(threadIdx.x, s.inv_cb);
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

// Starts the copy of a vector to a slot.
template <typename T, int V>
__device__ __forceinline__ void hold(const T* p, char* slot) {
  constexpr int kBytes = V * sizeof(T);
  if constexpr (kBytes >= 4) {  // (an asynchronous copy moves 4 bytes at least)
    copy_async<kUnit<T, V>, (kBytes > 16)>(slot, p);
    if constexpr (kBytes > 16) copy_async<16, true>(slot + 16 * blockDim.x, p + V / 2);
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
  const float w = rcp_approx(cnt), wn = n > 0.f ? cnt * rcp_approx(t) : 1.f, c = n * wn;
#pragma unroll
  for (int e = 0; e < EP; ++e)  // the means
    sum[e] = ONE ? both(quotient(sum[e].x + sum[e].y, cnt, w)) : quotient2(sum[e], cnt, w);
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

// The block's triples of its channels, where a vector's channels are of several
// groups: tab[rows][width] holds the pixel lanes' (mean, M2) (or, where a warp
// holds whole pixels, the warps'), cnt[row] their counts; merged by `lanes`
// threads a channel, then by one, into tab[0 .. width) and *n (the count).
template <int V, typename M>
__device__ __forceinline__ void channel_stats(int cb, int rl, int rows, int cols, int lane_px,
                                              int col, bool live, float n, M mean, M m2,
                                              float2* tab, float* cnt, float4* ps, float* total) {
  constexpr int P = Pairs<V>::n;
  const int width = cb * V, lane = threadIdx.x & 31;
  int row = lane_px;
  bool put = live;
  if (32 % cb == 0) {
    float c = n;
    for (int o = 16; o >= cb; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    const float w = rcp_approx(fmaxf(c, 1.f));
    Pairs<2 * P> m;
#pragma unroll
    for (int e = 0; e < P; ++e) m.p[e] = mul2(mean.p[e], both(n));
    for (int o = 16; o >= cb; o >>= 1)
#pragma unroll
      for (int e = 0; e < V; ++e) m[e] += __shfl_xor_sync(0xffffffffu, m[e], o);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      m.p[e] = quotient2(m.p[e], fmaxf(c, 1.f), w);
      const float2 d = add2(mean.p[e], make_float2(-m.p[e].x, -m.p[e].y));
      if (n > 0.f) m2.p[e] = fma2(mul2(d, d), both(n), m2.p[e]);
    }
    for (int o = 16; o >= cb; o >>= 1)
#pragma unroll
      for (int e = 0; e < V; ++e) m2[e] += __shfl_xor_sync(0xffffffffu, m2[e], o);
#pragma unroll
    for (int e = 0; e < P; ++e) mean.p[e] = m.p[e];
    n = c;
    row = threadIdx.x >> 5;
    put = lane < cb && col < cols;
  }
  if (put) {
#pragma unroll
    for (int e = 0; e < V; ++e) tab[row * width + col * V + e] = make_float2(mean[e], m2[e]);
    if (col == 0) cnt[row] = n;
  }
  __syncthreads();
  const int used = cols * V;
  const int lanes = (int)blockDim.x > used ? min((int)blockDim.x / used, rows) : 1;
  for (int i = threadIdx.x; i < lanes * used; i += blockDim.x) {
    const int l0 = i / used, c = i - l0 * used;
    float tn = 0.f, tm = 0.f, tq = 0.f;
    for (int l = l0; l < rows; l += lanes) {
      const float2 v = tab[l * width + c];
      merge(tn, tm, tq, cnt[l], v.x, v.y);
    }
    if (lanes > 1) {
      ps[i] = make_float4(tn, tm, tq, 0.f);
    } else {
      tab[c] = make_float2(tm, tq);  // (row 0's own entry: read above by this thread alone)
      if (c == 0) *total = tn;
    }
  }
  __syncthreads();
  if (lanes > 1) {
    for (int c = threadIdx.x; c < used; c += blockDim.x) {
      float tn = 0.f, tm = 0.f, tq = 0.f;
      for (int l = 0; l < lanes; ++l) {
        const float4 v = ps[l * used + c];
        merge(tn, tm, tq, v.x, v.y, v.z);
      }
      tab[c] = make_float2(tm, tq);
      if (c == 0) *total = tn;
    }
    __syncthreads();
  }
}

// f(group, lane, lanes) for the groups [0, ng) of a block, `lanes` neighbouring
// threads each, no more than 32 and no more than `most` is of use to; f runs in
// whole warps (and for groups at or past ng).
template <typename F>
__device__ __forceinline__ void each_group(int ng, int most, F&& f) {
  int lanes = 1;
  while (lanes < 32 && lanes < most && 2 * lanes * ng <= (int)blockDim.x) lanes *= 2;
  const int first = threadIdx.x / lanes;
  for (int g = first; g - first < ng; g += blockDim.x / lanes)
    f(g, (int)threadIdx.x & (lanes - 1), lanes);
}

// ONE: a vector's channels are all of one group; else channels are kept apart
// until the block's are merged.  Dynamic shared memory: the slots, the blocks'
// triples of the unit's groups, [3][cluster][ng], then (not ONE) the table of
// channel_stats and its partial triples.
template <typename T, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(kTeam, ONE || V < 8 ? 2 : 1)
    fwd_nhwc(Shape s, ColTeam tm, const T* x, const float* gamma, const float* beta, T* y,
             float* mean_out, float* rstd_out) {
  constexpr int P = Pairs<V>::n, EP = ONE ? 1 : P;
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ float2 ent[kTeam];
  __shared__ float cnts[kTeam];
  __shared__ float total_n;
  const bool many = tm.blocks > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const UnitCol<V> k(s, tm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int stride = kPieces<T, V> * kUnit<T, V> * blockDim.x;
  char* mine = reinterpret_cast<char*>(slots) + threadIdx.x * kUnit<T, V>;
  float* sn = reinterpret_cast<float*>(reinterpret_cast<char*>(slots) + (size_t)tm.held * stride);
  float* sm = sn + tm.blocks * tm.ng;
  float* sq = sm + tm.blocks * tm.ng;
  const int count = k.p1 > k.p0 ? (k.p1 - k.p0 + tm.rl - 1) / tm.rl : 0;  // this thread's pixels
  const int held = count < tm.held ? count : tm.held;
  const long long step = (long long)tm.rl * s.c;
  const T* px = x + k.base + (long long)k.p0 * s.c;
  {
    const T* p = px;
    char* slot = mine;
    for (int i = 0; i < held; ++i, p += step, slot += stride) {
      hold<T, V>(p, slot);
      if (i % kBatch == kBatch - 1 || i == held - 1) copy_group();
    }
  }
  float n = 0.f;
  Pairs<2 * EP> mean, m2;  // ONE: the first of a pair alone
#pragma unroll
  for (int e = 0; e < EP; ++e) mean.p[e] = m2.p[e] = both(0.f);
  // what is not held first: its loads go on behind the copies
  for (int i = held; i < count; i += kBatch)
    add_batch<V, ONE>(min(count - i, kBatch), n, mean, m2,
                      [&](int b, Pairs<V>& f) { load_vec<T, V>(px + (i + b) * step, f); });
  {
    const char* slot = mine;
    auto get = [&](int b, Pairs<V>& f) { take<T, V>(slot + b * stride, f); };
    int i = 0, open = (held + kBatch - 1) / kBatch;
    for (; i + kBatch <= held; i += kBatch, slot += kBatch * stride) {
      copy_wait(--open);
      add_batch<V, ONE>(kBatch, n, mean, m2, get);
    }
    if (i < held) {
      copy_wait(0);
      add_batch<V, ONE>(held - i, n, mean, m2, get);
    }
  }
  // the block's groups, to every block of the cluster
  auto send = [&](int g, int lane_g, int lanes, float gn, float gm, float gq) {
    const int at = k.rank * tm.ng + g;
    if (many) {
      for (int j = lane_g; j < tm.blocks; j += lanes) {
        store_cluster(&sn[at], j, gn);
        store_cluster(&sm[at], j, gm);
        store_cluster(&sq[at], j, gq);
      }
    } else if (lane_g == 0) {
      sn[at] = gn, sm[at] = gm, sq[at] = gq;
    }
  };
  if constexpr (ONE) {
    ent[threadIdx.x] = make_float2(mean.p[0].x, m2.p[0].x);
    cnts[threadIdx.x] = n;
    __syncthreads();
    if (many) cluster_wait();
    // a warp each: entries of every pixel lane and column
    const int cols = s.cpg / V;
    for (int g = warp; g < tm.ng; g += warps) {
      float ln = 0.f, lm = 0.f, lq = 0.f;
      for (int i = lane; i < cols * tm.rl; i += 32) {
        const int l = cols == 1 ? i : i / cols, th = l * tm.cb + g * cols + i - l * cols;
        const float2 v = ent[th];
        merge(ln, lm, lq, cnts[th], v.x, v.y);
      }
      const float c = warp_sum(ln);
      const float m = warp_sum(ln * lm) / fmaxf(c, 1.f);
      const float q = warp_sum(ln > 0.f ? fmaf(ln * (lm - m), lm - m, lq) : 0.f);
      send(g, lane, 32, c, m, q);
    }
  } else {
    float2* tab = reinterpret_cast<float2*>(sn + (3 * tm.blocks * tm.ng + 3) / 4 * 4);
    float4* ps = reinterpret_cast<float4*>(tab + ((tm.rows * tm.width + 1) & ~1));
    channel_stats<V>(tm.cb, tm.rl, tm.rows, tm.cb, k.lane, k.col, k.live, n, mean, m2, tab, cnts,
                     ps, &total_n);
    if (many) cluster_wait();
    const float cn = total_n;
    each_group(tm.ng, s.cpg, [&](int g, int lane_g, int lanes) {
      float ln = 0.f, lm = 0.f, lq = 0.f;
      if (g < tm.ng)
        for (int i = lane_g; i < s.cpg; i += lanes) {
          const float2 v = tab[g * s.cpg + i];
          merge(ln, lm, lq, cn, v.x, v.y);
        }
      const float c = row_sum(ln, lanes);
      const float m = row_sum(ln * lm, lanes) / fmaxf(c, 1.f);
      const float q = row_sum(ln > 0.f ? fmaf(ln * (lm - m), lm - m, lq) : 0.f, lanes);
      if (g < tm.ng) send(g, lane_g, lanes, c, m, q);
    });
  }
  if (many) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // a group's blocks, a lane each
  for (int g = warp; g < tm.ng; g += warps) {
    const int at = lane * tm.ng + g;
    const bool in = lane < tm.blocks && sn[at] > 0.f;
    const float mu = unit_mean(s, warp_sum(in ? sn[at] * sm[at] : 0.f));
    const float d = in ? sm[at] - mu : 0.f;
    const float var = warp_sum(in ? fmaf(sn[at] * d, d, sq[at]) : 0.f) * s.inv_total;
    const float rs = rsqrtf(var + s.eps);
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
    const float2 st = ent[quick_div(k.col * V + (ONE ? 0 : e), s.inv_cpg)];
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
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ float2 ps[kTeam];
  const bool many = tm.blocks > 1;
  if (many) cluster_arrive();
  pdl_wait();
  pdl_release();
  const UnitCol<V> k(s, tm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int stride = V * sizeof(T) * blockDim.x, stride_g = V * sizeof(SG) * blockDim.x;
  char* mine = reinterpret_cast<char*>(slots) + threadIdx.x * kUnit<T, V>;
  char* held_g = reinterpret_cast<char*>(slots) + (size_t)tm.held * stride;
  char* mine_g = held_g + threadIdx.x * kUnit<SG, V>;
  float2* tab = reinterpret_cast<float2*>(held_g + (size_t)tm.held * stride_g);
  float* sa = reinterpret_cast<float*>(tab + tm.rows * tm.width);
  float* sb = sa + tm.blocks * tm.ng;
  const int count = k.p1 > k.p0 ? (k.p1 - k.p0 + tm.rl - 1) / tm.rl : 0;
  const int held = count < tm.held ? count : tm.held;
  const long long step = (long long)tm.rl * s.c, off = k.base + (long long)k.p0 * s.c;
  {
    const T* p = x + off;
    const TG* pg = gy + off;
    char *slot = mine, *slot_g = mine_g;
    for (int i = 0; i < held; ++i) {
      hold<T, V>(p, slot);
      hold<TG, V>(pg, slot_g);
      if ((i & 1) || i == held - 1) copy_group();
      p += step, pg += step, slot += stride, slot_g += stride_g;
    }
  }
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
        const long long at = g0 + quick_div(k.col * V + e, s.inv_cpg);
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
  {
    const char* slot = mine;
    char* slot_g = mine_g;
    auto pixel = [&] {
      Pairs<V> f, d;
      take<T, V>(slot, f);
      take<TG, V>(slot_g, d);
      sums(f, d);
      if (KEEP) leave<V>(slot_g, d);
      slot += stride, slot_g += stride_g;
    };
    int open = (held + 1) / 2;
    for (int i = 0; i + 2 <= held; i += 2) {
      copy_wait(--open);
      pixel();
      pixel();
    }
    if (held & 1) {
      copy_wait(0);
      pixel();
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
      if (lane < tm.blocks) {
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
    const bool in = lane < tm.blocks;
    const float a1 = warp_sum(in ? sa[lane * tm.ng + q] : 0.f);
    const float b1 = warp_sum(in ? sb[lane * tm.ng + q] : 0.f);
    if (lane == 0) ps[q] = make_float2(a1 * s.inv_total, b1 * s.inv_total);
  }
  __syncthreads();
  if (!k.live) return;
  // grad_x = dz * (gamma * rstd) - rstd * s1 - xh * (rstd * s2)
  Pairs<ONE ? 1 : V> k1, k2;
  if (V == 1) k1.p[0] = k2.p[0] = both(0.f);
#pragma unroll
  for (int e = 0; e < (ONE ? 1 : V); ++e) {
    const float2 v = ps[quick_div(k.col * V + e, s.inv_cpg)];
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

// ---------------------------------------------------------------- two launches
//
// A thread streams its vectors through a ring of slots of its own: two batches
// arrive while one is worked on, without registers that wait.  The same loops
// on plain loads took, on 2 x 200 x 336 x 256 bf16 with SiLU, 69 us forward
// (now 43, bytes' time 20.3: x is read twice, the second time from L2) and
// 129 us backward (now 81, bytes' time 30.4).  Bound by instruction issue and
// by L2 for the second read.

// Whether a vector can be copied asynchronously (4 bytes at least).
template <typename T, int V>
constexpr bool kStreams = V * sizeof(T) >= 4;

// A block's slice of channels and share of pixels; neighbouring blocks take
// neighbouring slices of the same pixels.
template <int V>
struct Loose {
  long long base;  // of the image's first pixel, plus this column's channel
  int img, rank, slice, c0, cols, col, ch, lane, p0, count, g0, ng;  // groups [g0, g0 + ng)
  bool live;
  __device__ __forceinline__ Loose(const Shape& s, const ColTeam& tm, int img0) {
    const unsigned id = blockIdx.x / (unsigned)tm.slices;
    slice = (int)(blockIdx.x - id * tm.slices);
    const unsigned i = id / (unsigned)tm.blocks;
    rank = (int)(id - i * tm.blocks);
    img = img0 + (int)i;
    c0 = slice * tm.width;
    cols = min(tm.cb, (s.c - c0) / V);
    lane = quick_div(threadIdx.x, s.inv_cb);
    col = threadIdx.x - lane * tm.cb;
    live = lane < tm.rl && col < cols;
    ch = c0 + col * V;
    base = (long long)img * s.hw * s.c + ch;
    const long long first = (long long)rank * tm.span + lane;
    const long long end = min((long long)s.hw, (long long)(rank + 1) * tm.span);
    p0 = (int)first;
    count = live && first < end ? (int)((end - first + tm.rl - 1) / tm.rl) : 0;
    g0 = c0 / s.cpg;
    ng = (c0 + cols * V - 1) / s.cpg - g0 + 1;
  }
  // entry of group g (of the image) from this block: a group's entries are
  // [block][slice that shares it]
  __device__ __forceinline__ size_t entry(const Shape& s, const ColTeam& tm, int g) const {
    return (((size_t)img * s.groups + g) * tm.blocks + rank) * tm.shares +
           (slice - g * s.cpg / tm.width);
  }
};

// entry = (count, mean, M2) of a group's share of a block.
template <typename T, int V, bool ONE>
__global__ void __launch_bounds__(kTwo)
    stats_nhwc(Shape s, ColTeam tm, int img0, const T* x, float4* entry) {
  constexpr int P = Pairs<V>::n, EP = ONE ? 1 : P;
  // the ring's slots; then (not ONE) the table of channel_stats and its partial triples
  extern __shared__ __align__(128) uint4 slots[];
  float2* tab = reinterpret_cast<float2*>(slots);
  __shared__ float2 ent[kTwo];
  __shared__ float cnts[kTwo];
  __shared__ float total_n;
  pdl_wait();
  pdl_release();
  const Loose<V> k(s, tm, img0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long step = (long long)tm.rl * s.c;
  const T* px = x + k.base + (long long)k.p0 * s.c;
  float n = 0.f;
  Pairs<2 * EP> mean, m2;
#pragma unroll
  for (int e = 0; e < EP; ++e) mean.p[e] = m2.p[e] = both(0.f);
  if constexpr (kStreams<T, V>) {
    char* mine = reinterpret_cast<char*>(slots) + threadIdx.x * kUnit<T, V>;
    constexpr int stride = V * sizeof(T) * kTwo;
    through_ring<kBatch>(
        k.count,
        [&](int, int slot) {
          hold<T, V>(px, mine + slot * stride);
          px += step;
        },
        [&](int, int most, int slot) {
          const char* from = mine + slot * stride;
          auto get = [&](int b, Pairs<V>& f) { take<T, V>(from + b * stride, f); };
          if (most == kBatch)
            add_batch<V, ONE>(kBatch, n, mean, m2, get);
          else
            add_batch<V, ONE>(most, n, mean, m2, get);
        });
    __syncthreads();  // (the table takes the slots' place)
  } else {
    auto get = [&](int b, Pairs<V>& f) { load_vec<T, V>(px + b * step, f); };
    for (int i = 0; i < k.count; i += kBatch, px += kBatch * step)
      add_batch<V, ONE>(min(k.count - i, kBatch), n, mean, m2, get);
  }
  if constexpr (ONE) {
    ent[threadIdx.x] = make_float2(mean.p[0].x, m2.p[0].x);
    cnts[threadIdx.x] = n;
    __syncthreads();
    for (int q = warp; q < k.ng; q += kTwo / 32) {
      const int g = k.g0 + q;  // its columns in this block
      const int j0 = max(0, g * s.cpg - k.c0) / V;
      const int cols = min(k.cols, ((g + 1) * s.cpg - k.c0) / V) - j0;
      float ln = 0.f, lm = 0.f, lq = 0.f;
      for (int i = lane; i < cols * tm.rl; i += 32) {
        const int l = cols == 1 ? i : i / cols, th = l * tm.cb + j0 + i - l * cols;
        const float2 v = ent[th];
        merge(ln, lm, lq, cnts[th], v.x, v.y);
      }
      const float c = warp_sum(ln);
      const float m = warp_sum(ln * lm) / fmaxf(c, 1.f);
      const float t = warp_sum(ln > 0.f ? fmaf(ln * (lm - m), lm - m, lq) : 0.f);
      if (lane == 0) entry[k.entry(s, tm, g)] = make_float4(c, m, t, 0.f);
    }
  } else {
    float4* ps = reinterpret_cast<float4*>(tab + ((tm.rows * tm.width + 1) & ~1));
    channel_stats<V>(tm.cb, tm.rl, tm.rows, k.cols, k.lane, k.col, k.live, n, mean, m2, tab, cnts,
                     ps, &total_n);
    const float cn = total_n;
    const int used = k.cols * V;
    each_group(k.ng, s.cpg, [&](int q, int lane_g, int lanes) {
      const int g = k.g0 + q, c1 = min(used, (g + 1) * s.cpg - k.c0);
      float ln = 0.f, lm = 0.f, lq = 0.f;
      if (q < k.ng)
        for (int c = max(0, g * s.cpg - k.c0) + lane_g; c < c1; c += lanes) {
          const float2 v = tab[c];
          merge(ln, lm, lq, cn, v.x, v.y);
        }
      const float c = row_sum(ln, lanes);
      const float m = row_sum(ln * lm, lanes) / fmaxf(c, 1.f);
      const float t = row_sum(ln > 0.f ? fmaf(ln * (lm - m), lm - m, lq) : 0.f, lanes);
      if (q < k.ng && lane_g == 0) entry[k.entry(s, tm, g)] = make_float4(c, m, t, 0.f);
    });
  }
}

// The entries [first, first + count) of a group: its blocks', and in each the
// slices' that share it.
__device__ __forceinline__ size_t group_entry(const Shape& s, const ColTeam& tm, int img, int g,
                                              int i, int shared) {
  const int b = shared == 1 ? i : i / shared;
  return (((size_t)img * s.groups + g) * tm.blocks + b) * tm.shares + (i - b * shared);
}
__device__ __forceinline__ int group_shared(const Shape& s, const ColTeam& tm, int g) {
  return ((g + 1) * s.cpg - 1) / tm.width - g * s.cpg / tm.width + 1;
}

template <typename T, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(kTwo)
    apply_nhwc(Shape s, ColTeam tm, int img0, const T* x, const float* gamma, const float* beta,
               const float4* entry, T* y, float* mean_out, float* rstd_out) {
  constexpr int P = Pairs<V>::n;
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ float2 ent[kTwo];
  pdl_wait();
  pdl_release();
  const Loose<V> k(s, tm, img0);
  each_group(k.ng, 32, [&](int q, int lane, int lanes) {
    float n = 0.f, mean = 0.f, m2 = 0.f;
    const int g = k.g0 + q;
    if (q < k.ng) {
      const int shared = group_shared(s, tm, g);
#pragma unroll 4
      for (int i = lane; i < tm.blocks * shared; i += lanes) {
        const float4 v = entry[group_entry(s, tm, k.img, g, i, shared)];
        merge(n, mean, m2, v.x, v.y, v.z);
      }
    }
    const float mu = unit_mean(s, row_sum(n * mean, lanes));
    const float var =
        row_sum(n > 0.f ? fmaf(n * (mean - mu), mean - mu, m2) : 0.f, lanes) * s.inv_total;
    if (q < k.ng && lane == 0) {
      const float rs = rsqrtf(var + s.eps);
      ent[q] = make_float2(mu, rs);
      if (k.rank == 0 && g * s.cpg / tm.width == k.slice) {
        const long long to = (long long)k.img * s.groups + g;
        if (mean_out) mean_out[to] = mu;
        if (rstd_out) rstd_out[to] = rs;
      }
    }
  });
  __syncthreads();
  if (!k.live) return;
  Pairs<ONE ? 1 : V> mu;  // minus the mean
  Pairs<V> a, b;
  if (V == 1) a.p[0] = b.p[0] = mu.p[0] = both(0.f);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float2 st = ent[quick_div(k.ch + (ONE ? 0 : e), s.inv_cpg) - k.g0];
    mu[ONE ? 0 : e] = -st.x;
    a[e] = st.y * (gamma ? gamma[k.ch + e] : 1.f);
    b[e] = beta ? beta[k.ch + e] : 0.f;
  }
  const long long step = (long long)tm.rl * s.c;
  const T* px = x + k.base + (long long)k.p0 * s.c;
  T* to = y + k.base + (long long)k.p0 * s.c;
  // (an item's copy is done before its store, which may be in place)
  auto pixels = [&](int most, auto&& get) {
    Pairs<V> f[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i < most) get(i, f[i]);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i >= most) break;
#pragma unroll
      for (int e = 0; e < P; ++e)
        f[i].p[e] = act_fwd2<ACT>(fma2(add2(f[i].p[e], ONE ? both(mu[0]) : mu.p[ONE ? 0 : e]),
                                       a.p[e], b.p[e]), s.floor);
      store_vec<T, V>(to + i * step, f[i]);
    }
    to += kBatch * step;
  };
  if constexpr (kStreams<T, V>) {
    char* mine = reinterpret_cast<char*>(slots) + threadIdx.x * kUnit<T, V>;
    constexpr int stride = V * sizeof(T) * kTwo;
    through_ring<kBatch>(
        k.count,
        [&](int, int slot) {
          hold<T, V>(px, mine + slot * stride);
          px += step;
        },
        [&](int, int most, int slot) {
          const char* from = mine + slot * stride;
          pixels(most, [&](int i, Pairs<V>& f) { take<T, V>(from + i * stride, f); });
        });
  } else {
    for (int i = 0; i < k.count; i += kBatch, px += kBatch * step)
      pixels(min(k.count - i, kBatch),
             [&](int j, Pairs<V>& f) { load_vec<T, V>(px + j * step, f); });
  }
}

// part[rank][image * c + channel] as above; entry = a block's sums of gamma dz
// and gamma dz xh over a group's share.
template <typename T, typename TG, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(kTwo)
    sums_nhwc(Shape s, ColTeam tm, int img0, const T* x, const TG* gy, const float* gamma,
              const float* beta, const float* mean, const float* rstd, float2* part,
              float2* entry) {
  constexpr int P = Pairs<V>::n;
  extern __shared__ __align__(128) uint4 slots[];  // the ring's; then the table
  float2* tab = reinterpret_cast<float2*>(slots);
  pdl_wait();
  pdl_release();
  const Loose<V> k(s, tm, img0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
        const long long at = (long long)k.img * s.groups + quick_div(k.ch + e, s.inv_cpg);
        mu[ONE ? 0 : e] = -mean[at], rs[ONE ? 0 : e] = rstd[at];
      }
      g[e] = gamma ? gamma[k.ch + e] : 1.f;
      b[e] = beta ? beta[k.ch + e] : 0.f;
    }
  }
  const long long step = (long long)tm.rl * s.c, off = k.base + (long long)k.p0 * s.c;
  const T* px = x + off;
  const TG* pg = gy + off;
  auto pixel = [&](const Pairs<V>& f, const Pairs<V>& d) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const float2 xh = mul2(add2(f.p[e], ONE ? both(mu[0]) : mu.p[ONE ? 0 : e]),
                             ONE ? both(rs[0]) : rs.p[ONE ? 0 : e]);
      float2 dz = act_bwd2<ACT>(fma2(xh, g.p[e], b.p[e]), d.p[e], s.floor);
      if (V == 1) dz.y = 0.f;
      s1.p[e] = add2(s1.p[e], dz);
      s2.p[e] = fma2(dz, xh, s2.p[e]);
    }
  };
  if constexpr (kStreams<T, V> && kStreams<TG, V>) {
    char* mine = reinterpret_cast<char*>(slots) + threadIdx.x * kUnit<T, V>;
    char* mine_g = reinterpret_cast<char*>(slots) + kRing * 2 * V * sizeof(T) * kTwo +
                   threadIdx.x * kUnit<TG, V>;
    constexpr int stride = V * sizeof(T) * kTwo, stride_g = V * sizeof(TG) * kTwo;
    through_ring<2>(
        k.count,
        [&](int, int slot) {
          hold<T, V>(px, mine + slot * stride);
          hold<TG, V>(pg, mine_g + slot * stride_g);
          px += step;
          pg += step;
        },
        [&](int, int most, int slot) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i >= most) break;
            Pairs<V> f, d;
            take<T, V>(mine + (slot + i) * stride, f);
            take<TG, V>(mine_g + (slot + i) * stride_g, d);
            pixel(f, d);
          }
        });
    __syncthreads();  // (the table takes the slots' place)
  } else {
    for (int i = 0; i < k.count; ++i, px += step, pg += step) {
      Pairs<V> f, d;
      load_vec<T, V>(px, f);
      load_vec<TG, V>(pg, d);
      pixel(f, d);
    }
  }
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
    put = lane < tm.cb && k.col < k.cols;
  }
  if (put) {
#pragma unroll
    for (int e = 0; e < V; ++e) tab[row * tm.width + k.col * V + e] = make_float2(s1[e], s2[e]);
  }
  __syncthreads();
  const int width = k.cols * V;
  for (int c = threadIdx.x; c < width; c += kTwo) {
    float2 t = tab[c];
    for (int l = 1; l < tm.rows; ++l) {
      const float2 v = tab[l * tm.width + c];
      t.x += v.x;
      t.y += v.y;
    }
    part[((long long)k.rank * s.n + k.img) * s.c + k.c0 + c] = t;
    const float gm = gamma ? gamma[k.c0 + c] : 1.f;
    tab[c] = make_float2(gm * t.x, gm * t.y);
  }
  __syncthreads();
  for (int q = warp; q < k.ng; q += kTwo / 32) {
    const int gr = k.g0 + q;
    const int c1 = min(width, (gr + 1) * s.cpg - k.c0);
    float a1 = 0.f, b1 = 0.f;
    for (int c = max(0, gr * s.cpg - k.c0) + lane; c < c1; c += 32) {
      a1 += tab[c].x;
      b1 += tab[c].y;
    }
    a1 = warp_sum(a1);
    b1 = warp_sum(b1);
    if (lane == 0) entry[k.entry(s, tm, gr)] = make_float2(a1, b1);
  }
}

// Three blocks to an SM, as the grid is made for, are 80 registers a thread;
// the other activations' float32 gradients would spill there and have no bound,
// which is 0 (2 x 200 x 336 x 256: ReLU 144 -> 123 us, but SiLU 128 -> 147).
template <typename T, typename TG, int V, bool ONE, int ACT>
__global__ void __launch_bounds__(kTwo, ONE && (ACT == 0 || sizeof(TG) == 2) ? 3 : 0)
    grads_nhwc(Shape s, ColTeam tm, int img0, const T* x, const TG* gy, const float* gamma,
               const float* beta, const float* mean, const float* rstd, const float2* entry,
               T* gx) {
  constexpr int P = Pairs<V>::n;
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ float2 ent[kTwo];
  pdl_wait();
  pdl_release();
  const Loose<V> k(s, tm, img0);
  each_group(k.ng, 32, [&](int q, int lane, int lanes) {
    float a1 = 0.f, b1 = 0.f;
    const int g = k.g0 + q;
    if (q < k.ng) {
      const int shared = group_shared(s, tm, g);
#pragma unroll 4
      for (int i = lane; i < tm.blocks * shared; i += lanes) {
        const float2 v = entry[group_entry(s, tm, k.img, g, i, shared)];
        a1 += v.x;
        b1 += v.y;
      }
    }
    a1 = row_sum(a1, lanes);
    b1 = row_sum(b1, lanes);
    if (q < k.ng && lane == 0) ent[q] = make_float2(a1 * s.inv_total, b1 * s.inv_total);
  });
  __syncthreads();
  if (!k.live) return;
  // grad_x = dz * (gamma * rstd) - rstd * s1 - xh * (rstd * s2)
  Pairs<ONE ? 1 : V> mu, rs, k1, k2;
  Pairs<V> g, b;
  if (V == 1) {
    mu.p[0] = rs.p[0] = k1.p[0] = k2.p[0] = both(0.f);
    g.p[0] = b.p[0] = both(0.f);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (!ONE || e == 0) {
      const int gr = quick_div(k.ch + e, s.inv_cpg);
      const long long at = (long long)k.img * s.groups + gr;
      const float2 v = ent[gr - k.g0];
      mu[ONE ? 0 : e] = -mean[at], rs[ONE ? 0 : e] = rstd[at];
      k1[ONE ? 0 : e] = -rstd[at] * v.x, k2[ONE ? 0 : e] = -rstd[at] * v.y;
    }
    g[e] = gamma ? gamma[k.ch + e] : 1.f;
    b[e] = beta ? beta[k.ch + e] : 0.f;
  }
  const long long step = (long long)tm.rl * s.c, off = k.base + (long long)k.p0 * s.c;
  const T* px = x + off;
  const TG* pg = gy + off;
  T* to = gx + off;
  constexpr int B = 2;
  // (an item's copies are done before its store, which may be in place)
  auto pixels = [&](int most, auto&& get) {
    Pairs<V> f[B], d[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (i < most) get(i, f[i], d[i]);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (i >= most) break;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 r = ONE ? both(rs[0]) : rs.p[ONE ? 0 : e];
        const float2 xh = mul2(add2(f[i].p[e], ONE ? both(mu[0]) : mu.p[ONE ? 0 : e]), r);
        const float2 dz = act_bwd2<ACT>(fma2(xh, g.p[e], b.p[e]), d[i].p[e], s.floor);
        f[i].p[e] = fma2(xh, ONE ? both(k2[0]) : k2.p[ONE ? 0 : e],
                         fma2(dz, mul2(g.p[e], r), ONE ? both(k1[0]) : k1.p[ONE ? 0 : e]));
      }
      store_vec<T, V>(to + i * step, f[i]);
    }
    to += B * step;
  };
  if constexpr (kStreams<T, V> && kStreams<TG, V>) {
    char* mine = reinterpret_cast<char*>(slots) + threadIdx.x * kUnit<T, V>;
    char* mine_g = reinterpret_cast<char*>(slots) + kRing * 2 * V * sizeof(T) * kTwo +
                   threadIdx.x * kUnit<TG, V>;
    constexpr int stride = V * sizeof(T) * kTwo, stride_g = V * sizeof(TG) * kTwo;
    through_ring<B>(
        k.count,
        [&](int, int slot) {
          hold<T, V>(px, mine + slot * stride);
          hold<TG, V>(pg, mine_g + slot * stride_g);
          px += step;
          pg += step;
        },
        [&](int, int most, int slot) {
          pixels(most, [&](int i, Pairs<V>& f, Pairs<V>& d) {
            take<T, V>(mine + (slot + i) * stride, f);
            take<TG, V>(mine_g + (slot + i) * stride_g, d);
          });
        });
  } else {
    for (int i = 0; i < k.count; i += B, px += B * step, pg += B * step)
      pixels(min(k.count - i, B), [&](int j, Pairs<V>& f, Pairs<V>& d) {
        load_vec<T, V>(px + j * step, f);
        load_vec<TG, V>(pg + j * step, d);
      });
  }
}

}  // namespace

cudaError_t launch_nhwc(const NormPlan& p, const NormArgs& a, bool backward,
                             cudaStream_t st) {
  const int cpg = p.s.cpg;
  if (!backward)
    return by_dtype(a.dt, [&](auto t) {
      using T = decltype(t);
      return by_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        return by_width<T>(p.s.v, [&](auto w) {
          constexpr int V = decltype(w)::value;
          auto go = [&](auto kern) {
            return launch_team(kern, p, p.col.blocks, st, p.s, p.col, static_cast<const T*>(a.x),
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
      return by_width<T>(p.s.v, [&](auto w) {
        constexpr int V = decltype(w)::value;
        auto go = [&](auto kern) {
          return launch_team(kern, p, p.col.blocks, st, p.s, p.col, static_cast<const T*>(a.x),
                             static_cast<const TG*>(a.gy), a.gamma, a.beta,
                             static_cast<const float*>(a.mean), static_cast<const float*>(a.rstd),
                             static_cast<T*>(a.gx), reinterpret_cast<float2*>(a.ws));
        };
        return cpg % V ? go(bwd_nhwc<T, TG, V, false, ACT>) : go(bwd_nhwc<T, TG, V, true, ACT>);
      });
    });
  });
}

cudaError_t launch_two_nhwc(const NormPlan& p, const NormArgs& a, bool backward, bool second,
                            int img0, int count, cudaStream_t st) {
  const unsigned grid = (unsigned)count * p.col.blocks * p.col.slices;
  char* entry = a.ws + norm_part_bytes(p, a, backward);
  if (!backward)
    return by_dtype(a.dt, [&](auto t) {
      using T = decltype(t);
      const T* x = static_cast<const T*>(a.x);
      float4* e = reinterpret_cast<float4*>(entry);
      return by_width<T>(p.s.v, [&](auto w) {
        constexpr int V = decltype(w)::value;
        auto by_one = [&](auto one) {
          constexpr bool ONE = decltype(one)::value != 0;
          if (!second)
            return launch_smem(stats_nhwc<T, V, ONE>, grid, kTwo, p.smem, st, p.s, p.col, img0, x, e);
          return by_act(a.act, [&](auto act) {
            return launch_smem(apply_nhwc<T, V, ONE, decltype(act)::value>, grid, kTwo, p.smem, st,
                               p.s, p.col, img0, x, a.gamma, a.beta, static_cast<const float4*>(e),
                                static_cast<T*>(a.y), a.mean, a.rstd);
          });
        };
        return p.s.cpg % V ? by_one(Int<0>{}) : by_one(Int<1>{});
      });
    });
  return by_dtypes(a, [&](auto t, auto g) {
    using T = decltype(t);
    using TG = decltype(g);
    const T* x = static_cast<const T*>(a.x);
    const TG* gy = static_cast<const TG*>(a.gy);
    const float *mean = a.mean, *rstd = a.rstd;
    float2* e = reinterpret_cast<float2*>(entry);
    return by_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      return by_width<T>(p.s.v, [&](auto w) {
        constexpr int V = decltype(w)::value;
        auto by_one = [&](auto one) {
          constexpr bool ONE = decltype(one)::value != 0;
          if (!second)
            return launch_smem(sums_nhwc<T, TG, V, ONE, ACT>, grid, kTwo, p.smem, st, p.s, p.col, img0,
                               x, gy, a.gamma, a.beta, mean, rstd,
                               reinterpret_cast<float2*>(a.ws), e);
          return launch_smem(grads_nhwc<T, TG, V, ONE, ACT>, grid, kTwo, p.smem, st, p.s, p.col, img0,
                             x, gy, a.gamma, a.beta, mean, rstd, static_cast<const float2*>(e),
                              static_cast<T*>(a.gx));
        };
        return p.s.cpg % V ? by_one(Int<0>{}) : by_one(Int<1>{});
      });
    });
  });
}

}  // namespace dc
