// Group norm with an activation on [n][c][h][w] tensors, one launch.
//
// A group of an image is a unit: cpg rows of h * w consecutive elements, held
// in the shared memory of a cluster's blocks from the statistics to the
// results, so that x (and grad_y) come from memory once.  A lane copies the
// 16-byte vectors that it works on itself, asynchronously and all at once: no
// registers wait for the loads, and no barrier stands between a copy and its
// use.  The loops over the vectors stay rolled: a block runs its code once,
// and a body unrolled over the vectors costs more in instruction fetches than
// it saves.  What does not fit is read again (from L2) for the results.
#include "dc_norm.cuh"

namespace dc {
namespace {

// A warp's task t of a unit: 32 / lpr rows, one segment of each.
template <int VEC, bool EVEN>
struct UnitTask {
  long long row, off;  // off: the row's first vector in elements (aligned)
  int ch, part, mis, v0, v1, last, tail;  // tail: elements of the row in its vector `last`
  bool live;
  __device__ __forceinline__ UnitTask(const Shape& s, unsigned unit, int ch0, int t, int tasks) {
    const int lane = threadIdx.x & 31, per = 32 / s.t.lpr;
    const int blk = s.t.parts == 1 ? t : t / s.t.parts;
    part = t - blk * s.t.parts;
    const int local = blk * per + lane / s.t.lpr;
    live = t < tasks && local < s.cpg;
    row = (long long)unit * s.cpg + (live ? local : 0);
    ch = ch0 + (live ? local : 0);
    const long long first = row * s.hw;
    mis = EVEN ? 0 : (int)first & (VEC - 1);
    off = first - mis;
    v0 = part * s.t.seg + (lane & (s.t.lpr - 1));
    const int end = part * s.t.seg + s.t.seg, vr = row_vectors(s.hw, mis, VEC);
    v1 = !live ? v0 : end < vr ? end : vr;
    last = vr - 1;
    tail = s.hw + mis - last * VEC;
  }
  // the elements [lo, hi) of vector v lie in the row
  __device__ __forceinline__ int lo(int v) const { return EVEN || v ? 0 : mis; }
  __device__ __forceinline__ int hi(int v) const { return EVEN || v != last ? VEC : tail; }
};

// A vector of VEC elements as it lies in memory: one or two 16-byte pieces.
template <typename T, int VEC>
struct Raw {
  static constexpr int n = VEC * sizeof(T) / 16;
  uint4 w[n];
  __device__ __forceinline__ void unpack(Pairs<VEC>& f) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e)
      f.p[e] = sizeof(T) == 4
                   ? make_float2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]))
                   : make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u));
  }
};

// Starts the copies of a task's vectors to this thread's slots.
template <typename T, int VEC, bool EVEN>
__device__ __forceinline__ void hold_task(const Shape& s, const UnitTask<VEC, EVEN>& k, const T* x,
                                          uint4* slot) {
  for (int v = k.v0; v < k.v1; v += s.t.lpr) {
    const T* p = x + k.off + (long long)v * VEC;
    const int bytes = EVEN ? VEC * (int)sizeof(T) : k.hi(v) * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::n; ++i) {
      // (a piece past the row's end is skipped; its slot is not used)
      const int b = min(16, bytes - 16 * i);
      if (EVEN || b > 0)
        copy_async<16>(slot, reinterpret_cast<const char*>(p) + 16 * i, EVEN ? 16 : b);
      slot += blockDim.x;
    }
  }
}

// Vector v of a task, from this thread's slot or from memory; what lies
// outside the row is 0.
template <typename T, int VEC, bool EVEN>
__device__ __forceinline__ void fetch(const UnitTask<VEC, EVEN>& k, int v, const T* x, bool held,
                                      const uint4* slot, Pairs<VEC>& f) {
  const T* p = x + k.off + (long long)v * VEC;
  const int lo = k.lo(v), hi = k.hi(v);
  const bool full = EVEN || (lo == 0 && hi == VEC);
  if (held) {
    Raw<T, VEC> r;
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::n; ++i) r.w[i] = slot[i * blockDim.x];
    r.unpack(f);
    if (!full) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < lo || e >= hi) f[e] = 0.f;
    }
  } else if (full) {
    load_vec<T, VEC>(p, f);
  } else {
    float t[VEC];
    load_part<T, VEC>(p, lo, hi, t);
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = t[e];
  }
}

template <typename T, int VEC, bool EVEN>
__device__ __forceinline__ void put(const UnitTask<VEC, EVEN>& k, int v, T* y,
                                    const Pairs<VEC>& f) {
  T* p = y + k.off + (long long)v * VEC;
  const int lo = k.lo(v), hi = k.hi(v);
  if (EVEN || (lo == 0 && hi == VEC)) {
    store_vec<T, VEC>(p, f);
  } else {
    float t[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) t[e] = f[e];
    store_part<T, VEC>(p, lo, hi, t);
  }
}

// This thread's place: block `rank` of the cluster, warp w of the unit's.
struct Place {
  int rank, u, w, team, ch0;  // ch0: the unit's first channel
  unsigned unit;
  bool here;
  __device__ __forceinline__ Place(const Shape& s, const RowTeam& tm) {
    const int warp = threadIdx.x >> 5;
    rank = cluster_rank();
    u = tm.units == 1 ? 0 : warp / tm.warps;
    w = warp - u * tm.warps;
    unit = cluster_id() * tm.units + u;  // (n * c is below 2^31)
    here = unit < (unsigned)s.n * s.groups;
    if (!here) unit = 0;
    ch0 = (int)(unit % (unsigned)s.groups) * s.cpg;
    team = tm.cluster * tm.warps;
  }
  __device__ __forceinline__ int task(const RowTeam& tm, int r) const {
    return rank * tm.warps + w + r * team;
  }
};

// a and b (of lane 0) of every warp of the unit, in the unit's every block:
// entries [0, team) of sa, sb.
template <int N>
__device__ __forceinline__ const float* share(const RowTeam& tm, const Place& pl,
                                              float (&sm)[N][256], const float (&val)[N]) {
  const int lane = threadIdx.x & 31, at = pl.rank * tm.warps + pl.w;
  if (tm.cluster > 1) {
    cluster_wait();  // every block of the cluster runs
    if (lane < tm.cluster)
#pragma unroll
      for (int i = 0; i < N; ++i) store_cluster(&sm[i][at], lane, val[i]);
    cluster_arrive();
    cluster_wait();
    return sm[0];
  }
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) sm[i][threadIdx.x >> 5] = val[i];
  __syncthreads();
  return sm[0] + pl.u * tm.warps;
}

// The unit's mean and 1 / sqrt(var + eps) from its lanes' triples.
__device__ __forceinline__ float2 unit_stats(const Shape& s, const RowTeam& tm, const Place& pl,
                                             float (&sm)[3][256], float n, float mean, float m2) {
  float val[3];
  val[0] = warp_sum(n);
  val[1] = warp_sum(n * mean) / fmaxf(val[0], 1.f);
  val[2] = warp_sum(n > 0.f ? fmaf(n * (mean - val[1]), mean - val[1], m2) : 0.f);
  const float* sn = share<3>(tm, pl, sm, val);
  const int lane = threadIdx.x & 31;
  float sum = 0.f, q = 0.f;
  for (int i = lane; i < pl.team; i += 32) sum = fmaf(sn[i], sn[256 + i], sum);
  const float total = (float)s.hw * (float)s.cpg;
  const float mu = warp_sum(sum) / total;
  for (int i = lane; i < pl.team; i += 32) {
    const float d = sn[256 + i] - mu;
    if (sn[i] > 0.f) q += fmaf(sn[i] * d, d, sn[512 + i]);
  }
  return make_float2(mu, 1.f / sqrtf(warp_sum(q) / total + s.eps));
}

constexpr int kBatch = 4;

template <typename T, bool EVEN, int ACT>
__global__ void __launch_bounds__(kTeam, 2)
    fwd_nchw(Shape s, RowTeam tm, const T* x, const float* gamma, const float* beta, T* y,
             float* mean_out, float* rstd_out) {
  constexpr int VEC = VecOf<T>::n;
  extern __shared__ uint4 hold[];
  __shared__ float sm[3][256];
  if (tm.cluster > 1) cluster_arrive();
  pdl_wait();
  pdl_release();
  const Place pl(s, tm);
  const int tasks = pl.here ? tm.tasks : 0, pitch = tm.slots * blockDim.x;
  using Task = UnitTask<VEC, EVEN>;
  const Task first(s, pl.unit, pl.ch0, pl.task(tm, 0), tasks);
  auto task = [&](int r) {
    return r == 0 ? first : Task(s, pl.unit, pl.ch0, pl.task(tm, r), tasks);
  };
  uint4* mine = hold + threadIdx.x;
  for (int r = 0; r < tm.held; ++r) hold_task<T, VEC, EVEN>(s, task(r), x, mine + r * pitch);
  // what is not held first: its loads go on behind the copies
  float n = 0.f, mean = 0.f, m2 = 0.f;
  for (int r = tm.rounds - 1; r >= 0; --r) {
    const Task k = task(r);
    const bool held = r < tm.held;
    const uint4* slot = mine + r * pitch;
    if (r == tm.held - 1) copy_wait();
    for (int v0 = k.v0; v0 < k.v1; v0 += kBatch * s.t.lpr) {
      Pairs<VEC> f[kBatch];
      float2 sum = both(0.f), q = both(0.f);
      int cnt = 0;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int v = v0 + b * s.t.lpr;
        if (v >= k.v1) continue;
        fetch<T, VEC, EVEN>(k, v, x, held, slot + b * blockDim.x, f[b]);
        cnt += k.hi(v) - k.lo(v);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) sum = add2(sum, f[b].p[e]);
      }
      const float mb = (sum.x + sum.y) * rcp_approx((float)cnt);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int v = v0 + b * s.t.lpr;
        if (v >= k.v1) continue;
        if (!EVEN && k.hi(v) - k.lo(v) < VEC) {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (e < k.lo(v) || e >= k.hi(v)) f[b][e] = mb;  // adds nothing below
        }
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const float2 d = add2(f[b].p[e], both(-mb));
          q = fma2(d, d, q);
        }
      }
      merge(n, mean, m2, (float)cnt, mb, q.x + q.y);
      slot += kBatch * blockDim.x;
    }
  }
  const float2 st = unit_stats(s, tm, pl, sm, n, mean, m2);
  if (!pl.here) return;
  if (pl.rank == 0 && pl.w == 0 && (threadIdx.x & 31) == 0) {
    if (mean_out) mean_out[pl.unit] = st.x;
    if (rstd_out) rstd_out[pl.unit] = st.y;
  }
  for (int r = 0; r < tm.rounds; ++r) {
    const Task k = task(r);
    const bool held = r < tm.held;
    const uint4* slot = mine + r * pitch;
    const float a = st.y * (gamma ? gamma[k.ch] : 1.f), b = beta ? beta[k.ch] : 0.f;
#pragma unroll 2
    for (int v = k.v0; v < k.v1; v += s.t.lpr) {
      Pairs<VEC> f;
      fetch<T, VEC, EVEN>(k, v, x, held, slot, f);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) f.p[e] = fma2(add2(f.p[e], both(-st.x)), both(a), both(b));
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = act_fwd<ACT>(f[e], s.floor);
      put<T, VEC, EVEN>(k, v, y, f);
      slot += blockDim.x;
    }
  }
}

// Rows of whole vectors: a unit is one run of vectors, dealt evenly over the
// threads whatever the rows' length; a vector's channel follows from its
// place.
template <typename T, int ACT>
__global__ void __launch_bounds__(kTeam, 2)
    fwd_flat(Shape s, RowTeam tm, const T* x, const float* gamma, const float* beta, T* y,
             float* mean_out, float* rstd_out) {
  constexpr int VEC = VecOf<T>::n;
  extern __shared__ uint4 hold[];
  __shared__ float sm[3][256];
  if (tm.cluster > 1) cluster_arrive();
  pdl_wait();
  pdl_release();
  const Place pl(s, tm);
  const int threads = 32 * tm.warps, tid = threadIdx.x - pl.u * threads;
  const int vr = s.hw / VEC;
  const long long first = (long long)pl.unit * s.cpg * s.hw;
  const int begin = pl.rank * tm.span + tid;
  int end = s.cpg * vr;  // (a unit of over 2^30 vectors does not come here)
  if (end > (pl.rank + 1) * tm.span) end = (pl.rank + 1) * tm.span;
  if (!pl.here) end = 0;
  x += first;
  y += first;
  uint4* mine = hold + threadIdx.x;
  {
    uint4* slot = mine;
    for (int i = 0, v = begin; i < tm.held && v < end; ++i, v += threads, slot += blockDim.x)
      copy_async<16>(slot, x + (long long)v * VEC);
  }
  float n = 0.f, mean = 0.f, m2 = 0.f;
  auto batches = [&](int i0, int i1) {
    for (int i = i0; i < i1; i += kBatch) {
      const int v0 = begin + i * threads;
      if (v0 >= end) break;
      Pairs<VEC> f[kBatch];
      float2 sum = both(0.f), q = both(0.f);
      int cnt = 0;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int v = v0 + b * threads;
        if (i + b >= i1 || v >= end) continue;
        Raw<T, VEC> r;
        r.w[0] = i + b < tm.held ? mine[(i + b) * blockDim.x]
                                 : *reinterpret_cast<const uint4*>(x + (long long)v * VEC);
        r.unpack(f[b]);
        cnt += VEC;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) sum = add2(sum, f[b].p[e]);
      }
      const float mb = (sum.x + sum.y) * rcp_approx((float)cnt);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (i + b >= i1 || v0 + b * threads >= end) continue;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const float2 d = add2(f[b].p[e], both(-mb));
          q = fma2(d, d, q);
        }
      }
      merge(n, mean, m2, (float)cnt, mb, q.x + q.y);
    }
  };
  batches(tm.held, tm.slots);  // what is not held, behind the copies
  copy_wait();
  batches(0, tm.held);
  const float2 st = unit_stats(s, tm, pl, sm, n, mean, m2);
  if (!pl.here) return;
  if (pl.rank == 0 && tid == 0) {
    if (mean_out) mean_out[pl.unit] = st.x;
    if (rstd_out) rstd_out[pl.unit] = st.y;
  }
  // vector `begin + i * threads` lies in channel c, `at` vectors from its start
  int c = begin / vr, at = begin - c * vr;
  const float* gm = gamma ? gamma + pl.ch0 : nullptr;
  const float* bt = beta ? beta + pl.ch0 : nullptr;
#pragma unroll 2
  for (int i = 0, v = begin; v < end; ++i, v += threads) {
    const float a = st.y * (gm ? gm[c] : 1.f), b = bt ? bt[c] : 0.f;
    Raw<T, VEC> r;
    r.w[0] = i < tm.held ? mine[i * blockDim.x]
                         : *reinterpret_cast<const uint4*>(x + (long long)v * VEC);
    Pairs<VEC> f;
    r.unpack(f);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) f.p[e] = fma2(add2(f.p[e], both(-st.x)), both(a), both(b));
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = act_fwd<ACT>(f[e], s.floor);
    store_vec<T, VEC>(y + (long long)v * VEC, f);
    c += tm.step_c;
    at += tm.step_v;
    if (at >= vr) at -= vr, ++c;
  }
}

// part[segment][image * c + channel]: the sums of dz and dz * xh of a row's
// segment.
template <typename T, typename TG, bool EVEN, int ACT>
__global__ void __launch_bounds__(kTeam, 2)
    bwd_nchw(Shape s, RowTeam tm, const T* x, const TG* gy, const float* gamma, const float* beta,
             const float* mean, const float* rstd, T* gx, float2* part) {
  constexpr int VEC = VecOf<T>::n;
  constexpr int kX = Raw<T, VEC>::n, kG = Raw<TG, VEC>::n;
  extern __shared__ uint4 hold[];
  __shared__ float sm[2][256];
  if (tm.cluster > 1) cluster_arrive();
  pdl_wait();
  pdl_release();
  const Place pl(s, tm);
  const int tasks = pl.here ? tm.tasks : 0, pitch = tm.slots * blockDim.x;
  using Task = UnitTask<VEC, EVEN>;
  const Task first(s, pl.unit, pl.ch0, pl.task(tm, 0), tasks);
  auto task = [&](int r) {
    return r == 0 ? first : Task(s, pl.unit, pl.ch0, pl.task(tm, r), tasks);
  };
  uint4* mine = hold + threadIdx.x;
  uint4* mine_g = mine + (size_t)tm.held * pitch * kX;
  for (int r = 0; r < tm.held; ++r) {
    const Task k = task(r);
    hold_task<T, VEC, EVEN>(s, k, x, mine + r * pitch * kX);
    hold_task<TG, VEC, EVEN>(s, k, gy, mine_g + r * pitch * kG);
  }
  const float mu = pl.here ? mean[pl.unit] : 0.f, rs = pl.here ? rstd[pl.unit] : 0.f;
  float val[2] = {0.f, 0.f};
  for (int r = tm.rounds - 1; r >= 0; --r) {
    const Task k = task(r);
    const bool held = r < tm.held;
    const uint4* slot = mine + r * pitch * kX;
    const uint4* slot_g = mine_g + r * pitch * kG;
    if (r == tm.held - 1) copy_wait();
    const float g = gamma ? gamma[k.ch] : 1.f, b = beta ? beta[k.ch] : 0.f;
    float2 sa = both(0.f), sb = both(0.f);
#pragma unroll 2
    for (int v = k.v0; v < k.v1; v += s.t.lpr) {
      Pairs<VEC> f, d;  // (0 outside the row: dz is 0 there)
      fetch<T, VEC, EVEN>(k, v, x, held, slot, f);
      fetch<TG, VEC, EVEN>(k, v, gy, held, slot_g, d);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float2 xh = mul2(add2(f.p[e], both(-mu)), both(rs));
        const float2 z = fma2(xh, both(g), both(b));
        const float2 dz = make_float2(act_bwd<ACT>(z.x, d.p[e].x, s.floor),
                                      act_bwd<ACT>(z.y, d.p[e].y, s.floor));
        sa = add2(sa, dz);
        sb = fma2(dz, xh, sb);
      }
      slot += kX * blockDim.x;
      slot_g += kG * blockDim.x;
    }
    const float ra = row_sum(sa.x + sa.y, s.t.lpr), rb = row_sum(sb.x + sb.y, s.t.lpr);
    if (k.live && (threadIdx.x & (s.t.lpr - 1)) == 0) {
      part[(long long)k.part * s.n * s.c + k.row] = make_float2(ra, rb);
      val[0] = fmaf(g, ra, val[0]);
      val[1] = fmaf(g, rb, val[1]);
    }
  }
  val[0] = warp_sum(val[0]);
  val[1] = warp_sum(val[1]);
  const float* se = share<2>(tm, pl, sm, val);
  float ga = 0.f, gb = 0.f;
  for (int i = threadIdx.x & 31; i < pl.team; i += 32) {
    ga += se[i];
    gb += se[256 + i];
  }
  const float total = (float)s.hw * (float)s.cpg;
  const float s1 = rs * (warp_sum(ga) / total), s2 = rs * (warp_sum(gb) / total);
  if (!pl.here) return;
  for (int r = 0; r < tm.rounds; ++r) {
    const Task k = task(r);
    const bool held = r < tm.held;
    const uint4* slot = mine + r * pitch * kX;
    const uint4* slot_g = mine_g + r * pitch * kG;
    const float g = gamma ? gamma[k.ch] : 1.f, b = beta ? beta[k.ch] : 0.f;
    const float gr = g * rs;
#pragma unroll 2
    for (int v = k.v0; v < k.v1; v += s.t.lpr) {
      Pairs<VEC> f, d;
      fetch<T, VEC, EVEN>(k, v, x, held, slot, f);
      fetch<TG, VEC, EVEN>(k, v, gy, held, slot_g, d);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float2 xh = mul2(add2(f.p[e], both(-mu)), both(rs));
        const float2 z = fma2(xh, both(g), both(b));
        const float2 dz = make_float2(act_bwd<ACT>(z.x, d.p[e].x, s.floor),
                                      act_bwd<ACT>(z.y, d.p[e].y, s.floor));
        f.p[e] = fma2(xh, both(-s2), fma2(dz, both(gr), both(-s1)));
      }
      put<T, VEC, EVEN>(k, v, gx, f);
      slot += kX * blockDim.x;
      slot_g += kG * blockDim.x;
    }
  }
}

}  // namespace

cudaError_t launch_team_nchw(const NormPlan& p, const NormArgs& a, bool backward,
                             cudaStream_t st) {
  if (!backward)
    return by_dtype(a.dt, [&](auto t) {
      using T = decltype(t);
      return by_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        auto go = [&](auto kern) {
          return launch_team(kern, p, p.row.cluster, st, p.s, p.row, static_cast<const T*>(a.x),
                             a.gamma, a.beta, static_cast<T*>(a.y), a.mean, a.rstd);
        };
        if (p.row.span) return go(fwd_flat<T, ACT>);
        return a.hw % VecOf<T>::n ? go(fwd_nchw<T, false, ACT>) : go(fwd_nchw<T, true, ACT>);
      });
    });
  return by_dtypes(a, [&](auto t, auto g) {
    using T = decltype(t);
    using TG = decltype(g);
    return by_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      auto go = [&](auto kern) {
        return launch_team(kern, p, p.row.cluster, st, p.s, p.row, static_cast<const T*>(a.x),
                           static_cast<const TG*>(a.gy), a.gamma, a.beta,
                           static_cast<const float*>(a.mean), static_cast<const float*>(a.rstd),
                           static_cast<T*>(a.gx), reinterpret_cast<float2*>(a.ws));
      };
      return a.hw % VecOf<T>::n ? go(bwd_nchw<T, TG, false, ACT>) : go(bwd_nchw<T, TG, true, ACT>);
    });
  });
}

}  // namespace dc
