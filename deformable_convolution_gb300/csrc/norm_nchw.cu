// Group norm with an activation on [n][c][h][w] tensors.
//
// y = act(xh gamma + beta), xh = (x - mean) rstd over a group of an image; with
// dz = grad_y act'(xh gamma + beta) the gradient is
// rstd (gamma dz - avg(gamma dz) - xh avg(gamma dz xh)).  Statistics are
// triples (count, mean, M2), merged exactly.
//
// A group of an image is a unit: cpg rows of h * w consecutive elements, held
// in the shared memory of a cluster's blocks from the statistics to the
// results, so that x (and grad_y) come from memory once.  A lane copies the
// 16-byte vectors that it works on itself, asynchronously and all at once: no
// registers wait for the loads, and no barrier stands between a copy and its
// use.  The loops over the vectors stay rolled: a block runs its code once,
// and a body unrolled over the vectors costs more in instruction fetches than
// it saves.  A unit that no cluster holds goes to two launches (below).
//
// Measured on 8 x 256 x 56 x 56 bf16 with ReLU (launches alone, tensors in L2):
// forward 6.8 us, backward with a float32 gradient 15.4 us, where the tensors'
// bytes take 3.8 and 7.6 us from memory.  What bounds them is the chain of a
// block (load, reduce, cluster barrier, store) in two waves: the units' 25 and
// 150 KB leave an SM two blocks.  Three launches with x read twice took 34 us
// for that backward.
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
    const int lane = threadIdx.x & 31, per = 32 / s.lpr;
    const int blk = tasks < 1 << 20 ? quick_div(t, s.inv_parts) : t / s.parts;
    part = t - blk * s.parts;
    const int local = blk * per + (s.lpr == 32 ? 0 : lane / s.lpr);
    live = t < tasks && local < s.cpg;
    row = (long long)unit * s.cpg + (live ? local : 0);
    ch = ch0 + (live ? local : 0);
    const long long first = row * s.hw;
    mis = EVEN ? 0 : (int)first & (VEC - 1);
    off = first - mis;
    v0 = part * s.seg + (lane & (s.lpr - 1));
    const int end = part * s.seg + s.seg, vr = row_vectors(s.hw, mis, VEC);
    v1 = !live ? v0 : end < vr ? end : vr;
    last = vr - 1;
    tail = s.hw + mis - last * VEC;
  }
  // the elements [lo, hi) of vector v lie in the row
  __device__ __forceinline__ int lo(int v) const { return EVEN || v ? 0 : mis; }
  __device__ __forceinline__ int hi(int v) const { return EVEN || v != last ? VEC : tail; }
};

// 16-byte pieces of a vector of VEC elements.
template <typename T, int VEC>
constexpr int kPieces = VEC * sizeof(T) / 16;

// A held vector: its pieces lie `plane` apart.
template <typename T, int VEC>
__device__ __forceinline__ void take(const uint4* slot, int plane, Pairs<VEC>& f) {
  uint32_t u[4 * kPieces<T, VEC>];
#pragma unroll
  for (int i = 0; i < kPieces<T, VEC>; ++i) {
    const uint4 v = slot[i * plane];
    u[4 * i] = v.x, u[4 * i + 1] = v.y, u[4 * i + 2] = v.z, u[4 * i + 3] = v.w;
  }
  unpack<T, VEC>(u, f);
}

// Held vectors: a warp's segments one after the other, a round after the other,
// in planes of 16-byte pieces.  The lane's first slot of a round:
__device__ __forceinline__ int first_slot(const Shape& s) {
  const int lane = threadIdx.x & 31, per = 32 / s.lpr;
  return ((threadIdx.x >> 5) * per + (s.lpr == 32 ? 0 : lane / s.lpr)) * s.seg +
         (lane & (s.lpr - 1));
}
__device__ __forceinline__ int round_slots(const Shape& s) {
  return (blockDim.x >> 5) * (32 / s.lpr) * s.seg;
}

// Starts the copy of vector v of a task, at p.
template <typename T, int VEC, bool EVEN>
__device__ __forceinline__ void hold(const UnitTask<VEC, EVEN>& k, int v, const T* p, uint4* slot,
                                     int plane) {
  const int bytes = k.hi(v) * (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < kPieces<T, VEC>; ++i) {
    // (a piece past the row's end is skipped; its slot is not used)
    const int b = min(16, bytes - 16 * i);
    if (EVEN || b > 0)
      copy_async<16, (kPieces<T, VEC> > 1)>(
          slot + i * plane, reinterpret_cast<const char*>(p) + 16 * i, EVEN ? 16 : b);
  }
}

// Vector v of a task at p, held or from memory; what lies outside the row is 0.
template <typename T, int VEC, bool EVEN, bool HELD>
__device__ __forceinline__ void fetch(const UnitTask<VEC, EVEN>& k, int v, const T* p,
                                      const uint4* slot, int plane, Pairs<VEC>& f) {
  const int lo = k.lo(v), hi = k.hi(v);
  const bool full = EVEN || (lo == 0 && hi == VEC);
  if (HELD) {
    take<T, VEC>(slot, plane, f);
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
__device__ __forceinline__ void put(const UnitTask<VEC, EVEN>& k, int v, T* p,
                                    const Pairs<VEC>& f) {
  const int lo = k.lo(v), hi = k.hi(v);
  if (EVEN || (lo == 0 && hi == VEC))
    store_vec<T, VEC>(p, f);
  else
    store_part<T, VEC>(p, lo, hi, reinterpret_cast<const float*>(f.p));
}

// This thread's place: block `rank` of the cluster, warp w of the unit's.
struct Place {
  int rank, u, w, team, ch0;  // ch0: the unit's first channel
  unsigned unit;
  bool here;
  __device__ __forceinline__ Place() {}
  __device__ __forceinline__ Place(const Shape& s, const RowTeam& tm) {
    const int warp = threadIdx.x >> 5;
    rank = cluster_rank();
    u = tm.units == 1 ? 0 : warp / tm.warps;
    w = warp - u * tm.warps;
    unit = cluster_id() * tm.units + u;  // (n * c is below 2^31)
    here = unit < (unsigned)s.n * s.groups;
    if (!here) unit = 0;
    ch0 = (int)(unit % (unsigned)s.groups) * s.cpg;
    team = tm.blocks * tm.warps;
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
  if (tm.blocks > 1) {
    cluster_wait();  // every block of the cluster runs
    if (lane < tm.blocks)
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
  val[1] = quotient(warp_sum(n * mean), fmaxf(val[0], 1.f), rcp_approx(fmaxf(val[0], 1.f)));
  val[2] = warp_sum(n > 0.f ? fmaf(n * (mean - val[1]), mean - val[1], m2) : 0.f);
  const float* sn = share<3>(tm, pl, sm, val);
  const int lane = threadIdx.x & 31;
  float sum = 0.f, q = 0.f;
  for (int i = lane; i < pl.team; i += 32) sum = fmaf(sn[i], sn[256 + i], sum);
  const float mu = unit_mean(s, warp_sum(sum));
  for (int i = lane; i < pl.team; i += 32) {
    const float d = sn[256 + i] - mu;
    if (sn[i] > 0.f) q += fmaf(sn[i] * d, d, sn[512 + i]);
  }
  return make_float2(mu, rsqrtf(warp_sum(q) * s.inv_total + s.eps));
}

constexpr int kBatch = 4;

// A lane's (n, mean, m2) merged with those of B vectors, cnt elements; get(b, f)
// fetches vector b, fix(b, f, m) sets to m what of it does not count.
template <int VEC, int B, typename GET, typename FIX>
__device__ __forceinline__ void add_batch(int most, int cnt, float& n, float& mean, float& m2,
                                          GET&& get, FIX&& fix) {
  Pairs<VEC> f[B];
  float2 sum = both(0.f), q = both(0.f);
#pragma unroll
  for (int b = 0; b < B; ++b) {
    if (b >= most) continue;
    get(b, f[b]);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) sum = add2(sum, f[b].p[e]);
  }
  const float mb = quotient(sum.x + sum.y, (float)cnt, rcp_approx((float)cnt));
#pragma unroll
  for (int b = 0; b < B; ++b) {
    if (b >= most) continue;
    fix(b, f[b], mb);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float2 d = add2(f[b].p[e], both(-mb));
      q = fma2(d, d, q);
    }
  }
  merge(n, mean, m2, (float)cnt, mb, q.x + q.y);
}

// The statistics of one task (held: `open` groups of copies are under way).
template <typename T, int VEC, bool EVEN, bool HELD>
__device__ __forceinline__ void task_stats(const Shape& s, const UnitTask<VEC, EVEN>& k, const T* x,
                                           const uint4* slot, int& open, float& n, float& mean,
                                           float& m2) {
  const T* p = x + k.off + (long long)k.v0 * VEC;
  const int lpr = s.lpr;
  for (int v0 = k.v0; v0 < k.v1; v0 += kBatch * lpr) {
    const int most = (k.v1 - v0 + lpr - 1) / lpr;
    if (HELD) copy_wait(--open);
    int cnt = 0;
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (b < most) cnt += k.hi(v0 + b * lpr) - k.lo(v0 + b * lpr);
    add_batch<VEC, kBatch>(
        most, cnt, n, mean, m2,
        [&](int b, Pairs<VEC>& f) {
          fetch<T, VEC, EVEN, HELD>(k, v0 + b * lpr, p + b * lpr * VEC, slot + b * lpr, 0, f);
        },
        [&](int b, Pairs<VEC>& f, float m) {
          if (EVEN) return;
          const int lo = k.lo(v0 + b * lpr), hi = k.hi(v0 + b * lpr);
          if (hi - lo < VEC) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
              if (e < lo || e >= hi) f[e] = m;
          }
        });
    slot += kBatch * lpr;
    p += kBatch * lpr * VEC;
  }
}

template <typename T, int VEC, bool EVEN, bool HELD, int ACT>
__device__ __forceinline__ void task_apply(const Shape& s, const UnitTask<VEC, EVEN>& k, const T* x,
                                           T* y, const uint4* slot, float mu, float a, float b) {
  constexpr int B = HELD ? 1 : 4;  // (loads ahead of the stores, which may be in place)
  const T* p = x + k.off + (long long)k.v0 * VEC;
  T* to = y + k.off + (long long)k.v0 * VEC;
  const int lpr = s.lpr;
#pragma unroll(HELD ? 2 : 1)
  for (int v0 = k.v0; v0 < k.v1; v0 += B * lpr) {
    Pairs<VEC> f[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (v0 + i * lpr < k.v1)
        fetch<T, VEC, EVEN, HELD>(k, v0 + i * lpr, p + i * lpr * VEC, slot + i * lpr, 0, f[i]);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (v0 + i * lpr >= k.v1) break;
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e)
        f[i].p[e] = act_fwd2<ACT>(fma2(add2(f[i].p[e], both(-mu)), both(a), both(b)), s.floor);
      put<T, VEC, EVEN>(k, v0 + i * lpr, to + i * lpr * VEC, f[i]);
    }
    slot += B * lpr;
    p += B * lpr * VEC;
    to += B * lpr * VEC;
  }
}

// Rows that are no whole vectors.
template <typename T, int ACT>
__global__ void __launch_bounds__(kTeam, 2)
    fwd_nchw(Shape s, RowTeam tm, const T* x, const float* gamma, const float* beta, T* y,
             float* mean_out, float* rstd_out) {
  constexpr int VEC = VecOf<T>::n;
  constexpr bool EVEN = false;
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ float sm[3][256];
  if (tm.blocks > 1) cluster_arrive();
  pdl_wait();
  pdl_release();
  const Place pl(s, tm);
  const int tasks = pl.here ? tm.tasks : 0, pitch = round_slots(s);
  using Task = UnitTask<VEC, EVEN>;
  const Task first(s, pl.unit, pl.ch0, pl.task(tm, 0), tasks);
  auto task = [&](int r) {
    return r == 0 ? first : Task(s, pl.unit, pl.ch0, pl.task(tm, r), tasks);
  };
  uint4* mine = slots + first_slot(s);
  int open = 0;  // groups of copies under way: of kBatch vectors, or the task's last
  for (int r = 0; r < tm.rounds; ++r) {
    const Task k = task(r);
    const T* p = x + k.off + (long long)k.v0 * VEC;
    uint4* slot = mine + r * pitch;
    for (int v0 = k.v0; v0 < k.v1; v0 += kBatch * s.lpr, ++open) {
      for (int v = v0; v < k.v1 && v < v0 + kBatch * s.lpr; v += s.lpr) {
        hold<T, VEC, EVEN>(k, v, p, slot, 0);
        slot += s.lpr;
        p += s.lpr * VEC;
      }
      copy_group();
    }
  }
  float n = 0.f, mean = 0.f, m2 = 0.f;
  for (int r = 0; r < tm.rounds; ++r)
    task_stats<T, VEC, EVEN, true>(s, task(r), x, mine + r * pitch, open, n, mean, m2);
  const float2 st = unit_stats(s, tm, pl, sm, n, mean, m2);
  if (!pl.here) return;
  if (pl.rank == 0 && pl.w == 0 && (threadIdx.x & 31) == 0) {
    if (mean_out) mean_out[pl.unit] = st.x;
    if (rstd_out) rstd_out[pl.unit] = st.y;
  }
  for (int r = 0; r < tm.rounds; ++r) {
    const Task k = task(r);
    const float a = st.y * (gamma ? gamma[k.ch] : 1.f), b = beta ? beta[k.ch] : 0.f;
    task_apply<T, VEC, EVEN, true, ACT>(s, k, x, y, mine + r * pitch, st.x, a, b);
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
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ float sm[3][256];
  if (tm.blocks > 1) cluster_arrive();
  pdl_wait();
  pdl_release();
  const Place pl(s, tm);
  const int threads = 32 * tm.warps, tid = threadIdx.x - pl.u * threads;
  const int vr = s.hw / VEC, step = threads * VEC;
  const int begin = pl.rank * tm.span + tid;
  int end = s.cpg * vr;  // (a unit of 2^30 vectors or more does not come here)
  if (end > (pl.rank + 1) * tm.span) end = (pl.rank + 1) * tm.span;
  if (!pl.here) end = 0;
  const int held = begin < end ? (end - begin + threads - 1) / threads : 0;  // vectors
  const long long off = (long long)pl.unit * s.cpg * s.hw + (long long)begin * VEC;
  uint4* mine = slots + threadIdx.x;
  {
    const T* p = x + off;
    uint4* slot = mine;
    for (int i = 0; i < held; ++i, p += step, slot += blockDim.x) {
      copy_async<16>(slot, p);
      if (i % kBatch == kBatch - 1 || i == held - 1) copy_group();
    }
  }
  // vector i of this thread lies in channel c, `at` vectors from its start
  int c = begin / vr, at = begin - c * vr;
  float n = 0.f, mean = 0.f, m2 = 0.f;
  auto keep = [](int, Pairs<VEC>&, float) {};
  {
    const uint4* slot = mine;
    auto get = [&](int b, Pairs<VEC>& f) { take<T, VEC>(slot + b * blockDim.x, 0, f); };
    int i = 0, open = (held + kBatch - 1) / kBatch;
    for (; i + kBatch <= held; i += kBatch, slot += kBatch * blockDim.x) {
      copy_wait(--open);
      add_batch<VEC, kBatch>(kBatch, kBatch * VEC, n, mean, m2, get, keep);
    }
    if (i < held) {
      copy_wait(0);
      add_batch<VEC, kBatch>(held - i, (held - i) * VEC, n, mean, m2, get, keep);
    }
  }
  const float2 st = unit_stats(s, tm, pl, sm, n, mean, m2);
  if (!pl.here) return;
  if (pl.rank == 0 && tid == 0) {
    if (mean_out) mean_out[pl.unit] = st.x;
    if (rstd_out) rstd_out[pl.unit] = st.y;
  }
  const float* gm = gamma ? gamma + pl.ch0 : nullptr;
  const float* bt = beta ? beta + pl.ch0 : nullptr;
  T* to = y + off;
  auto apply = [&](Pairs<VEC>& f) {
    const float a = st.y * (gm ? gm[c] : 1.f), b = bt ? bt[c] : 0.f;
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e)
      f.p[e] = act_fwd2<ACT>(fma2(add2(f.p[e], both(-st.x)), both(a), both(b)), s.floor);
    store_vec<T, VEC>(to, f);
    to += step;
    c += tm.step_c;
    at += tm.step_v;
    if (at >= vr) at -= vr, ++c;
  };
#pragma unroll 4
  for (int i = 0; i < held; ++i) {
    Pairs<VEC> f;
    take<T, VEC>(mine + i * blockDim.x, 0, f);
    apply(f);
  }
}

// A task's sums of dz and dz * xh (held: `open` groups of copies are under
// way).  KEEP: dz takes grad_y's place in the slot
// (in float32), so that the results need the activation's slope no more.
template <typename T, typename TG, int VEC, bool EVEN, bool HELD, bool KEEP, int ACT>
__device__ __forceinline__ void task_sums(const Shape& s, const UnitTask<VEC, EVEN>& k, const T* x,
                                          const TG* gy, const uint4* slot, uint4* slot_g,
                                          int plane, int& open, float mu, float rs, float g,
                                          float b, float2& sa, float2& sb) {
  const long long off = k.off + (long long)k.v0 * VEC;
  const T* p = x + off;
  const TG* pg = gy + off;
  auto vector = [&](int v) {
    Pairs<VEC> f, d;  // (0 outside the row: dz is 0 there)
    fetch<T, VEC, EVEN, HELD>(k, v, p, slot, plane, f);
    fetch<TG, VEC, EVEN, HELD>(k, v, pg, slot_g, plane, d);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const float2 xh = mul2(add2(f.p[e], both(-mu)), both(rs));
      d.p[e] = act_bwd2<ACT>(fma2(xh, both(g), both(b)), d.p[e], s.floor);
      sa = add2(sa, d.p[e]);
      sb = fma2(d.p[e], xh, sb);
    }
    if (HELD && KEEP) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i)
        *reinterpret_cast<float4*>(slot_g + i * plane) = make_float4(
            d.p[2 * i].x, d.p[2 * i].y, d.p[2 * i + 1].x, d.p[2 * i + 1].y);
    }
    slot += s.lpr;
    slot_g += s.lpr;
    p += s.lpr * VEC;
    pg += s.lpr * VEC;
  };
  for (int v = k.v0; v < k.v1; v += 2 * s.lpr) {
    if (HELD) copy_wait(--open);
    vector(v);
    if (v + s.lpr < k.v1) vector(v + s.lpr);
  }
}

// grad_x = dz * gr - s1 - xh * s2 (gr = gamma * rstd; s1, s2 times rstd)
template <typename T, typename TG, int VEC, bool EVEN, bool HELD, bool KEEP, int ACT>
__device__ __forceinline__ void task_grads(const Shape& s, const UnitTask<VEC, EVEN>& k, const T* x,
                                           const TG* gy, T* gx, const uint4* slot,
                                           const uint4* slot_g, int plane, float mu, float rs,
                                           float g, float b, float s1, float s2) {
  const long long off = k.off + (long long)k.v0 * VEC;
  const T* p = x + off;
  const TG* pg = gy + off;
  T* to = gx + off;
  const float gr = g * rs;
  constexpr int B = HELD ? 1 : 2;  // (loads ahead of the stores, which may be in place)
  const int lpr = s.lpr;
#pragma unroll(HELD ? 2 : 1)
  for (int v0 = k.v0; v0 < k.v1; v0 += B * lpr) {
    Pairs<VEC> f[B], d[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int v = v0 + i * lpr;
      if (v >= k.v1) break;
      fetch<T, VEC, EVEN, HELD>(k, v, p + i * lpr * VEC, slot + i * lpr, plane, f[i]);
      if (HELD && KEEP)
        take<float, VEC>(slot_g + i * lpr, plane, d[i]);
      else
        fetch<TG, VEC, EVEN, HELD>(k, v, pg + i * lpr * VEC, slot_g + i * lpr, plane, d[i]);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int v = v0 + i * lpr;
      if (v >= k.v1) break;
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) {
        const float2 xh = mul2(add2(f[i].p[e], both(-mu)), both(rs));
        if (!(HELD && KEEP))
          d[i].p[e] = act_bwd2<ACT>(fma2(xh, both(g), both(b)), d[i].p[e], s.floor);
        f[i].p[e] = fma2(xh, both(-s2), fma2(d[i].p[e], both(gr), both(-s1)));
      }
      put<T, VEC, EVEN>(k, v, to + i * lpr * VEC, f[i]);
    }
    slot += B * lpr;
    slot_g += B * lpr;
    p += B * lpr * VEC;
    pg += B * lpr * VEC;
    to += B * lpr * VEC;
  }
}

// part[segment][image * c + channel]: the sums of dz and dz * xh of a row's
// segment.
template <typename T, typename TG, bool EVEN, int ACT>
__global__ void __launch_bounds__(kTeam, 2)
    bwd_nchw(Shape s, RowTeam tm, const T* x, const TG* gy, const float* gamma, const float* beta,
             const float* mean, const float* rstd, T* gx, float2* part) {
  constexpr int VEC = VecOf<T>::n;
  constexpr bool KEEP = keep_dz(sizeof(TG) == 4, ACT);
  constexpr int kG = KEEP ? VEC / 4 : kPieces<TG, VEC>;  // pieces of a slot of grad_y
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ float sm[2][256];
  if (tm.blocks > 1) cluster_arrive();
  pdl_wait();
  pdl_release();
  const Place pl(s, tm);
  const int tasks = pl.here ? tm.tasks : 0, pitch = round_slots(s);
  using Task = UnitTask<VEC, EVEN>;
  const Task first(s, pl.unit, pl.ch0, pl.task(tm, 0), tasks);
  auto task = [&](int r) {
    return r == 0 ? first : Task(s, pl.unit, pl.ch0, pl.task(tm, r), tasks);
  };
  uint4* mine = slots + first_slot(s);
  uint4* mine_g = mine + (size_t)tm.rounds * pitch;
  int open = 0;  // groups of copies under way: of two vectors, or the task's last
  for (int r = 0; r < tm.rounds; ++r) {
    const Task k = task(r);
    const long long off = k.off + (long long)k.v0 * VEC;
    const T* p = x + off;
    const TG* pg = gy + off;
    uint4* slot = mine + r * pitch;
    uint4* slot_g = mine_g + r * pitch * kG;
    for (int v0 = k.v0; v0 < k.v1; v0 += 2 * s.lpr, ++open) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (v0 + i * s.lpr >= k.v1) break;
        hold<T, VEC, EVEN>(k, v0 + i * s.lpr, p, slot, pitch);
        hold<TG, VEC, EVEN>(k, v0 + i * s.lpr, pg, slot_g, pitch);
        slot += s.lpr;
        slot_g += s.lpr;
        p += s.lpr * VEC;
        pg += s.lpr * VEC;
      }
      copy_group();
    }
  }
  const float mu = pl.here ? mean[pl.unit] : 0.f, rs = pl.here ? rstd[pl.unit] : 0.f;
  float val[2] = {0.f, 0.f};
  for (int r = 0; r < tm.rounds; ++r) {
    const Task k = task(r);
    const float g = gamma ? gamma[k.ch] : 1.f, b = beta ? beta[k.ch] : 0.f;
    float2 sa = both(0.f), sb = both(0.f);
    task_sums<T, TG, VEC, EVEN, true, KEEP, ACT>(s, k, x, gy, mine + r * pitch,
                                                 mine_g + r * pitch * kG, pitch, open, mu, rs, g, b,
                                                 sa, sb);
    const float ra = row_sum(sa.x + sa.y, s.lpr), rb = row_sum(sb.x + sb.y, s.lpr);
    if (k.live && (threadIdx.x & (s.lpr - 1)) == 0) {
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
  const float s1 = rs * (warp_sum(ga) * s.inv_total), s2 = rs * (warp_sum(gb) * s.inv_total);
  if (!pl.here) return;
  for (int r = 0; r < tm.rounds; ++r) {
    const Task k = task(r);
    const float g = gamma ? gamma[k.ch] : 1.f, b = beta ? beta[k.ch] : 0.f;
    task_grads<T, TG, VEC, EVEN, true, KEEP, ACT>(s, k, x, gy, gx, mine + r * pitch,
                                                  mine_g + r * pitch * kG, pitch, mu, rs, g, b, s1,
                                                  s2);
  }
}

// ---------------------------------------------------------------- two launches
//
// For units that no cluster holds, and where the plan finds it faster: sums of
// blocks' shares into the workspace, then the results, the second read from L2.
// The backward's lanes stream their vectors through rings of slots of their
// own: 69 us on 2 x 200 x 336 x 256 bf16 with SiLU, where loads into registers
// took 84 and the bytes take 30.4 once.  Bound by the second read and the
// launches' latency.

// This thread's place where a unit's blocks are no cluster.
__device__ __forceinline__ Place loose_place(const Shape& s, const RowTeam& tm, unsigned unit0) {
  Place pl;
  const unsigned id = blockIdx.x / (unsigned)tm.blocks;
  pl.rank = (int)(blockIdx.x - id * tm.blocks);
  pl.u = 0;
  pl.w = threadIdx.x >> 5;
  pl.unit = unit0 + id;
  pl.here = true;
  pl.ch0 = (int)(pl.unit % (unsigned)s.groups) * s.cpg;
  pl.team = tm.blocks * tm.warps;
  return pl;
}

// entry[unit * blocks + rank] = (count, mean, M2) of a block's share.
template <typename T, bool EVEN>
__global__ void __launch_bounds__(kTwo)
    stats_nchw(Shape s, RowTeam tm, unsigned unit0, const T* x, float4* entry) {
  constexpr int VEC = VecOf<T>::n;
  __shared__ float sm[3][kTwo / 32];
  pdl_wait();
  pdl_release();
  const Place pl = loose_place(s, tm, unit0);
  float n = 0.f, mean = 0.f, m2 = 0.f;
  if constexpr (EVEN) {
    const BlockRun run(s.cpg, s.hw / VEC, tm.span, pl.rank);
    const int tid = threadIdx.x;
    const T* p = x + (long long)pl.unit * s.cpg * s.hw + (run.begin + tid) * VEC;
    const int count = tid < run.count ? (run.count - tid + kTwo - 1) / kTwo : 0;
    auto get = [&](int b, Pairs<VEC>& f) { load_vec<T, VEC>(p + b * kTwo * VEC, f); };
    auto keep = [](int, Pairs<VEC>&, float) {};
    int i = 0;
    for (; i + kBatch <= count; i += kBatch, p += kBatch * kTwo * VEC)
      add_batch<VEC, kBatch>(kBatch, kBatch * VEC, n, mean, m2, get, keep);
    if (i < count) add_batch<VEC, kBatch>(count - i, (count - i) * VEC, n, mean, m2, get, keep);
  } else {
    int none = 0;
    for (int r = 0; r < tm.rounds; ++r)
      task_stats<T, VEC, EVEN, false>(
          s, UnitTask<VEC, EVEN>(s, pl.unit, pl.ch0, pl.task(tm, r), tm.tasks), x, nullptr, none,
          n, mean, m2);
  }
  const float wn = warp_sum(n), wm = warp_sum(n * mean) / fmaxf(wn, 1.f);
  const float wq = warp_sum(n > 0.f ? fmaf(n * (mean - wm), mean - wm, m2) : 0.f);
  if ((threadIdx.x & 31) == 0) sm[0][pl.w] = wn, sm[1][pl.w] = wm, sm[2][pl.w] = wq;
  __syncthreads();
  if (threadIdx.x == 0) {
    n = mean = m2 = 0.f;
    for (int w = 0; w < kTwo / 32; ++w) merge(n, mean, m2, sm[0][w], sm[1][w], sm[2][w]);
    entry[(size_t)pl.unit * tm.blocks + pl.rank] = make_float4(n, mean, m2, 0.f);
  }
}

template <typename T, bool EVEN, int ACT>
__global__ void __launch_bounds__(kTwo)
    apply_nchw(Shape s, RowTeam tm, unsigned unit0, const T* x, const float* gamma,
               const float* beta, const float4* entry, T* y, float* mean_out, float* rstd_out) {
  constexpr int VEC = VecOf<T>::n;
  pdl_wait();
  pdl_release();
  const Place pl = loose_place(s, tm, unit0);
  const int lane = threadIdx.x & 31;
  const float4* mine = entry + (size_t)pl.unit * tm.blocks;
  float n = 0.f, mean = 0.f, m2 = 0.f;
  for (int i = lane; i < tm.blocks; i += 32) {
    const float4 v = mine[i];
    merge(n, mean, m2, v.x, v.y, v.z);
  }
  const float mu = unit_mean(s, warp_sum(n * mean));
  const float var = warp_sum(n > 0.f ? fmaf(n * (mean - mu), mean - mu, m2) : 0.f) * s.inv_total;
  const float rs = rsqrtf(var + s.eps);
  if (pl.rank == 0 && threadIdx.x == 0) {
    if (mean_out) mean_out[pl.unit] = mu;
    if (rstd_out) rstd_out[pl.unit] = rs;
  }
  if constexpr (EVEN) {
    const int vr = s.hw / VEC;
    const BlockRun run(s.cpg, vr, tm.span, pl.rank);
    const long long begin = run.begin + threadIdx.x;
    const long long off = (long long)pl.unit * s.cpg * s.hw + begin * VEC;
    const T* p = x + off;
    T* to = y + off;
    int c = (int)(begin / vr), at = (int)(begin - (long long)c * vr);
    for (int v0 = threadIdx.x; v0 < run.count; v0 += kBatch * kTwo) {
      Pairs<VEC> f[kBatch];  // (loads ahead of the stores, which may be in place)
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (v0 + i * kTwo < run.count) load_vec<T, VEC>(p + i * kTwo * VEC, f[i]);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (v0 + i * kTwo >= run.count) break;
        const float a = rs * (gamma ? gamma[pl.ch0 + c] : 1.f), b = beta ? beta[pl.ch0 + c] : 0.f;
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
          f[i].p[e] = act_fwd2<ACT>(fma2(add2(f[i].p[e], both(-mu)), both(a), both(b)), s.floor);
        store_vec<T, VEC>(to + i * kTwo * VEC, f[i]);
        c += tm.step_c;
        at += tm.step_v;
        if (at >= vr) at -= vr, ++c;
      }
      p += kBatch * kTwo * VEC;
      to += kBatch * kTwo * VEC;
    }
  } else {
    for (int r = 0; r < tm.rounds; ++r) {
      const UnitTask<VEC, EVEN> k(s, pl.unit, pl.ch0, pl.task(tm, r), tm.tasks);
      task_apply<T, VEC, EVEN, false, ACT>(s, k, x, y, nullptr, mu,
                                           rs * (gamma ? gamma[k.ch] : 1.f),
                                           beta ? beta[k.ch] : 0.f);
    }
  }
}

// Whether a backward's vectors go through the ring: not those of float32
// gradients of bf16 tensors, two pieces each, whose slots leave three blocks to
// an SM (2 x 200 x 336 x 256, ReLU: 87 us with loads into registers, 109 with
// the ring).
template <typename T, typename TG>
constexpr bool kStreams = sizeof(T) == sizeof(TG);

// A backward task's vectors through the ring, work(v, f, d) on each.  Dynamic
// shared memory: the slots of x, then of grad_y.
template <typename T, typename TG, int VEC, bool EVEN, typename WORK>
__device__ __forceinline__ void stream_task(const Shape& s, const UnitTask<VEC, EVEN>& k,
                                            const T* x, const TG* gy, WORK&& work) {
  extern __shared__ __align__(128) uint4 slots[];
  constexpr int pitch = kPieces<T, VEC> * kTwo, pitch_g = kPieces<TG, VEC> * kTwo;
  uint4* mine = slots + threadIdx.x;
  uint4* mine_g = mine + kRing * 2 * pitch;
  const long long off = k.off + (long long)k.v0 * VEC;
  const T* p = x + off;
  const TG* pg = gy + off;
  through_ring<2>(
      (k.v1 - k.v0 + s.lpr - 1) / s.lpr,
      [&](int i, int slot) {
        const int v = k.v0 + i * s.lpr;
        hold<T, VEC, EVEN>(k, v, p, mine + slot * pitch, kTwo);
        hold<TG, VEC, EVEN>(k, v, pg, mine_g + slot * pitch_g, kTwo);
        p += s.lpr * VEC;
        pg += s.lpr * VEC;
      },
      [&](int i, int most, int slot) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (j >= most) break;
          const int v = k.v0 + (i + j) * s.lpr;
          Pairs<VEC> f, d;  // (0 outside the row: dz is 0 there)
          fetch<T, VEC, EVEN, true>(k, v, nullptr, mine + (slot + j) * pitch, kTwo, f);
          fetch<TG, VEC, EVEN, true>(k, v, nullptr, mine_g + (slot + j) * pitch_g, kTwo, d);
          work(v, f, d);
        }
      });
}

// part as above; entry[unit * blocks + rank] = the block's sums of gamma dz and
// gamma dz xh.
template <typename T, typename TG, bool EVEN, int ACT>
__global__ void __launch_bounds__(kTwo)
    sums_nchw(Shape s, RowTeam tm, unsigned unit0, const T* x, const TG* gy, const float* gamma,
              const float* beta, const float* mean, const float* rstd, float2* part,
              float2* entry) {
  constexpr int VEC = VecOf<T>::n;
  __shared__ float2 sm[kTwo / 32];
  pdl_wait();
  pdl_release();
  const Place pl = loose_place(s, tm, unit0);
  const float mu = mean[pl.unit], rs = rstd[pl.unit];
  float ga = 0.f, gb = 0.f;
  for (int r = 0; r < tm.rounds; ++r) {
    const UnitTask<VEC, EVEN> k(s, pl.unit, pl.ch0, pl.task(tm, r), tm.tasks);
    const float g = gamma ? gamma[k.ch] : 1.f, b = beta ? beta[k.ch] : 0.f;
    float2 sa = both(0.f), sb = both(0.f);
    if constexpr (kStreams<T, TG>) {
      stream_task<T, TG, VEC, EVEN>(s, k, x, gy, [&](int, Pairs<VEC>& f, Pairs<VEC>& d) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const float2 xh = mul2(add2(f.p[e], both(-mu)), both(rs));
          const float2 dz = act_bwd2<ACT>(fma2(xh, both(g), both(b)), d.p[e], s.floor);
          sa = add2(sa, dz);
          sb = fma2(dz, xh, sb);
        }
      });
    } else {
      int none = 0;
      task_sums<T, TG, VEC, EVEN, false, false, ACT>(s, k, x, gy, nullptr, nullptr, 0, none, mu,
                                                     rs, g, b, sa, sb);
    }
    const float ra = row_sum(sa.x + sa.y, s.lpr), rb = row_sum(sb.x + sb.y, s.lpr);
    if (k.live && (threadIdx.x & (s.lpr - 1)) == 0) {
      part[(long long)k.part * s.n * s.c + k.row] = make_float2(ra, rb);
      ga = fmaf(g, ra, ga);
      gb = fmaf(g, rb, gb);
    }
  }
  ga = warp_sum(ga);
  gb = warp_sum(gb);
  if ((threadIdx.x & 31) == 0) sm[pl.w] = make_float2(ga, gb);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kTwo / 32; ++w) ga += sm[w].x, gb += sm[w].y;
    entry[(size_t)pl.unit * tm.blocks + pl.rank] = make_float2(ga, gb);
  }
}

template <typename T, typename TG, bool EVEN, int ACT>
__global__ void __launch_bounds__(kTwo)
    grads_nchw(Shape s, RowTeam tm, unsigned unit0, const T* x, const TG* gy, const float* gamma,
               const float* beta, const float* mean, const float* rstd, const float2* entry,
               T* gx) {
  constexpr int VEC = VecOf<T>::n;
  pdl_wait();
  pdl_release();
  const Place pl = loose_place(s, tm, unit0);
  const float mu = mean[pl.unit], rs = rstd[pl.unit];
  const float2* e = entry + (size_t)pl.unit * tm.blocks;
  float ga = 0.f, gb = 0.f;
  for (int i = threadIdx.x & 31; i < tm.blocks; i += 32) {
    const float2 v = e[i];
    ga += v.x;
    gb += v.y;
  }
  const float s1 = rs * (warp_sum(ga) * s.inv_total), s2 = rs * (warp_sum(gb) * s.inv_total);
  for (int r = 0; r < tm.rounds; ++r) {
    const UnitTask<VEC, EVEN> k(s, pl.unit, pl.ch0, pl.task(tm, r), tm.tasks);
    const float g = gamma ? gamma[k.ch] : 1.f, b = beta ? beta[k.ch] : 0.f;
    if constexpr (kStreams<T, TG>) {
      const float gr = g * rs;
      T* to = gx + k.off + (long long)k.v0 * VEC;
      stream_task<T, TG, VEC, EVEN>(s, k, x, gy, [&](int v, Pairs<VEC>& f, Pairs<VEC>& d) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          const float2 xh = mul2(add2(f.p[e], both(-mu)), both(rs));
          const float2 dz = act_bwd2<ACT>(fma2(xh, both(g), both(b)), d.p[e], s.floor);
          f.p[e] = fma2(xh, both(-s2), fma2(dz, both(gr), both(-s1)));
        }
        put<T, VEC, EVEN>(k, v, to, f);
        to += s.lpr * VEC;
      });
    } else {
      task_grads<T, TG, VEC, EVEN, false, false, ACT>(s, k, x, gy, gx, nullptr, nullptr, 0, mu, rs,
                                                      g, b, s1, s2);
    }
  }
}

}  // namespace

cudaError_t launch_nchw(const NormPlan& p, const NormArgs& a, bool backward,
                             cudaStream_t st) {
  if (!backward)
    return by_dtype(a.dt, [&](auto t) {
      using T = decltype(t);
      return by_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        auto go = [&](auto kern) {
          return launch_team(kern, p, p.row.blocks, st, p.s, p.row, static_cast<const T*>(a.x),
                             a.gamma, a.beta, static_cast<T*>(a.y), a.mean, a.rstd);
        };
        return a.hw % VecOf<T>::n ? go(fwd_nchw<T, ACT>) : go(fwd_flat<T, ACT>);
      });
    });
  return by_dtypes(a, [&](auto t, auto g) {
    using T = decltype(t);
    using TG = decltype(g);
    return by_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      auto go = [&](auto kern) {
        return launch_team(kern, p, p.row.blocks, st, p.s, p.row, static_cast<const T*>(a.x),
                           static_cast<const TG*>(a.gy), a.gamma, a.beta,
                           static_cast<const float*>(a.mean), static_cast<const float*>(a.rstd),
                           static_cast<T*>(a.gx), reinterpret_cast<float2*>(a.ws));
      };
      return a.hw % VecOf<T>::n ? go(bwd_nchw<T, TG, false, ACT>) : go(bwd_nchw<T, TG, true, ACT>);
    });
  });
}

cudaError_t launch_two_nchw(const NormPlan& p, const NormArgs& a, bool backward, bool second,
                            int img0, int count, cudaStream_t st) {
  const unsigned unit0 = (unsigned)img0 * a.groups;
  const unsigned grid = (unsigned)count * a.groups * p.row.blocks;
  char* entry = a.ws + norm_part_bytes(p, a, backward);
  if (!backward)
    return by_dtype(a.dt, [&](auto t) {
      using T = decltype(t);
      const T* x = static_cast<const T*>(a.x);
      float4* e = reinterpret_cast<float4*>(entry);
      auto by_even = [&](auto even) {
        constexpr bool EVEN = decltype(even)::value != 0;
        if (!second)
          return launch_plain(stats_nchw<T, EVEN>, grid, kTwo, st, p.s, p.row, unit0, x, e);
        return by_act(a.act, [&](auto act) {
          return launch_plain(apply_nchw<T, EVEN, decltype(act)::value>, grid, kTwo, st, p.s,
                              p.row, unit0, x, a.gamma, a.beta, static_cast<const float4*>(e),
                              static_cast<T*>(a.y), a.mean, a.rstd);
        });
      };
      return a.hw % VecOf<T>::n ? by_even(Int<0>{}) : by_even(Int<1>{});
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
      auto by_even = [&](auto even) {
        constexpr bool EVEN = decltype(even)::value != 0;
        if (!second)
          return launch_smem(sums_nchw<T, TG, EVEN, ACT>, grid, kTwo, p.smem, st, p.s, p.row, unit0, x,
                              gy, a.gamma, a.beta, mean, rstd, reinterpret_cast<float2*>(a.ws), e);
        return launch_smem(grads_nchw<T, TG, EVEN, ACT>, grid, kTwo, p.smem, st, p.s, p.row, unit0, x, gy,
                            a.gamma, a.beta, mean, rstd, static_cast<const float2*>(e),
                            static_cast<T*>(a.gx));
      };
      return a.hw % VecOf<T>::n ? by_even(Int<0>{}) : by_even(Int<1>{});
    });
  });
}

}  // namespace dc
