// Group norm with an activation, forward and backward, between deformable
// layers (no counterpart on the explainer page; the definitions are in the
// ABI header): how a call runs, and the parameters' gradients.
#include <math.h>

#include "dc_norm.cuh"

namespace dc {
namespace {

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

// ---------------------------------------------------------------- the plan

// A call is one launch of clusters that hold their units on the chip, or, for
// units over kMaxCluster * kBlockBytes (and where plan_rows or plan_cols says
// so), two launches that read their inputs twice.  us of clusters / two
// launches, inputs out of L2: forward 32 x 256 x 56 x 56 bf16 ReLU 23.5 / 27.4,
// 16 x 100 x 168 x 256 SiLU 69 / 74, backward 8 x 256 x 56 x 56 ReLU with a
// float32 gradient 19.6 / 23.3.
constexpr int kSms = 152;
// Most of a unit in a cluster's block: two blocks to an SM (with 50 KB, four to
// an SM, that backward took a tenth longer).
constexpr int kBlockBytes = 92 * 1024;
constexpr int kLeastBytes = 16 * 1024;  // not split further to make more blocks

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Blocks of a unit of `bytes`: enough that it fits, and that every SM gets two,
// as long as a block keeps work worth its launch.
int cluster_of(double bytes, long long units) {
  long long k = (long long)ceil(bytes / kBlockBytes), most = (long long)(bytes / kLeastBytes);
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

Shape make_shape(const NormArgs& a) {
  Shape s{};
  const int vec = a.dt == DC_BF16 ? 8 : 4;
  s.n = a.n;
  s.c = a.c;
  s.groups = a.groups;
  s.cpg = a.cpg;
  s.hw = a.hw;
  s.floor = a.act == DC_ACT_RELU ? 0.f : -INFINITY;
  s.eps = a.eps;
  // 16 bytes, or 8 where only that much is of one group (or divides c)
  s.v = a.c % vec == 0 && (vec == 4 || a.cpg % 8 != 4) ? vec : a.c % 4 == 0 ? 4 : 1;
  const int vr = row_vectors(a.hw, a.hw % vec ? vec - 1 : 0, vec);
  s.lpr = 1;
  while (s.lpr < 32 && s.lpr < vr) s.lpr *= 2;
  return s;
}

// Of a pass's inputs, left in L2 (129 MB) between two launches: 64 MB, which
// makes a turn of every image, took 61 us where 96 MB take 43 (forward on
// 2 x 200 x 336 x 256 bf16).
constexpr double kImagesBytes = 96e6;
// What a pass reads of an image.
double image_bytes(const NormArgs& a, bool backward) {
  const int elt = a.dt == DC_BF16 ? 2 : 4, gelt = a.gdt == DC_F32 ? 4 : 2;
  return (double)a.c * a.hw * (elt + (backward ? gelt : 0));
}

// A cluster that holds the unit; false where it does not fit one, or where two
// launches are faster.
bool plan_rows(const NormArgs& a, bool backward, int planes, NormPlan* p) {
  Shape& s = p->s;
  RowTeam& r = p->row;
  const int vec = a.dt == DC_BF16 ? 8 : 4;
  const long long groups = (long long)a.n * a.groups;
  const int vr = row_vectors(a.hw, a.hw % vec ? vec - 1 : 0, vec);
  const double bytes = (double)a.cpg * vr * 16 * planes;
  if (bytes > (double)kMaxCluster * kBlockBytes) return false;
  r.blocks = cluster_of(bytes, groups);
  r.units = 1;
  if (!backward && a.hw % vec == 0) {
    r.span = (int)ceil_div_ll((long long)a.cpg * vr, r.blocks);
    r.warps = threads_of(r.span) / 32;
    if (r.warps * 32 > r.span) r.warps = (int)ceil_div_ll(r.span, 32);
    if (r.blocks == 1)
      while (r.units * r.warps < 4 && groups / (2 * r.units) >= 4 * kSms) r.units *= 2;
    const int threads = 32 * r.warps;
    r.step_c = threads / vr;
    r.step_v = threads % vr;
    p->threads = threads * r.units;
    p->smem = (size_t)16 * p->threads * ceil_div_ll(r.span, threads);
  } else {
    const int per = 32 / s.lpr;
    const long long blks = ceil_div_ll(a.cpg, per), run = (long long)a.cpg * vr;
    // tasks for every warp the blocks want, of no less than four vectors a
    // lane; more blocks where the rounding up would not fit
    for (;; ++r.blocks) {
      if (r.blocks > kMaxCluster) return false;
      const int want = threads_of((double)run / r.blocks) / 32;
      long long parts = (r.blocks * want + blks / 2) / blks;
      if (parts > vr / (4 * s.lpr)) parts = vr / (4 * s.lpr);
      if (parts < 1) parts = 1;
      s.seg = (int)ceil_div_ll(vr, parts);
      s.parts = (int)ceil_div_ll(vr, s.seg);
      r.tasks = (int)(blks * s.parts);
      const int blocks = r.blocks < r.tasks ? r.blocks : r.tasks;
      r.rounds = (int)ceil_div_ll(r.tasks, blocks * 16);
      r.warps = (int)ceil_div_ll(r.tasks, blocks * r.rounds);
      const long long block = (long long)r.rounds * r.warps * per * s.seg * 16 * planes;
      if (block > kBlockBytes) continue;
      r.blocks = blocks;
      break;
    }
    if (r.blocks == 1)
      while (r.units * r.warps < 4 && groups / (2 * r.units) >= 4 * kSms) r.units *= 2;
    p->threads = 32 * r.warps * r.units;
    p->smem = (size_t)r.rounds * r.units * r.warps * per * s.seg * 16 * planes;
    p->parts = s.parts;
  }
  p->blocks = (unsigned)(ceil_div_ll(groups, r.units) * r.blocks);
  // As in plan_cols, but with less to gain: us of a bf16 SiLU backward on
  // h x w x 256, clusters / two launches: 8 x 56 x 56 (512 blocks) 19 / 21,
  // 16 x 56 x 56 (1024) 36 / 27, 24 x 56 x 56 47 / 39, 48 x 56 x 56 84 / 77,
  // 4 x 112 x 112 39 / 27, 16 x 112 x 112 126 / 127; but with units of one block
  // (64 x 28 x 28) 26 / 34, with rows of a vector a lane (64 x 14 x 14 x 1024 in
  // 8 groups) 60 / 78.  ReLU gains where all is one turn and loses in several
  // (18 x 56 x 56 27 / 25, 4 x 112 x 112 29 / 24, 24 x 56 x 56 32 / 35,
  // 16 x 112 x 112 87 / 104) and stays with clusters, as does GELU, whose slope
  // is worked out twice (131 / 164).  With float32 gradients one turn under
  // SiLU, ReLU: 12 x 56 x 56 30 / 35, 28 / 28; 16 x 56 x 56 38 / 39, 35 / 32;
  // 4 x 112 x 112 42 / 39, 38 / 32; several, which read past L2 through
  // registers: 20 x 56 x 56 44 / 66, 41 / 50; 48 x 56 x 56 88 / 113, 81 / 97;
  // 16 x 112 x 112 134 / 149, 121 / 128; 32 x 64 x 64 x 320 95 / 192, 87 / 141.
  const bool gains = a.gdt == DC_F32 ? a.act != DC_ACT_GELU && image_bytes(a, true) * a.n <= kImagesBytes
                                     : a.act == DC_ACT_SILU;
  return !(backward && a.dt == DC_BF16 && gains && r.blocks > 1 && vr >= 256 &&
           p->blocks > 4 * kSms);
}

// The forward's table of channel statistics and its partial triples.
size_t stats_table(const ColTeam& c, int threads) {
  return ((size_t)c.rows * c.width + 1) / 2 * 2 * sizeof(float2) + (size_t)threads * sizeof(float4);
}

bool plan_cols(const NormArgs& a, bool backward, bool keep, NormPlan* p) {
  ColTeam& c = p->col;
  const int v = p->s.v, elt = a.dt == DC_BF16 ? 2 : 4;
  const long long base = (long long)a.cpg / gcd(a.cpg, v) * v;  // whole groups, whole vectors
  if (base / v > 256 || v * elt < 4) return false;  // (an asynchronous copy moves 4 bytes at least)
  const int slices_most = (int)(a.c / base);
  const int held_bytes = v * (elt + (backward ? (keep ? 4 : 2) : 0));  // of a pixel's column
  // the narrowest slice of 128 bytes a pixel, or of 64 where that leaves few
  // blocks or does not fit in a cluster (32 bytes, one sector of a line, took
  // 32 us on the forward of 2 x 150 x 250 x 256 where two launches take 28, and
  // 170 on the backward of 16 x 112 x 112 x 256 where they take 114)
  for (int bytes = 128; bytes >= 64; bytes /= 2) {
    int m = 1;
    while (m < slices_most && (m * base * elt < bytes || slices_most % m)) ++m;
    while (m > 1 && (m * base / v > 256 || m * base / a.cpg > kMaxGroups || slices_most % m)) --m;
    c.width = (int)(m * base);
    c.slices = a.c / c.width;
    c.cb = c.width / v;
    c.ng = c.width / a.cpg;
    c.blocks = cluster_of((double)a.hw * c.cb * held_bytes, (long long)a.n * c.slices);
    const bool fits = (double)a.hw * c.cb * held_bytes <= (double)kMaxCluster * kBlockBytes;
    if (fits && (bytes == 64 || (long long)a.n * c.slices * c.blocks >= 2 * kSms)) break;
  }
  if (c.ng > kMaxGroups || (double)a.hw * c.cb * held_bytes > (double)kMaxCluster * kBlockBytes)
    return false;
  const long long units = (long long)a.n * c.slices;
  if (units * c.blocks > INT_MAX) return false;
  c.span = (int)ceil_div_ll(a.hw, c.blocks);
  c.rl = threads_of((double)c.span * c.cb) / c.cb;
  if (c.rl < 1) c.rl = 1;
  if (c.rl > c.span) c.rl = c.span;
  const int slots = (int)ceil_div_ll(c.span, c.rl);
  p->threads = (int)ceil_div_ll((long long)c.rl * c.cb, 32) * 32;
  const long long slot = (long long)p->threads * held_bytes;
  c.held = slot * slots <= kBlockBytes ? slots : (int)(kBlockBytes / slot);
  c.rows = 32 % c.cb ? c.rl : p->threads / 32;
  p->smem = (size_t)(slot * c.held) +
            (size_t)(c.blocks * c.ng * (backward ? 2 : 3) + 3) / 4 * 4 * sizeof(float);
  if (backward)
    p->smem += (size_t)c.rows * c.width * sizeof(float2);
  else if (a.cpg % v)
    p->smem += stats_table(c, p->threads);
  p->blocks = (unsigned)(units * c.blocks);
  p->parts = c.blocks;
  // A backward block reads nothing while it works on what it holds, so where
  // the blocks are more than run at once, of units that take three blocks or
  // more, two launches are faster: us of a bf16 SiLU backward on h x w x 256,
  // clusters / two launches: 4 x 56 x 56 (224 blocks) 12 / 18.5, 8 x 56 x 56
  // (448) 24 / 24, 16 x 56 x 56 (896) 46 / 31, 64 x 28 x 28 39 / 33, but with
  // units of one block, 512 x 14 x 14, 59 / 76, and of float32 tensors 46 / 50
  // on 16 x 56 x 56.  With float32 gradients 45 / 37 under ReLU, 8 x 56 x 56
  // 24 / 26, but with channels of two groups in a vector (10 a group of 320)
  // 70 / 94.
  const bool gains = a.dt == DC_BF16 && c.blocks > 2 && (a.gdt == DC_BF16 || a.cpg % v == 0);
  return !(backward && gains && p->blocks > 3 * kSms);
}

// Two launches: blocks of a unit, `vectors` of it in all, as many as an SM runs
// at once (`per_sm`; a third more of them wait for a whole turn, 43 us become
// 51 on the forward of 2 x 200 x 336 x 256).
int loose_blocks(long long units, double vectors, int per_sm) {
  long long k = per_sm * kSms / units;
  const long long most = (long long)(vectors / (8 * kTwo));
  if (k > most) k = most;
  return (int)(k < 1 ? 1 : k);
}

void plan_two(const NormArgs& a, bool backward, int planes, NormPlan* p) {
  Shape& s = p->s;
  const int vec = a.dt == DC_BF16 ? 8 : 4, elt = a.dt == DC_BF16 ? 2 : 4;
  const int gelt = a.gdt == DC_F32 ? 4 : 2;
  const double images = kImagesBytes / image_bytes(a, backward);
  p->images = images < 1 ? 1 : images >= a.n ? a.n : (int)images;
  // as many at a time in every turn
  p->images = (int)ceil_div_ll(a.n, ceil_div_ll(a.n, p->images));
  p->threads = kTwo;
  if (!a.nhwc) {
    RowTeam& r = p->row;
    const int vr = row_vectors(a.hw, a.hw % vec ? vec - 1 : 0, vec);
    const long long units = (long long)p->images * a.groups, run = (long long)a.cpg * vr;
    r.blocks = loose_blocks(units, (double)run, 4);
    if (ceil_div_ll(run, r.blocks) > 1 << 30) r.blocks = (int)ceil_div_ll(run, 1 << 30);
    r.units = 1;
    r.warps = kTwo / 32;
    r.span = (int)ceil_div_ll(run, r.blocks);
    r.step_c = kTwo / vr;
    r.step_v = kTwo % vr;
    s.parts = (int)ceil_div_ll(vr, 16 * s.lpr);
    s.seg = (int)ceil_div_ll(vr, s.parts);
    s.parts = (int)ceil_div_ll(vr, s.seg);
    r.tasks = (int)(ceil_div_ll(a.cpg, 32 / s.lpr) * s.parts);
    r.rounds = (int)ceil_div_ll(r.tasks, (long long)r.blocks * r.warps);
    p->parts = s.parts;
    // the ring's slots, of x and of grad_y in 16-byte pieces
    if (backward && elt == gelt) p->smem = (size_t)kRing * 2 * vec * (elt + gelt) * kTwo;
    return;
  }
  ColTeam& c = p->col;
  const int cols = a.c / s.v;
  c.slices = (int)ceil_div_ll(cols, 16);
  c.cb = (int)ceil_div_ll(cols, c.slices);
  c.slices = (int)ceil_div_ll(cols, c.cb);
  c.width = c.cb * s.v;
  c.rl = kTwo / c.cb;
  c.blocks = loose_blocks((long long)p->images * c.slices, (double)a.hw * c.cb, 3);
  c.span = (int)ceil_div_ll(a.hw, c.blocks);
  c.shares = c.slices == 1 ? 1 : (a.cpg + c.width - 2) / c.width + 1;
  c.rows = 32 % c.cb ? c.rl : kTwo / 32;
  // the ring's slots, and in their place after them the tables
  const size_t ring = backward ? (size_t)kRing * 2 * s.v * (elt + gelt) * kTwo
                               : (size_t)kRing * 4 * s.v * elt * kTwo;
  const size_t table = backward ? (size_t)c.rows * c.width * sizeof(float2)
                                : a.cpg % s.v ? stats_table(c, kTwo) : 0;
  p->smem = ring > table ? ring : table;
  p->parts = c.blocks;
}

void set_reciprocals(const NormArgs& a, NormPlan* p) {
  Shape& s = p->s;
  s.inv_total = (float)(1.0 / ((double)a.hw * a.cpg));
  s.inv_cpg = 1.f / a.cpg;
  s.inv_parts = s.parts ? 1.f / s.parts : 0.f;
  s.inv_cb = p->col.cb ? 1.f / p->col.cb : 0.f;
}

NormPlan make_plan(const NormArgs& a, bool backward) {
  NormPlan p{};
  p.s = make_shape(a);
  p.parts = 1;
  if (a.n == 0) return p;
  const bool keep = keep_dz(a.gdt == DC_F32, a.act == DC_ACT_SILU || a.act == DC_ACT_GELU);
  // 16-byte pieces of a held vector of x, and of one of grad_y
  const int planes = 1 + (backward ? (keep && a.dt == DC_BF16 ? 2 : 1) : 0);
  p.cluster = a.nhwc ? plan_cols(a, backward, keep, &p) : plan_rows(a, backward, planes, &p);
  if (!p.cluster) {
    p = NormPlan{};
    p.s = make_shape(a);
    plan_two(a, backward, planes, &p);
  }
  set_reciprocals(a, &p);
  return p;
}

}  // namespace

bool norm_supported(const NormArgs& a) {
  constexpr long long kGrid = (1LL << 31) - 1;
  if (a.c > 1 << 20 || (long long)a.n * a.c > kGrid) return false;
  if ((double)a.n * a.c * a.hw < 1e9) return true;
  for (int backward = 0; backward < 2; ++backward) {
    const NormPlan p = make_plan(a, backward != 0);
    if (p.cluster || a.n == 0) continue;
    const double blocks = a.nhwc ? (double)p.images * p.col.slices * p.col.blocks
                                 : (double)p.images * a.groups * p.row.blocks;
    const double tasks = a.nhwc ? 0 : ceil((double)a.cpg * p.s.lpr / 32) * p.s.parts;
    if (blocks > kGrid || tasks > 1 << 30) return false;
  }
  return true;
}

size_t norm_workspace_bytes(const NormArgs& a, bool backward) {
  if (a.n == 0) return 0;
  const NormPlan p = make_plan(a, backward);
  const size_t part = norm_part_bytes(p, a, backward);
  if (p.cluster) return part;
  const size_t entries = (size_t)a.n * a.groups *
                         (a.nhwc ? (size_t)p.col.blocks * p.col.shares : (size_t)p.row.blocks);
  return part + (entries * (backward ? sizeof(float2) : sizeof(float4)) + 255) / 256 * 256;
}

NormTurns norm_turns(const NormArgs& a, bool backward) {
  const NormPlan p = make_plan(a, backward);
  return NormTurns{p.cluster, p.cluster ? a.n : p.images};
}

cudaError_t launch_norm(const NormArgs& a, bool backward, cudaStream_t st) {
  const NormPlan p = make_plan(a, backward);
  return a.nhwc ? launch_nhwc(p, a, backward, st) : launch_nchw(p, a, backward, st);
}

cudaError_t launch_norm_two(const NormArgs& a, bool backward, bool second, int img0, int count,
                            cudaStream_t st) {
  const NormPlan p = make_plan(a, backward);
  return a.nhwc ? launch_two_nhwc(p, a, backward, second, img0, count, st)
                : launch_two_nchw(p, a, backward, second, img0, count, st);
}

cudaError_t launch_norm_params(const NormArgs& a, cudaStream_t st) {
  const NormPlan p = make_plan(a, true);
  return launch_plain(sum_images, (unsigned)ceil_div_ll(a.c, 32), 1024, st,
                      (long long)p.parts * a.n, a.c, reinterpret_cast<const float2*>(a.ws),
                      a.ggamma, a.gbeta);
}

}  // namespace dc
