// Host-side checks of group norm's plans (compiled and run by
// tests/test_host_layout.py; no GPU).
//
//  * two launches over whole-vector rows: the blocks' runs cover a unit's
//    vectors in order and exactly once, up to the largest sizes accepted;
//  * a kernel's limit of dynamic shared memory is set to one value whatever the
//    problem (host threads that launch a kernel at the same time cannot lower it
//    under one another), and every launch stays within it;
//  * a cluster's blocks on [n][c][h][w] have a slot for every vector they take,
//    and take all of their unit's.
#include <cuda_runtime.h>

#include <set>

// Launches and limits are recorded, not made.
static std::set<int> limits;
static size_t launched_smem, most_smem;
template <typename K>
static cudaError_t record_attribute(K, cudaFuncAttribute attr, int value) {
  if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) limits.insert(value);
  return cudaSuccess;
}
template <typename K, typename... A>
static cudaError_t record_launch(const cudaLaunchConfig_t* c, K, A...) {
  launched_smem = c->dynamicSmemBytes;
  if (launched_smem > most_smem) most_smem = launched_smem;
  return cudaSuccess;
}
#define cudaFuncSetAttribute record_attribute
#define cudaLaunchKernelEx record_launch

#include "../../deformable_convolution_gb300/csrc/group_norm.cu"

#include <cstdio>
#include <random>

namespace dc {
void note_launches(unsigned) {}
cudaError_t launch_nchw(const NormPlan&, const NormArgs&, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_nhwc(const NormPlan&, const NormArgs&, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_two_nchw(const NormPlan&, const NormArgs&, bool, bool, int, int, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_two_nhwc(const NormPlan&, const NormArgs&, bool, bool, int, int, cudaStream_t) {
  return cudaSuccess;
}
}  // namespace dc

using namespace dc;

static long long failures = 0, runs = 0, wide = 0, held = 0;
#define CHECK(cond, ...)                  \
  do {                                    \
    if (!(cond)) {                        \
      if (failures < 20) {                \
        printf("FAIL %s: ", #cond);       \
        printf(__VA_ARGS__);              \
        printf("\n");                     \
      }                                   \
      ++failures;                         \
    }                                     \
  } while (0)

static NormArgs make_args(int n, int groups, int cpg, long long hw, dc_dtype dt, dc_dtype gdt,
                          bool nhwc, int act) {
  NormArgs a{};
  a.n = n;
  a.c = groups * cpg;
  a.groups = groups;
  a.cpg = cpg;
  a.hw = (int)hw;
  a.nhwc = nhwc;
  a.act = act;
  a.eps = 1e-5f;
  a.dt = dt;
  a.gdt = gdt;
  return a;
}

static void check_runs(const NormArgs& a, const NormPlan& p) {
  const int vec = a.dt == DC_BF16 ? 8 : 4;
  if (a.hw % vec) return;
  const int vr = a.hw / vec;
  const long long total = (long long)a.cpg * vr;
  long long at = 0;
  for (int rank = 0; rank < p.row.blocks; ++rank) {
    const BlockRun r(a.cpg, vr, p.row.span, rank);
    if (r.count == 0) continue;
    CHECK(r.begin == at, "c %d hw %d rank %d: from %lld, not %lld", a.cpg, a.hw, rank, r.begin, at);
    CHECK(r.count > 0 && r.count <= 1 << 30, "c %d hw %d rank %d: %d vectors", a.cpg, a.hw, rank,
          r.count);
    at = r.begin + r.count;
  }
  CHECK(at == total, "c %d hw %d: %lld of %lld vectors", a.cpg, a.hw, at, total);
  ++runs;
  wide += total > INT_MAX;
}

__global__ void some_kernel(int) {}

static void check_smem(const NormArgs& a, const NormPlan& p) {
  launched_smem = 0;
  if (p.cluster)
    launch_team(some_kernel, p, a.nhwc ? p.col.blocks : p.row.blocks, nullptr, 0);
  else
    launch_smem(some_kernel, 1, p.threads, p.smem, nullptr, 0);
  CHECK(launched_smem == p.smem, "%zu bytes planned, %zu launched", p.smem, launched_smem);
}

static void check_slots(const NormArgs& a, const NormPlan& p, bool backward) {
  const RowTeam& r = p.row;
  const int vec = a.dt == DC_BF16 ? 8 : 4, threads = 32 * r.warps;
  const bool wide = keep_dz(a.gdt == DC_F32, a.act == DC_ACT_SILU || a.act == DC_ACT_GELU);
  const int planes = 1 + (backward ? (wide && a.dt == DC_BF16 ? 2 : 1) : 0);
  const long long slots = (long long)p.smem / 16 / planes;
  CHECK(p.threads == threads * r.units && p.threads <= kTeam, "%d threads", p.threads);
  CHECK((r.span != 0) == (!backward && a.hw % vec == 0), "hw %d: span %d", a.hw, r.span);
  if (r.span) {
    CHECK((long long)r.span * r.blocks >= (long long)a.cpg * (a.hw / vec), "span %d", r.span);
    CHECK(ceil_div_ll(r.span, threads) * p.threads <= slots, "hw %d: %lld slots", a.hw, slots);
  } else {
    const int per = 32 / p.s.lpr, vr = row_vectors(a.hw, a.hw % vec ? vec - 1 : 0, vec);
    CHECK((long long)p.s.seg * p.s.parts >= vr, "hw %d: segments", a.hw);
    CHECK((long long)r.rounds * r.blocks * r.warps >= r.tasks &&
              (long long)r.tasks * per >= (long long)a.cpg * p.s.parts, "hw %d: %d tasks", a.hw, r.tasks);
    CHECK((long long)r.rounds * r.warps * r.units * per * p.s.seg <= slots, "hw %d: %lld slots",
          a.hw, slots);
  }
  ++held;
}

static void check(const NormArgs& a) {
  if (!norm_supported(a)) return;
  for (int backward = 0; backward < 2; ++backward) {
    const NormPlan p = make_plan(a, backward != 0);
    if (!p.cluster && !a.nhwc && !backward) check_runs(a, p);
    if (p.cluster && !a.nhwc) check_slots(a, p, backward != 0);
    check_smem(a, p);
  }
}

int main() {
  // a group of 2^31 vectors, and the sizes around it
  for (const int cpg : {63, 64, 65, 72})
    check(make_args(1, 1, cpg, 1LL << 28, DC_BF16, DC_BF16, false, DC_ACT_SILU));
  check(make_args(1, 1, 24, 1LL << 30, DC_BF16, DC_BF16, false, DC_ACT_SILU));
  check(make_args(1, 1, 1024, 1LL << 30, DC_BF16, DC_BF16, false, DC_ACT_NONE));
  check(make_args(2, 3, 1 << 16, 1 << 20, DC_F32, DC_F32, false, DC_ACT_RELU));
  // a bf16 backward with a float32 gradient reads its inputs twice only where
  // L2 holds all of them
  for (const int n : {16, 18, 20, 48})
    for (const int act : {DC_ACT_RELU, DC_ACT_SILU}) {
      const NormArgs a = make_args(n, 32, 8, 56 * 56, DC_BF16, DC_F32, false, act);
      CHECK(make_plan(a, true).cluster == (n > 19), "%d images", n);
    }
  std::mt19937_64 rng(1);
  auto spread = [&](double lo, double hi) {
    return (long long)std::lround(
        std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng)));
  };
  for (int i = 0; i < 300000; ++i) {
    const int groups = (int)spread(1, 64), cpg = (int)spread(1, 4000), n = (int)spread(1, 600);
    long long hw = spread(1, 1 << 30);
    if (rng() % 4) hw = (hw + 7) / 8 * 8;
    if (hw > 1 << 30 || (double)n * groups * cpg * (double)hw > (double)(1LL << 40)) continue;
    const dc_dtype dt = rng() % 2 ? DC_BF16 : DC_F32;
    check(make_args(n, groups, cpg, hw, dt, rng() % 2 ? DC_F32 : dt, rng() % 2, (int)(rng() % 4)));
  }
  // 227 KB are a block's at most, of which the static arrays take up to 8
  CHECK(limits.size() == 1 && *limits.begin() <= (227 - 8) * 1024, "%zu limits, the largest %d",
        limits.size(), *limits.rbegin());
  CHECK(most_smem <= (size_t)*limits.begin(), "%zu bytes launched", most_smem);
  printf("%lld sizes in runs, %lld of them past 32 bits, %lld held by clusters, %lld failures\n", runs,
         wide, held, failures);
  return failures || runs < 1000 || wide < 100 || held < 1000;
}
