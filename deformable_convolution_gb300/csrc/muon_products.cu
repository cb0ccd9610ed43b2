// The Newton-Schulz steps on the 5th-generation tensor cores, all of them in
// one launch.
//
// X (rows x cols, kept times 2^12 as a pair of 16-bit floats, high and low
// part) goes through
//   gram: A = X X^T                  (tall: X^T X)        A = R + diag(d)
//   poly: P = b A + c A A                                 P = S + diag(e)
//   apply: X' = a X + P X            (tall: a X + X P)
// with float32 accumulators.  The diagonals d and e are kept apart in float32:
//   R R gives A A = R R + (d_i + d_j) R + diag(d^2), and P X = S X + diag(e) X,
// so what is rounded to 16 bits for a product is the part off the diagonal,
// small where the rows come close to being orthogonal.  DC_ORTHO_16 multiplies
// the high parts (11 bits): relative error 1e-3 or less for gradients and
// random matrices from 64 x 64 to 1024 x 1024, against 2e-3 .. 4e-3 with the
// diagonal left in.  DC_ORTHO_32 (and a side under 64) adds high low + low high
// (low low is below the last bit kept).  The tensor cores truncate their sums
// after each product of 16, so these small terms of a block come first, and an
// accumulator runs over kRun blocks, whose sums are added up in registers:
// relative error against 64 bits 2.6e-6 for 600 x 1000 and 2048 x 2048, 3.3e-6
// for 700 x 70000, 1e-6 for 256 x 2304 (float32 arithmetic: 3.1e-6, 3.6e-6,
// 1.4e-5, 2e-6).  Four of 2048 x 2048 take 1538 us so; runs of 16 blocks 1394 us
// and 5.4e-6, a tile in one run 1289 us and 1.1e-5.
//
// CTAs work in pairs on tiles of 256 x bn (tc_pair.cuh).  A and P are
// symmetric: of their tiles only those that reach below the diagonal are
// computed, and what lies left of a diagonal block is stored at its mirrored
// place too.  X enters as it lies, whichever side is contracted: the tensor
// cores read 16-bit tiles in both orders.  A gram of few tiles splits its long
// side over several pairs: each leaves its sums in the workspace, and tiles of a
// kind of their own (sum: 16 columns of a tile) add them up in order.
//
// The launch is cooperative and walks one list of tiles, step by step, kind by
// kind, matrix by matrix, dealt to the pairs in turn; a tile waits (on a count
// in the workspace) for its own matrix's tiles of the kind before it.  Those
// stand before it in the list, so the first unfinished tile never waits.  A
// launch for each of the 15 kinds and steps took 6 to 7 us where the matrices
// are small (prologue, drain and cold caches each time), a wait takes 2.
//
// Warps of each CTA: 0-7 results, 8 TMA loads, 9 (of the first CTA) MMAs.
#include <cuda.h>

#include "muon.cuh"
#include "once.cuh"
#include "tc_pair.cuh"

namespace dc {

__device__ unsigned int g_muon_error;  // raised by this file's bounded waits

namespace {

using namespace pair;

constexpr int kBK = 64, kBox = 64 * 128;  // a box: 64 lines of 64 elements
constexpr int kEpiWarps = 8, kWarpTma = 8, kWarpMma = 9, kThreads = 320;
constexpr int kPart = 2 * kBox;           // one part of a factor in a stage: 128 lines
constexpr int kStage = 2 * kPart;         // one part of both factors
constexpr int kStages = 5, kRing = kStages * kStage;
constexpr int kSumCols = 16;              // columns of a tile that a sum adds up
constexpr int kRun = 8;                   // blocks of 64 that an accumulator with low parts' terms runs over
constexpr int kBuf = 4096;                // a warp's 32 x 32 results, and as much for their own terms
constexpr size_t kSmem = 1024 + kRing + kEpiWarps * 2 * kBuf + 256;
static_assert(kSmem <= 227 * 1024, "shared memory");
enum { GRAM = 0, SUM = 1, POLY = 2, APPLY = 3, KINDS = 4 };

struct Item {
  CUtensorMap x[2], gram, poly;
  MuonMat m;
  int start[KINDS];            // first tile in the lists of the kinds
  int tiles[KINDS];            // in a step (gram: of its splits; sum: 0 where it has one)
  int tiles_n[KINDS], bn[KINDS];
  int splits, per_split;       // of gram, in blocks of 64
  int vec;                     // the result's rows are whole 16-byte pieces
  int pairs;                   // the low parts are multiplied
};

template <int CAP>
struct Items {
  int count, steps;
  int n[KINDS];                // tiles of a kind in one step
  bool update;
  float lr;
  const float* grad_scale;
  const float* lr_device;
  Item item[CAP];
};

static_assert(sizeof(Items<kMuonMats>) <= 32 * 1024 - 4, "kernel arguments");

// Of the tiles of a symmetric result those that reach below the diagonal, row
// of tiles by row: row i has min(tiles_n, (i + 1) * 256 / bn) of them.
int lower_tiles(int rows, int tiles_n, int bn) {
  int n = 0;
  for (int i = 0; i * 256 < rows; ++i) n += (i + 1) * (256 / bn) < tiles_n ? (i + 1) * (256 / bn) : tiles_n;
  return n;
}

struct Tile {
  const Item* t;
  int which, step, index, m0, n0, bn, split, begin, end;
  bool diagonal;  // the rows of both factors are the same ones
};

template <int CAP>
__device__ __forceinline__ Tile tile_of(const Items<CAP>& g, int w) {
  Tile q;
  const int per = g.n[0] + g.n[1] + g.n[2] + g.n[3];
  q.step = w / per;
  int r = w - q.step * per;
  q.which = GRAM;
#pragma unroll
  for (int k = 0; k < KINDS - 1; ++k)
    if (q.which == k && r >= g.n[k]) r -= g.n[k], q.which = k + 1;
  int lo = 0, hi = g.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.item[mid].start[q.which] <= r)
      lo = mid;
    else
      hi = mid - 1;
  }
  q.t = &g.item[lo];
  const Item& t = *q.t;
  r -= t.start[q.which];
  // (a matrix without sums shares its place in their list with the next one)
  q.bn = t.bn[q.which];
  q.split = 0;
  q.begin = 0;
  q.end = (t.m.side + kBK - 1) / kBK;
  int chunk = 0;
  if (q.which == GRAM) {
    const int whole = t.tiles[GRAM] / t.splits;
    q.split = r / whole;
    r -= q.split * whole;
    q.begin = q.split * t.per_split;
    q.end = min(((t.m.tall ? t.m.rows : t.m.cols) + kBK - 1) / kBK, q.begin + t.per_split);
  } else if (q.which == SUM) {
    const int chunks = q.bn / kSumCols;
    chunk = r % chunks;
    r /= chunks;
    q.end = 0;
  }
  q.index = r;
  int i = 0;
  const int tn = t.tiles_n[q.which];
  if (q.which == APPLY) {
    i = r / tn;
    r -= i * tn;
  } else {
    for (;; ++i) {
      const int n = min(tn, (i + 1) * (256 / q.bn));
      if (r < n) break;
      r -= n;
    }
  }
  q.m0 = i * 256;
  q.n0 = r * q.bn;
  q.diagonal = q.bn == 256 && q.m0 == q.n0 && q.which != APPLY;
  if (q.which == SUM) q.split = chunk;  // the columns of the tile that it adds up
  return q;
}

// The tiles that this one reads are done: all CTAs' of the kind before it (of
// gram: of the step before it).
__device__ __forceinline__ bool inputs_done(const Tile& q) {
  const Item& t = *q.t;
  const int before = q.which == GRAM ? APPLY : q.which == POLY && t.splits == 1 ? GRAM : q.which - 1;
  const unsigned int want = 2u * (unsigned)t.tiles[before] * (unsigned)(q.which == GRAM ? q.step : q.step + 1);
  const unsigned int* count = t.m.done + before;
  // relaxed loads, one fence at the end: an acquire empties the L1 cache each time
  for (uint32_t i = 0; i < (1u << 22); ++i) {
    unsigned int v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
    if (v >= want) {
      asm volatile("fence.acq_rel.gpu;" ::: "memory");
      return true;
    }
    __nanosleep(64);
  }
  atomicOr(&g_muon_error, 1u);
  return false;
}

__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void epi_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// As that; whether `ok` holds for all.
__device__ __forceinline__ bool epi_all(bool ok) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, 1, 256, p;\n selp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)ok)
      : "memory");
  return r != 0;
}
// Generic and asynchronous accesses to global memory, in order.
__device__ __forceinline__ void fence_global_proxies() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Eight values as high and low parts, two in a word.
__device__ __forceinline__ void to_pairs(const float* v, uint4* hi, uint4* lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 a = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    const float2 b = __half22float2(a);
    const __half2 c = __floats2half2_rn(v[2 * i] - b.x, v[2 * i + 1] - b.y);
    h[i] = *reinterpret_cast<const uint32_t*>(&a);
    l[i] = *reinterpret_cast<const uint32_t*>(&c);
  }
  *hi = make_uint4(h[0], h[1], h[2], h[3]);
  *lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void from_pairs(uint4 hi, uint4 lo, float* v) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&l[i]));
    v[2 * i] = a.x + b.x;
    v[2 * i + 1] = a.y + b.y;
  }
}

// A warp's 32 x 32 results in shared memory: row r's 16-byte piece u stands at
// u ^ swizzle(r), so that rows' pieces, pairs of them and columns are read and
// written without two lanes in a bank.
__device__ __forceinline__ int swizzle(int r) { return ((r & 7) ^ ((r >> 3) << 1)) & 7; }

// The result of the last step: eight values of row r from column c on, written
// out or subtracted from the parameters.
template <int CAP>
__device__ __forceinline__ void write_result(const Items<CAP>& g, const Item& t, float lr, int r, int c, const float* x) {
  const long long at = (long long)r * t.m.cols + c;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i] * (1.f / kOrthoScale);
  const bool bf16 = t.m.out_dtype == DC_BF16;
  void* out = g.update ? t.m.param : t.m.out;
  if (g.update) {
    const float keep = 1.f - lr * t.m.weight_decay, rate = lr * t.m.rate;
    float p[8];
    if (t.vec) {
      if (t.m.master || !bf16) {
        const float4* f = reinterpret_cast<const float4*>((t.m.master ? t.m.master : static_cast<float*>(out)) + at);
        const float4 a = __ldcg(f), b = __ldcg(f + 1);
        p[0] = a.x, p[1] = a.y, p[2] = a.z, p[3] = a.w, p[4] = b.x, p[5] = b.y, p[6] = b.z, p[7] = b.w;
      } else {
        const uint4 a = __ldcg(reinterpret_cast<const uint4*>(static_cast<__nv_bfloat16*>(out) + at));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        p[i] = c + i >= t.m.cols ? 0.f
               : t.m.master      ? t.m.master[at + i]
               : bf16            ? __bfloat162float(static_cast<__nv_bfloat16*>(out)[at + i])
                                 : static_cast<float*>(out)[at + i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i] * keep - v[i] * rate;
  }
  if (t.vec) {
    if (!bf16 || (g.update && t.m.master)) {
      float4* f = reinterpret_cast<float4*>((bf16 ? t.m.master : static_cast<float*>(out)) + at);
      f[0] = make_float4(v[0], v[1], v[2], v[3]);
      f[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    if (bf16) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c + i < t.m.cols) {
        if (!bf16 || (g.update && t.m.master)) (bf16 ? t.m.master : static_cast<float*>(out))[at + i] = v[i];
        if (bf16) static_cast<__nv_bfloat16*>(out)[at + i] = __float2bfloat16_rn(v[i]);
      }
    }
  }
}

// A result warp's columns (32 each of `chunks`) of a tile of several runs, added
// up in registers and put back in place of the last run's.  j: as in the kernel,
// of the first run (whose sums are there); returns the last one's, or -1 where a
// wait expired.  (Not inline: its registers would be taken from the rest.)
__device__ __noinline__ int add_runs(uint32_t acc, int chunks, int runs, int j, uint64_t* tfull, uint32_t drained) {
  float total[4][32];
#pragma unroll 1
  for (int u = 0;; ++u, ++j) {
    if (u) {
      if (!epi_all(warp_wait(&tfull[j & 1], (j >> 1) & 1, &g_muon_error))) return -1;
      tc_after();
    }
    const uint32_t from = acc + (j & 1) * 256;
    const bool last = u + 1 == runs;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c < chunks) {
        uint32_t r[32];
        tmem_ld32(from + c * 32, r);
        tmem_ld_wait();
#pragma unroll
        for (int v = 0; v < 32; ++v) total[c][v] = (u ? total[c][v] : 0.f) + __uint_as_float(r[v]);
        if (last) tmem_st32(from + c * 32, total[c]);
      }
    }
    if (last) break;
    tc_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive_at(drained + 8 * (j & 1));
  }
  tmem_st_wait();
  return j;
}

// PAIRS: some of the matrices have their low parts multiplied, RUNS: some of
// their tiles have more than one run.
template <int CAP, bool PAIRS, bool RUNS>
__global__ void __launch_bounds__(kThreads, 1) muon_steps(const __grid_constant__ Items<CAP> g) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = px::align1024(smem_raw);
  unsigned char* stg = smem + kRing;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + kEpiWarps * 2 * kBuf);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* drained = tfull + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(drained + 2);

  // a step whose scale is not finite is skipped, by all alike
  if (g.update && g.grad_scale && !(fabsf(*g.grad_scale) <= 3.402823466e38f)) return;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int first = (int)blockIdx.x >> 1, stride = (int)gridDim.x >> 1;
  const int work = (g.n[0] + g.n[1] + g.n[2] + g.n[3]) * g.steps;

  if (warp == 0) tmem_alloc(holder);
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&drained[b], 2 * kEpiWarps);
    }
    px::fence_mbar_init();
  }
  tc_before();
  __syncthreads();
  cluster_sync();
  tc_after();
  const uint32_t tmem = *holder;
  bool ok = true;

  // Accumulators are two, by turns, one for a run: a tile or, where low parts are
  // multiplied, kRun blocks of it, added up in the result warps' registers.  j:
  // this pair's runs so far; each waits for the run before last to be read.
  if (warp == kWarpTma) {
    const bool issuer = elect_one();
    // both CTAs' copies count on the first one's barrier
    const uint32_t bar0 = in_cta(smem_u32(full), 0), ring = smem_u32(smem);
    int s = 0, round = 0;
    for (int w = first; w < work && ok; w += stride) {
      const Tile q = tile_of(g, w);
      if (q.which == SUM) continue;
      const MuonMat& m = q.t->m;
      bool here = true;
      if (lane == 0) here = inputs_done(q);
      here = __all_sync(0xffffffffu, here);
      __syncwarp();  // (a vote does not order memory: the other lanes read what lane 0 has waited for)
      if (!here) {
        ok = false;
        break;
      }
      fence_global_proxies();
      // factors and whether their contracted side runs across lines
      const CUtensorMap* x = &q.t->x[q.step & 1];
      const CUtensorMap* ta = q.which == GRAM ? x : q.which == POLY ? &q.t->gram : m.tall ? x : &q.t->poly;
      const CUtensorMap* tb = q.which == GRAM ? x : q.which == POLY ? &q.t->gram : m.tall ? &q.t->poly : x;
      const bool a_mn = q.which == GRAM && m.tall, b_mn = (q.which == GRAM && m.tall) || (q.which == APPLY && !m.tall);
      const int m0 = q.m0 + (int)rank * 128, n0 = q.n0 + (int)rank * (q.bn / 2);
      // boxes of B: none where its rows are A's
      const int nb = q.diagonal ? 0 : q.bn == 256 ? 2 : 1;
      const uint32_t bytes = 2u * (uint32_t)(2 + nb) * kBox;
      const int parts = PAIRS ? 1 + q.t->pairs : 1;
      for (int kb = q.begin; kb < q.end && ok; ++kb) {
        // the high parts in one stage, the low ones in the next
        for (int p = 0; p < parts; ++p) {
          if (round && !warp_wait(&empty[s], (round - 1) & 1, &g_muon_error)) {
            ok = false;
            break;
          }
          if (issuer) {
            const uint32_t bar = bar0 + s * 8, sa = ring + s * kStage, sb = sa + kPart;
            if (rank == 0) mbar_expect_tx(&full[s], bytes);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tma_load(sa + h * kBox, ta, bar, a_mn ? m0 + 64 * h : kb * kBK, a_mn ? kb * kBK : m0 + 64 * h, p);
              if (h < nb) tma_load(sb + h * kBox, tb, bar, b_mn ? n0 + 64 * h : kb * kBK, b_mn ? kb * kBK : n0 + 64 * h, p);
            }
          }
          __syncwarp();
          if (++s == kStages) s = 0, ++round;
        }
      }
    }
    if (!ok) let_copies_land();
  } else if (warp == kWarpMma) {
    if (rank == 0) {
      const bool issuer = elect_one();
      // along lines a step of 16 elements is 32 bytes on, across them 16 lines on
      const uint64_t along = sdesc(smem_u32(smem), 16, 1024), across = sdesc(smem_u32(smem), kBox, 1024);
      int s = 0, round = 0, j = 0;
      for (int w = first; w < work && ok; w += stride) {
        const Tile q = tile_of(g, w);
        if (q.which == SUM) continue;
        const bool a_mn = q.which == GRAM && q.t->m.tall;
        const bool b_mn = (q.which == GRAM && q.t->m.tall) || (q.which == APPLY && !q.t->m.tall);
        const bool pairs = PAIRS && q.t->pairs;
        const int run = RUNS && pairs ? kRun - 1 : INT_MAX;
        uint32_t acc = tmem;
        const uint32_t idesc = (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
                               ((uint32_t)(q.bn >> 3) << 17) | ((256u >> 4) << 24);
        const uint64_t a0 = a_mn ? across : along;
        const uint64_t b0 = (b_mn ? across : along) + (q.diagonal ? 0 : kPart >> 4);
        const uint32_t ka = a_mn ? 128 : 2, kb_step = b_mn ? 128 : 2;
        for (int kb = q.begin; kb < q.end; ++kb) {
          const bool begins = ((kb - q.begin) & run) == 0, ends = kb + 1 == q.end || ((kb + 1 - q.begin) & run) == 0;
          if (begins) {
            if (j >= 2 && !warp_wait(&drained[j & 1], ((j >> 1) - 1) & 1, &g_muon_error)) {
              ok = false;
              break;
            }
            acc = tmem + (j & 1) * 256;
          }
          const int s0 = s;
          bool here = warp_wait(&full[s0], round & 1, &g_muon_error);
          if (++s == kStages) s = 0, ++round;
          const int s1 = s;
          if (pairs) {
            here = here && warp_wait(&full[s1], round & 1, &g_muon_error);
            if (++s == kStages) s = 0, ++round;
          }
          if (!here) {
            ok = false;
            break;
          }
          tc_after();
          const uint64_t ah = a0 + (uint64_t)(s0 * (kStage >> 4)), bh = b0 + (uint64_t)(s0 * (kStage >> 4));
          const uint64_t al = a0 + (uint64_t)(s1 * (kStage >> 4)), bl = b0 + (uint64_t)(s1 * (kStage >> 4));
          const uint32_t more = begins ? 0u : 1u;
          if (issuer) {
            if (pairs) {  // small terms first, while the sums are
#pragma unroll
              for (int k = 0; k < kBK / 16; ++k)  // high low
                umma_f16(acc, ah + k * ka, bl + k * kb_step, idesc, k ? 1u : more);
#pragma unroll
              for (int k = 0; k < kBK / 16; ++k)  // low high
                umma_f16(acc, al + k * ka, bh + k * kb_step, idesc, 1u);
              commit_both(&empty[s1]);
            }
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)  // high high
              umma_f16(acc, ah + k * ka, bh + k * kb_step, idesc, k || pairs ? 1u : more);
            commit_both(&empty[s0]);
            if (ends) commit_both(&tfull[j & 1]);
          }
          __syncwarp();
          j += ends;
        }
      }
    }
  } else {
    const int quad = warp & 3, half = warp >> 2;
    float* buf = reinterpret_cast<float*>(stg + warp * 2 * kBuf);
    const unsigned char* terms = reinterpret_cast<const unsigned char*>(buf) + kBuf;
    const float lr = g.lr_device ? *g.lr_device : g.lr;
    const int sub = lane >> 2, piece = lane & 3;  // eight columns of a row for a lane, rows 8 i + sub
    int j = 0;  // runs so far
    for (int w = first; w < work; w += stride) {
      const Tile q = tile_of(g, w);
      const Item& t = *q.t;
      const MuonMat& m = t.m;
      const int rows = q.which == APPLY ? m.rows : m.side;
      const int cols = q.which == APPLY ? m.cols : q.which == SUM ? min(m.side, q.n0 + (q.split + 1) * kSumCols) : m.side;
      const long long ld = q.which == APPLY ? m.ld : m.lds;
      const long long low = q.which == APPLY ? muon_x_low(m) : muon_p_low(m);
      const __half* add = q.which == POLY ? m.gram : m.x[q.step & 1];
      const bool gram = q.which == GRAM || q.which == SUM;
      __half* out = gram ? m.gram : q.which == POLY ? m.poly : m.x[1 - (q.step & 1)];
      const bool last_step = q.which == APPLY && q.step + 1 == g.steps;
      const bool pairs = PAIRS && t.pairs;
      const bool store_low = q.which != POLY || pairs;
      float* diag_out = gram ? m.gram_diag : m.poly_diag;
      const int chunks = q.which == SUM ? 1 : q.bn / 64;  // of 32 columns, for each half of the columns
      const int row0 = q.m0 + (int)rank * 128 + quad * 32;
      const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
      const bool split = q.which == GRAM && t.splits > 1;  // sums to the workspace
      // 16-byte pieces of a split's 32 columns of a tile, in the order that warps hold them
      auto place = [&](int k, int chunk) {
        const int whole = t.tiles[GRAM] / t.splits;
        return reinterpret_cast<float4*>(m.sums) +
               ((((long long)k * whole + q.index) * 2 + rank) * (q.bn / 32) + chunk) * 1024 + quad * 256 + lane;
      };

      // The result is mul * sum + (c0 + cr * row's diagonal + cc * column's) *
      // own term: X, or R.  Terms come through shared memory by asynchronous
      // copies, a chunk ahead; a lane reads those that it copied.
      const bool tall_apply = q.which == APPLY && m.tall;
      const float unit = 1.f / kOrthoScale;
      const float mul = q.which == POLY ? kOrthoC * unit : unit;
      const float c0 = q.which == POLY ? kOrthoB : kOrthoA;
      const float cr = q.which == POLY ? kOrthoC : tall_apply ? 0.f : 1.f;
      const float cc = q.which == POLY ? kOrthoC : tall_apply ? 1.f : 0.f;
      const float* diag = q.which == POLY ? m.gram_diag : m.poly_diag;
      float row_diag = 0.f, col_diag[8], next_diag[8];  // row_diag: of row `lane`
      auto load_terms = [&](int c) {
        const int col = q.n0 + (half * chunks + c) * 32 + 8 * piece;
        if (!gram && col < cols) {
          const __half* from = add + (row0 + sub) * ld + col;
          const uint32_t to = smem_u32(terms) + lane * 16;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (row0 + 8 * i + sub < rows) {
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 512), "l"(from + 8 * i * ld) : "memory");
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 512 + 2048), "l"(from + 8 * i * ld + low)
                           : "memory");
            }
          }
          if (cc != 0.f) {
            const float4 a = __ldcg(reinterpret_cast<const float4*>(diag + col));
            const float4 b = __ldcg(reinterpret_cast<const float4*>(diag + col) + 1);
            next_diag[0] = a.x, next_diag[1] = a.y, next_diag[2] = a.z, next_diag[3] = a.w;
            next_diag[4] = b.x, next_diag[5] = b.y, next_diag[6] = b.z, next_diag[7] = b.w;
          }
        }
      };
#pragma unroll
      for (int k = 0; k < 8; ++k) next_diag[k] = 0.f;
      bool here = true;
      if (lane == 0) here = inputs_done(q);
      here = __all_sync(0xffffffffu, here);
      __syncwarp();
      if (here) {
        if (!gram && cr != 0.f && row0 + lane < rows) row_diag = __ldcg(diag + row0 + lane);
        load_terms(0);
      }
      // (all warps go on or none: they meet at barriers below)
      ok = epi_all(here && (q.which == SUM || warp_wait(&tfull[j & 1], (j >> 1) & 1, &g_muon_error)));
      if (!ok) break;
      tc_after();

      auto release = [&] {
        tc_before();
        __syncwarp();
        if (lane == 0) arrive_at(in_cta(smem_u32(&drained[j & 1]), 0));
      };
      if (RUNS && pairs && q.end - q.begin > kRun) {
        j = add_runs(lanes + half * chunks * 32, chunks, (q.end - q.begin + kRun - 1) / kRun, j, tfull,
                     in_cta(smem_u32(drained), 0));
        ok = j >= 0;
        if (!ok) break;
      }
      const uint32_t acc = lanes + (j & 1) * 256;
      auto results = [&](int c, uint32_t* r) {
        const uint32_t at = acc + (half * chunks + c) * 32;
        tmem_ld32(at, r);
        tmem_ld_wait();
      };
      if (split) {
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          const int chunk = half * chunks + c;
          uint32_t r[32];
          results(c, r);
          if (row0 < rows && q.n0 + chunk * 32 < cols) {
            float4* to = place(q.split, chunk);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              __stcg(to + 32 * v, make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                              __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3])));
          }
        }
        release();
      }
      const bool mirror = q.which != APPLY && q.n0 + q.bn <= q.m0;
#pragma unroll 1
      for (int c = split ? chunks : 0; c < chunks; ++c) {
        const int col0 = q.n0 + (q.which == SUM ? q.split * kSumCols : (half * chunks + c) * 32), col = col0 + 8 * piece;
        float4* line = reinterpret_cast<float4*>(buf + lane * 32);
        if (q.which == SUM) {
          // each half of the warps adds up half of the splits, in order; the first adds the second's sums to its own
          constexpr int kPieces = kSumCols / 4;
          float4 f[kPieces];
#pragma unroll
          for (int v = 0; v < kPieces; ++v) f[v] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row0 < rows && col0 < cols) {
            const int middle = (t.splits + 1) / 2, end = half ? t.splits : middle;
            const float4* from = place(half ? middle : 0, q.split / 2) + q.split % 2 * kPieces * 32;
            const long long next = place(1, 0) - place(0, 0);
#pragma unroll 6
            for (int k = half ? middle : 0; k < end; ++k, from += next) {
#pragma unroll
              for (int v = 0; v < kPieces; ++v) {
                const float4 u = __ldcg(from + 32 * v);
                f[v].x += u.x, f[v].y += u.y, f[v].z += u.z, f[v].w += u.w;
              }
            }
          }
          const float4* second = reinterpret_cast<const float4*>(stg + (warp | 4) * 2 * kBuf) + lane * 8;
          if (half) {
#pragma unroll
            for (int v = 0; v < kPieces; ++v) line[v ^ swizzle(lane)] = f[v];
          }
          epi_barrier();
          if (!half) {
#pragma unroll
            for (int v = 0; v < kPieces; ++v) {
              const float4 u = second[v ^ swizzle(lane)];
              line[v ^ swizzle(lane)] = make_float4(f[v].x + u.x, f[v].y + u.y, f[v].z + u.z, f[v].w + u.w);
            }
          }
        } else {
          uint32_t r[32];
          results(c, r);
          if (c == chunks - 1) release();
#pragma unroll
          for (int v = 0; v < 8; ++v)
            line[v ^ swizzle(lane)] = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                                  __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) col_diag[k] = next_diag[k];
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if (q.which == SUM && half) break;  // (the warp's one chunk)
        if (q.which != APPLY && (unsigned)(col0 - row0) < 32u) {
          // the diagonal, where R is 0: b d + c d^2 and the sum's (of gram d is 0 so far)
          const int cl = lane - (col0 - row0);  // this row's column of the chunk
          if (cl >= 0 && row0 + lane < min(rows, cols)) {
            float* on = buf + lane * 32 + (((cl >> 2) ^ swizzle(lane)) << 2) + (cl & 3);
            diag_out[row0 + lane] = *on * (mul * unit) + (kOrthoB + kOrthoC * row_diag) * row_diag;
            *on = 0.f;
          }
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rl = 8 * i + sub, r = row0 + rl;
          const float f = c0 + cr * __shfl_sync(0xffffffffu, row_diag, rl);
          if (r < rows && col < cols) {
            float4* p0 = reinterpret_cast<float4*>(buf + rl * 32) + ((2 * piece) ^ swizzle(rl));
            float4* p1 = reinterpret_cast<float4*>(buf + rl * 32) + ((2 * piece + 1) ^ swizzle(rl));
            const float4 a = *p0, b = *p1;
            float e[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) e[k] *= mul;
            if (!gram) {
              float x[8];
              const uint4* own = reinterpret_cast<const uint4*>(terms + i * 512) + lane;
              from_pairs(own[0], own[128], x);
#pragma unroll
              for (int k = 0; k < 8; ++k) e[k] += (f + cc * col_diag[k]) * x[k];
            }
            if (mirror || last_step) {
              *p0 = make_float4(e[0], e[1], e[2], e[3]);
              *p1 = make_float4(e[4], e[5], e[6], e[7]);
            }
            if (!last_step) {
              // whole 16-byte pieces: what lies past the last column is of no meaning
              uint4 h, l;
              to_pairs(e, &h, &l);
              *reinterpret_cast<uint4*>(out + r * ld + col) = h;
              if (store_low) *reinterpret_cast<uint4*>(out + low + r * ld + col) = l;
            }
          }
        }
        if (c + 1 < chunks) load_terms(c + 1);
        if (mirror || last_step) {
          __syncwarp();
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            float e[8];
            if (mirror) {
              // the mirrored place: eight rows of a column for a lane; columns left of a diagonal block are rows that exist
              const int cl = 8 * i + sub;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int rl = 8 * piece + k;
                e[k] = buf[rl * 32 + (((cl >> 2) ^ swizzle(rl)) << 2) + (cl & 3)];
              }
              if (row0 + 8 * piece < rows && col0 + cl < cols) {
                uint4 h, l;
                to_pairs(e, &h, &l);
                __half* to = out + (col0 + cl) * ld + row0 + 8 * piece;
                *reinterpret_cast<uint4*>(to) = h;
                if (store_low) *reinterpret_cast<uint4*>(to + low) = l;
              }
            } else {
              const int rl = 8 * i + sub;
              const float4 a = reinterpret_cast<const float4*>(buf + rl * 32)[(2 * piece) ^ swizzle(rl)];
              const float4 b = reinterpret_cast<const float4*>(buf + rl * 32)[(2 * piece + 1) ^ swizzle(rl)];
              e[0] = a.x, e[1] = a.y, e[2] = a.z, e[3] = a.w, e[4] = b.x, e[5] = b.y, e[6] = b.z, e[7] = b.w;
              if (row0 + rl < rows && col < cols) write_result(g, t, lr, row0 + rl, col, e);
            }
          }
        }
        __syncwarp();
      }
      if (q.which != SUM) ++j;
      // this CTA's part of the tile is done
      fence_global_proxies();
      epi_barrier();
      if (threadIdx.x == 0) {
        __threadfence();
        asm volatile("red.relaxed.gpu.global.add.u32 [%0], %1;" ::"l"(m.done + q.which), "r"(1u) : "memory");
      }
    }
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  cluster_sync();
  tc_after();
  if (warp == 0) tmem_free(tmem);
}

// ---------------------------------------------------------------- host side

constexpr int kPairs = 76;  // of 152 SMs

bool pair_map(CUtensorMap* m, const void* base, int rows, int cols, int ld) {
  const unsigned long long dims[3] = {(unsigned long long)cols, (unsigned long long)rows, 2};
  const unsigned long long strides[2] = {2ull * ld, 2ull * ld * rows};
  const unsigned box[3] = {64, 64, 1};
  return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

int tiles_of(int which, int bn, int rows, int cols) {
  const int tiles_n = (cols + bn - 1) / bn;
  return which == APPLY ? (rows + 255) / 256 * tiles_n : lower_tiles(rows, tiles_n, bn);
}

// A matrix's tiles and splits go by its own size: its result does not depend on
// the matrices beside it.  Wide tiles read less of shared memory for each
// product, narrow ones fill more pairs and are finished sooner: the widest of
// which a matrix has enough.  Of gram 256 columns wherever there are as many,
// since a diagonal tile then has one factor to load instead of two (and the
// pairs are filled by splits).
int width_of(int which, int rows, int cols) {
  if (which == GRAM || which == SUM) return cols > 128 ? 256 : cols > 64 ? 128 : 64;
  return tiles_of(which, 256, rows, cols) >= 32 ? 256 : tiles_of(which, 128, rows, cols) >= 16 ? 128 : 64;
}

// Splits of a gram's long side, three blocks of 64 or more each, so that a
// matrix of one or three tiles (a short side up to 512) keeps up to 24 pairs
// busy.  (Eight of 1024 x 1024 split over four lost 40 us of 130 a step to
// adding up.  The rule was measured on those and on 256 x 2304; one matrix alone
// takes 136 us with 512 a side, 157 with 513, 152 with 640, 194 with 1024.)
int gram_splits(const MuonMat& t) {
  const int tiles = tiles_of(GRAM, width_of(GRAM, t.side, t.side), t.side, t.side);
  const int nkb = (int)ceil_div_ll(t.tall ? t.rows : t.cols, kBK);
  int want = tiles == 1 ? 12 : tiles == 3 ? 8 : 1;
  if (want > nkb / 3) want = nkb / 3;
  // And no accumulator of few tiles runs over more than 16 blocks (up to 48
  // splits), none over more than 256: the tensor cores truncate it after each of
  // 4 products a block (cross terms' tiles add up shorter runs).
  const int runs = (nkb + 15) / 16, least = (nkb + 255) / 256;
  if (tiles <= 3 && want < runs) want = runs < 48 ? runs : 48;
  if (want < least) want = least;
  if (want < 2) return 1;
  const int per = (nkb + want - 1) / want;
  return (nkb + per - 1) / per;
}

// (products of a short side under 64 cost nothing, and its matrix has few values
// for the roundings to average over)
bool takes_pairs(const MuonGroup& g, const MuonMat& t) { return g.precision == DC_ORTHO_32 || t.side < 64; }

template <int CAP, bool PAIRS, bool RUNS>
cudaError_t launch_as(const MuonGroup& m, cudaStream_t s) {
  Items<CAP> g;
  g.count = m.count;
  g.steps = m.steps;
  g.update = m.update;
  g.lr = m.lr;
  g.grad_scale = m.grad_scale;
  g.lr_device = m.lr_device;
  for (int k = 0; k < KINDS; ++k) g.n[k] = 0;
  for (int i = 0; i < m.count; ++i) {
    const MuonMat& t = m.mat[i];
    Item& q = g.item[i];
    q.m = t;
    const int nkb = (int)ceil_div_ll(t.tall ? t.rows : t.cols, kBK);
    q.splits = gram_splits(t);
    q.per_split = (nkb + q.splits - 1) / q.splits;
    for (int k = 0; k < KINDS; ++k) {
      const int rows = k == APPLY ? t.rows : t.side, cols = k == APPLY ? t.cols : t.side;
      q.bn[k] = width_of(k, rows, cols);
      q.tiles_n[k] = (cols + q.bn[k] - 1) / q.bn[k];
      q.tiles[k] = tiles_of(k, q.bn[k], rows, cols);
      if (k == GRAM) q.tiles[k] *= q.splits;
      if (k == SUM) q.tiles[k] = q.splits > 1 ? q.tiles[k] * (q.bn[k] / kSumCols) : 0;
      q.start[k] = g.n[k];
      g.n[k] += q.tiles[k];
    }
    const int e = t.out_dtype == DC_BF16 ? 2 : 4;
    const void* out = m.update ? t.param : t.out;
    q.pairs = takes_pairs(m, t);
    q.vec = t.cols % 8 == 0 && (uintptr_t)out % 16 == 0 && (uintptr_t)t.master % 16 == 0 && (t.cols * e) % 16 == 0;
    if (!pair_map(&q.x[0], t.x[0], t.rows, t.cols, t.ld) || !pair_map(&q.x[1], t.x[1], t.rows, t.cols, t.ld) ||
        !pair_map(&q.gram, t.gram, t.side, t.side, t.lds) || !pair_map(&q.poly, t.poly, t.side, t.side, t.lds))
      return cudaErrorInvalidValue;
  }
  static std::atomic<bool> allowed[kOnceDevices];
  cudaError_t e = allow_smem_once(muon_steps<CAP, PAIRS, RUNS>, kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * kPairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // pairs that run at once: all of them have to, for tiles wait for one another
  static std::atomic<int> at_once[kOnceDevices];
  int dev = 0, most = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < kOnceDevices) most = at_once[dev].load(std::memory_order_relaxed);
  if (most == 0) {
    e = cudaOccupancyMaxActiveClusters(&most, muon_steps<CAP, PAIRS, RUNS>, &cfg);
    if (e != cudaSuccess) return e;
    if (dev < kOnceDevices) at_once[dev].store(most, std::memory_order_relaxed);
  }
  int widest = 0;  // more pairs than the widest kind of a step has tiles would only wait
  for (int k = 0; k < KINDS; ++k)
    if (g.n[k] > widest) widest = g.n[k];
  if (most > widest) most = widest;
  if (most > kPairs) most = kPairs;
  if (most < 1) return cudaErrorLaunchOutOfResources;
  cfg.gridDim = dim3(2u * (unsigned)most);
  attr[1].id = cudaLaunchAttributeCooperative;
  attr[1].val.cooperative = 1;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, muon_steps<CAP, PAIRS, RUNS>, g);
  note_launches(1);
  return e;
}

// (one kernel for all took 630 us in place of 545 for four of 2048 x 2048, high
// parts only, and 237 in place of 200 for four pairs of 256 x 2304 and 18 x 2304
// with the low ones: the sums of runs take registers from all the rest)
template <int CAP>
cudaError_t launch(const MuonGroup& g, cudaStream_t s) {
  bool pairs = false, runs = false;
  for (int i = 0; i < g.count; ++i) {
    const MuonMat& t = g.mat[i];
    if (!takes_pairs(g, t)) continue;
    const int nkb = (int)ceil_div_ll(t.tall ? t.rows : t.cols, kBK), splits = gram_splits(t);
    pairs = true;
    runs = runs || t.side > kRun * kBK || (nkb + splits - 1) / splits > kRun;
  }
  return runs ? launch_as<CAP, true, true>(g, s)
         : pairs ? launch_as<CAP, true, false>(g, s) : launch_as<CAP, false, false>(g, s);
}

}  // namespace

size_t muon_sums_bytes(const MuonMat& t) {
  const int splits = gram_splits(t), bn = width_of(GRAM, t.side, t.side);
  return splits > 1 ? (size_t)splits * tiles_of(GRAM, bn, t.side, t.side) * 256 * bn * sizeof(float) : 0;
}

cudaError_t launch_muon_steps(const MuonGroup& g, cudaStream_t s) {
  if (g.count <= 2) return launch<2>(g, s);
  if (g.count <= 10) return launch<10>(g, s);
  return launch<kMuonMats>(g, s);
}

// This file's share of dc_device_error (2 = unreadable).
unsigned int muon_read_error(int clear) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_muon_error, sizeof(v)) != cudaSuccess) return 2u;
  if (clear && cudaMemcpyToSymbol(g_muon_error, &zero, sizeof(zero)) != cudaSuccess) return 2u;
  return v;
}

}  // namespace dc
