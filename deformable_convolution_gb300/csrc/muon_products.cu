// The products of the Newton-Schulz steps on the 5th-generation tensor cores.
//
// X (rows x cols, kept times 2^12 as a pair of 16-bit floats, high and low
// part) goes through
//   gram: A = X X^T          (tall: X^T X)
//   poly: P = b A + c A A
//   apply: X' = a X + P X    (tall: a X + X P)
// with float32 accumulators.  A factor's two parts hold 22 bits or more; a
// product of pairs is high high + high low + low high, three MMAs on tiles that
// are loaded once (low low is below the last bit kept).  DC_ORTHO_16 takes X's
// high part alone: one MMA for A and two for P X; A A keeps all three, it is
// the small product of a long matrix.
//
// All of a group's matrices run in one launch of each kind.  CTAs work in
// pairs on tiles of 256 x BN (tc_pair.cuh), persistent.  A and P are symmetric:
// of their tiles only those that reach below the diagonal are computed, and
// what lies below a diagonal block is stored at its mirrored place too.  X
// enters as it lies, whichever side is contracted: the tensor cores read 16-bit
// tiles in both orders.  A gram of few tiles splits its long side over several
// pairs: each leaves its sums in the workspace, the last one to arrive adds
// them up in order (no result depends on who that is).
//
// Warps of each CTA: 0-7 results, 8 TMA loads, 9 (of the first CTA) MMAs.
#include <cuda.h>

#include "muon.cuh"
#include "tc_pair.cuh"

namespace dc {

__device__ unsigned int g_muon_error;  // raised by this file's bounded waits

namespace {

using namespace pair;

constexpr int kBK = 64, kBox = 64 * 128;  // a box: 64 lines of 64 elements
constexpr int kEpiWarps = 8, kWarpTma = 8, kWarpMma = 9, kThreads = 320;

struct Item {
  CUtensorMap a, b;
  const __half* add;  // the pair that the result's own term comes from (poly, apply)
  __half* out;
  float* part;        // splits: sums of [split][tile][rank], else null
  unsigned int* count;
  long long ld, low;  // of add and out
  int rows, cols, nkb, tiles_n, tiles, splits, per_split;
  int start;          // first work item
  int a_mn, b_mn;     // the contracted side is the factor's rows
  int a_low, b_low;   // the factor's low part is used
};

template <int CAP>
struct Items {
  int which, count, work;
  Item item[CAP];
};

template <int BN>
struct Cfg {
  static constexpr int kA = 2 * kBox, kB = BN / 128 * kBox;  // one part of a factor in a stage
  static constexpr int kStage = 2 * (kA + kB);
  static constexpr int kStages = BN == 256 ? 3 : 4;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 256;
};

// Of the tiles of a symmetric result those that reach below the diagonal, row
// of tiles by row: row i has min(tiles_n, (i + 1) * 256 / BN) of them.
template <int BN>
__host__ __device__ inline int lower_tiles(int rows, int tiles_n) {
  int n = 0;
  for (int i = 0; i * 256 < rows; ++i) n += (i + 1) * (256 / BN) < tiles_n ? (i + 1) * (256 / BN) : tiles_n;
  return n;
}

struct Tile {
  const Item* t;
  int index, m0, n0, split, begin, end;
};

template <int BN, int CAP>
__device__ __forceinline__ Tile tile_of(const Items<CAP>& g, int w) {
  int lo = 0, hi = g.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.item[mid].start <= w)
      lo = mid;
    else
      hi = mid - 1;
  }
  Tile q;
  q.t = &g.item[lo];
  const Item& t = *q.t;
  int r = w - t.start;
  q.split = r / t.tiles;
  r -= q.split * t.tiles;
  q.index = r;
  if (g.which == 2) {
    const int i = r / t.tiles_n;
    q.m0 = i * 256;
    q.n0 = (r - i * t.tiles_n) * BN;
  } else {
    int i = 0;
    for (;; ++i) {
      const int n = min(t.tiles_n, (i + 1) * (256 / BN));
      if (r < n) break;
      r -= n;
    }
    q.m0 = i * 256;
    q.n0 = r * BN;
  }
  q.begin = q.split * t.per_split;
  q.end = min(t.nkb, q.begin + t.per_split);
  return q;
}

__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A value as high and low part.
__device__ __forceinline__ void to_pair(float v, __half* hi, __half* lo) {
  *hi = __float2half_rn(v);
  *lo = __float2half_rn(v - __half2float(*hi));
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

template <int BN, int CAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    muon_mm(const __grid_constant__ Items<CAP> g) {
  using C = Cfg<BN>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = px::align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* drained = tfull + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(drained + 2);
  uint32_t* arrived = holder + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int first = (int)blockIdx.x >> 1, stride = (int)gridDim.x >> 1;

  if (warp == 0) tmem_alloc(holder);
  if (threadIdx.x == 32) {
    for (int s = 0; s < C::kStages; ++s) {
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
  pdl_wait();
  pdl_release();

  if (warp == kWarpTma) {
    if (lane == 0) {
      int it = 0;
      for (int w = first; w < g.work && ok; w += stride) {
        const Tile q = tile_of<BN>(g, w);
        const Item& t = *q.t;
        const int m0 = q.m0 + (int)rank * 128, n0 = q.n0 + (int)rank * (BN / 2);
        const uint32_t bytes = 2u * (C::kA * (1 + t.a_low) + C::kB * (1 + t.b_low));
        for (int kb = q.begin; kb < q.end; ++kb, ++it) {
          const int s = it % C::kStages;
          if (it >= C::kStages && !mbar_wait(&empty[s], ((it / C::kStages) - 1) & 1, &g_muon_error)) {
            ok = false;
            break;
          }
          const uint32_t bar = in_cta(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_expect_tx(&full[s], bytes);
          const uint32_t sa = smem_u32(smem + s * C::kStage), sb = sa + 2 * C::kA;
          for (int p = 0; p <= t.a_low; ++p)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load(sa + p * C::kA + h * kBox, &t.a, bar, t.a_mn ? m0 + 64 * h : kb * kBK,
                       t.a_mn ? kb * kBK : m0 + 64 * h, p);
          for (int p = 0; p <= t.b_low; ++p)
#pragma unroll
            for (int h = 0; h < BN / 128; ++h)
              tma_load(sb + p * C::kB + h * kBox, &t.b, bar, t.b_mn ? n0 + 64 * h : kb * kBK,
                       t.b_mn ? kb * kBK : n0 + 64 * h, p);
        }
      }
      if (!ok) let_copies_land();
    }
  } else if (warp == kWarpMma) {
    if (rank == 0 && lane == 0) {
      int it = 0, j = 0;
      for (int w = first; w < g.work && ok; w += stride, ++j) {
        const Tile q = tile_of<BN>(g, w);
        const int a_mn = q.t->a_mn, b_mn = q.t->b_mn, a_low = q.t->a_low, b_low = q.t->b_low;
        if (j >= 2 && !mbar_wait(&drained[j & 1], ((j >> 1) - 1) & 1, &g_muon_error)) {
          ok = false;
          break;
        }
        tc_after();
        const uint32_t acc = tmem + (j & 1) * 256;
        const uint32_t idesc = (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
                               ((uint32_t)(BN >> 3) << 17) | ((256u >> 4) << 24);
        for (int kb = q.begin; kb < q.end; ++kb, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&full[s], (it / C::kStages) & 1, &g_muon_error)) {
            ok = false;
            break;
          }
          tc_after();
          const uint32_t sa = smem_u32(smem + s * C::kStage), sb = sa + 2 * C::kA;
#pragma unroll
          for (int p = 0; p < 3; ++p) {  // high high, high low, low high
            if ((p == 1 && !b_low) || (p == 2 && !a_low)) continue;
            const uint32_t pa = sa + (p == 2 ? C::kA : 0), pb = sb + (p == 1 ? C::kB : 0);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) {
              // along lines: 32 bytes on; across them: 16 lines on
              const uint64_t da = a_mn ? sdesc(pa + k * 2048, kBox, 1024) : sdesc(pa + k * 32, 16, 1024);
              const uint64_t db = b_mn ? sdesc(pb + k * 2048, kBox, 1024) : sdesc(pb + k * 32, 16, 1024);
              umma_f16(acc, da, db, idesc, (kb > q.begin || p > 0 || k > 0) ? 1u : 0u);
            }
          }
          commit_both(&empty[s]);
        }
        commit_both(&tfull[j & 1]);
      }
    }
  } else {
    const int quad = warp & 3, half = warp >> 2;
    constexpr int kChunks = BN / 64;  // of 32 columns, for each half of the columns
    int j = 0;
    for (int w = first; w < g.work; w += stride, ++j) {
      const Tile q = tile_of<BN>(g, w);
      const Item& t = *q.t;
      // (all warps go on or none: they meet at barriers below)
      ok = epi_all(mbar_wait(&tfull[j & 1], (j >> 1) & 1, &g_muon_error));
      if (!ok) break;
      tc_after();
      const uint32_t acc = tmem + (j & 1) * 256 + ((uint32_t)(quad * 32) << 16);
      const int row = q.m0 + (int)rank * 128 + quad * 32 + lane;
      const bool split = t.splits > 1;
      // this CTA's sums of a split, 16-byte pieces in the order that warps hold them
      auto place = [&](int k, int c) {
        return reinterpret_cast<float4*>(t.part) +
               (((((long long)k * t.tiles + q.index) * 2 + rank) * kEpiWarps + warp) * kChunks + c) * 256 + lane;
      };
      if (split) {
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          uint32_t r[32];
          tmem_ld32(acc + (half * kChunks + c) * 32, r);
          tmem_ld_wait();
          float4* to = place(q.split, c);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            __stcg(to + 32 * v, make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                            __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3])));
        }
        tc_before();
        __syncwarp();
        if (lane == 0) arrive_at(in_cta(smem_u32(&drained[j & 1]), 0));
        __threadfence();
        epi_barrier();
        if (threadIdx.x == 0) {
          unsigned int* count = t.count + q.index * 2 + rank;
          const unsigned int before = atomicAdd(count, 1u);
          if (before == (unsigned)t.splits - 1) *count = 0u;  // for the next launch
          __threadfence();
          *arrived = before;
        }
        epi_barrier();
        const bool last = *arrived == (unsigned)t.splits - 1;
        epi_barrier();  // (read by all before the next tile writes it)
        if (!last) continue;
        __threadfence();
      }
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        const int col0 = q.n0 + (half * kChunks + c) * 32;
        float f[32];
        if (split) {
#pragma unroll
          for (int v = 0; v < 32; ++v) f[v] = 0.f;
          for (int k = 0; k < t.splits; ++k) {
            const float4* from = place(k, c);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const float4 u = __ldcg(from + 32 * v);
              f[4 * v] += u.x, f[4 * v + 1] += u.y, f[4 * v + 2] += u.z, f[4 * v + 3] += u.w;
            }
          }
        } else {
          uint32_t r[32];
          tmem_ld32(acc + (half * kChunks + c) * 32, r);
          tmem_ld_wait();
          if (c == kChunks - 1) {
            tc_before();
            __syncwarp();
            if (lane == 0) arrive_at(in_cta(smem_u32(&drained[j & 1]), 0));
          }
#pragma unroll
          for (int v = 0; v < 32; ++v) f[v] = __uint_as_float(r[v]);
        }
        if (row < t.rows && col0 < t.cols) {
          const float unit = 1.f / kOrthoScale;
          const float own = g.which == 1 ? kOrthoB : kOrthoA, mul = g.which == 1 ? kOrthoC * unit : unit;
          const long long at = (long long)row * t.ld + col0;
          // eight columns at a time: lines are whole 16-byte pieces, what lies past the last column is of no meaning
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (col0 + 8 * v < t.cols) {
              float e[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) e[i] = f[8 * v + i] * mul;
              if (g.which) {
                const uint4 hi = __ldcg(reinterpret_cast<const uint4*>(t.add + at + 8 * v));
                const uint4 lo = __ldcg(reinterpret_cast<const uint4*>(t.add + t.low + at + 8 * v));
                const __half2* h2 = reinterpret_cast<const __half2*>(&hi);
                const __half2* l2 = reinterpret_cast<const __half2*>(&lo);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 a = __half22float2(h2[i]), b = __half22float2(l2[i]);
                  e[2 * i] += own * (a.x + b.x);
                  e[2 * i + 1] += own * (a.y + b.y);
                }
              }
              union {
                __half h[8];
                uint4 q;
              } hi, lo;
#pragma unroll
              for (int i = 0; i < 8; ++i) to_pair(e[i], &hi.h[i], &lo.h[i]);
              *reinterpret_cast<uint4*>(t.out + at + 8 * v) = hi.q;
              *reinterpret_cast<uint4*>(t.out + t.low + at + 8 * v) = lo.q;
              if (g.which != 2 && q.n0 + BN <= q.m0) {  // left of the diagonal block: the mirrored place, 32 rows side by side
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  __half* m = t.out + (long long)(col0 + 8 * v + i) * t.ld + row;
                  m[0] = hi.h[i];
                  m[t.low] = lo.h[i];
                }
              }
            }
          }
        }
        __syncwarp();  // together again for the next columns' read
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

// Tiles of a product of `rows` x `cols`.
int tiles_of(int which, int bn, int rows, int cols) {
  const int tiles_n = (cols + bn - 1) / bn;
  if (which == 2) return (rows + 255) / 256 * tiles_n;
  return bn == 256 ? lower_tiles<256>(rows, tiles_n) : lower_tiles<128>(rows, tiles_n);
}

// Splits of a gram's long side: by the matrix's own size (its result does not
// depend on the matrices beside it), over the pairs that its tiles leave idle,
// four blocks of 64 or more each.
int gram_splits(const MuonMat& t) {
  const int tiles = tiles_of(0, 128, t.side, t.side);
  const int nkb = (int)ceil_div_ll(t.tall ? t.rows : t.cols, kBK);
  int want = kPairs / tiles;
  if (want > nkb / 4) want = nkb / 4;
  if (want > kMuonSplits) want = kMuonSplits;
  return want < 1 ? 1 : want;
}

template <int BN, int CAP>
cudaError_t launch(const MuonGroup& m, int which, int from, cudaStream_t s) {
  Items<CAP> g;
  g.which = which;
  g.count = m.count;
  const int x_low = m.precision == DC_ORTHO_32;  // X's low part is used
  int work = 0;
  for (int i = 0; i < m.count; ++i) {
    const MuonMat& t = m.mat[i];
    Item& q = g.item[i];
    q.rows = which == 2 ? t.rows : t.side;
    q.cols = which == 2 ? t.cols : t.side;
    q.ld = which == 2 ? t.ld : t.lds;
    q.low = which == 2 ? muon_x_low(t) : muon_p_low(t);
    const int depth = which == 0 ? (t.tall ? t.rows : t.cols) : t.side;
    q.nkb = (depth + kBK - 1) / kBK;
    q.add = which == 1 ? t.gram : which == 2 ? t.x[from] : nullptr;
    q.out = which == 0 ? t.gram : which == 1 ? t.poly : t.x[1 - from];
    q.tiles_n = (q.cols + BN - 1) / BN;
    q.tiles = tiles_of(which, BN, q.rows, q.cols);
    q.a_low = which == 0 || (which == 2 && t.tall) ? x_low : 1;
    q.b_low = which == 0 || (which == 2 && !t.tall) ? x_low : 1;
    q.splits = which == 0 ? gram_splits(t) : 1;
    q.per_split = (int)ceil_div_ll(q.nkb, q.splits);
    q.splits = (int)ceil_div_ll(q.nkb, q.per_split);
    q.part = q.splits > 1 ? t.sums : nullptr;
    q.count = t.arrivals;
    q.start = work;
    work += q.tiles * q.splits;
    bool made = true;
    if (which == 0) {
      made = pair_map(&q.a, t.x[from], t.rows, t.cols, t.ld);
      q.b = q.a;
      q.a_mn = q.b_mn = t.tall;
    } else if (which == 1) {
      made = pair_map(&q.a, t.gram, t.side, t.side, t.lds);
      q.b = q.a;
      q.a_mn = q.b_mn = 0;
    } else {
      CUtensorMap x, p;
      made = pair_map(&x, t.x[from], t.rows, t.cols, t.ld) && pair_map(&p, t.poly, t.side, t.side, t.lds);
      q.a = t.tall ? x : p;
      q.b = t.tall ? p : x;
      q.a_mn = 0;
      q.b_mn = !t.tall;
    }
    if (!made) return cudaErrorInvalidValue;
  }
  g.work = work;
  cudaError_t e = cudaFuncSetAttribute(muon_mm<BN, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<BN>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(work < kPairs ? work : kPairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<BN>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, muon_mm<BN, CAP>, g);
  note_launches(1);
  return e;
}

}  // namespace

size_t muon_sums_bytes(const MuonMat& t) {
  const int splits = gram_splits(t);
  if (splits == 1) return 0;
  const size_t narrow = (size_t)tiles_of(0, 128, t.side, t.side) * 128, wide = (size_t)tiles_of(0, 256, t.side, t.side) * 256;
  return splits * (narrow > wide ? narrow : wide) * 256 * sizeof(float);
}

cudaError_t launch_muon_product(const MuonGroup& g, int which, int from, cudaStream_t s) {
  // tiles of 256 x 128 fill the pairs better, those of 256 x 256 read less of
  // shared memory for each product: wide ones where they are enough for two rounds
  long long wide = 0;
  for (int i = 0; i < g.count; ++i) {
    const MuonMat& t = g.mat[i];
    wide += tiles_of(which, 256, which == 2 ? t.rows : t.side, which == 2 ? t.cols : t.side);
  }
  const bool bn256 = wide >= 2 * kPairs;
  if (g.count <= 2) return bn256 ? launch<256, 2>(g, which, from, s) : launch<128, 2>(g, which, from, s);
  if (g.count <= 12) return bn256 ? launch<256, 12>(g, which, from, s) : launch<128, 12>(g, which, from, s);
  return bn256 ? launch<256, kMuonMats>(g, which, from, s) : launch<128, kMuonMats>(g, which, from, s);
}

// This file's share of dc_device_error (2 = unreadable).
unsigned int muon_read_error(int clear) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_muon_error, sizeof(v)) != cudaSuccess) return 2u;
  if (clear && cudaMemcpyToSymbol(g_muon_error, &zero, sizeof(zero)) != cudaSuccess) return 2u;
  return v;
}

}  // namespace dc
