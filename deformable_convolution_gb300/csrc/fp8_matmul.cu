// Products of matrices in 8-bit floating point with block scales, on the
// 5th-generation tensor cores.
//
// D = A B^T with A = 2^ea a, B = 2^eb b in blocks of 128 values along k.  The
// scales are powers of two, which tcgen05's block-scaled form multiplies in as
// it reads the codes (kind::mxf8f6f4: an 8-bit exponent for each row and 32 of
// k; a block of 128 is four of its steps with one exponent).  So the whole
// reduction stays in one float32 accumulator: a float32 scale for each block
// would have to be multiplied in by CUDA cores every 128 of k, reading the
// accumulator out of tensor memory each time.
//
// The tensor cores cut the sum off after each product of 32, always towards zero:
// a sum of one sign over 2^20 of k came out 3e-3 too small in one accumulator.  So
// an accumulator runs over at most kRun blocks (256 products; 8192 of k: 5e-6 too
// small at most), and the runs of a longer reduction are added up in float32 in
// the workspace or D, by TMA reductions of one thread, one behind the other: their
// order, and so the result's bits, stay the same.  2048 x 2048 over 2^20: 4.8e-6 at
// most.  A run's end costs 2.5 us (2048 x 2048 over 33600: 90 us against 80 in one
// accumulator, which is 2.8e-5 too small; over 2^18: 626 against 556).
//
// CTAs work in pairs on tiles of 256 x BN (tc_pair.cuh).  The tensor cores read
// 128 rows of A and BN / 2 of B per SM from shared memory for 128 x BN results,
// at 256 x 256 as many bytes as shared memory gives in the time of the MMAs;
// one CTA alone (128 x 256) would need half as many again.
//
// Warps of each CTA: 0-7 read accumulators out of tensor memory and store them
// (two to a quarter of the lanes, each half of the columns), 8-11 copy scales
// into tensor memory, 12 issues TMA loads into a ring of stages, 13 (of the
// first CTA) issues the MMAs.  Persistent: pairs walk the tiles; a tile's
// results leave while the next one's MMAs run.  Tensor memory holds two
// accumulators: at BN = 256 they share 32 columns, which the first one's
// readers take first, so that 32 columns remain for scales.
#include <cuda.h>

#include "fp8.cuh"
#include "once.cuh"
#include "tc_pair.cuh"

namespace dc {

__device__ unsigned int g_fp8_error;  // raised by this file's bounded waits

namespace {

using namespace pair;

constexpr int kBK = 128;        // bytes of k in a stage: one scale block
constexpr int kEpiWarps = 8, kScaleWarps = 4;
constexpr int kWarpTma = kEpiWarps + kScaleWarps, kWarpMma = kWarpTma + 1;
constexpr int kThreads = (kWarpMma + 1) * 32;
constexpr int kPairs = 76;      // of 152 SMs
constexpr int kRun = DC_FP8_RUN / kBK;  // most blocks of an accumulator
constexpr int kStageBuf = 4096; // store staging of a warp: 32 rows of 128 bytes, or twice 32 of 64

template <int BN>
struct Cfg {
  static constexpr int kA = 128 * kBK, kB = BN / 2 * kBK, kStage = kA + kB;
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr int kAcc1 = BN == 256 ? 224 : BN;  // second accumulator's first column
  static constexpr int kShared = BN == 256 ? 32 : 0;  // columns that the two share
  static constexpr int kScaleCol = 480;               // two slots of 4 (A) + BN / 32 (B) columns
  static constexpr int kSlot = 16;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kEpiWarps * kStageBuf + 256;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Args {
  int m, n, sum, a_shared, b_shared;
  int nkb;                  // scale blocks along k
  int a_fmt, b_fmt;
  int tiles_m, tiles_n, splits, per_split;  // per_split: blocks of the reduction for one split
  int total;                // blocks of a tile's whole reduction
  int work;                 // tiles * splits (or batch)
  int m_first;              // tiles run down m first
  int add_runs;             // reductions have more than kRun blocks: the later runs are added to D
  int tma_out;              // D by TMA, else element by element
  int out_f32;
  int beside;               // what it reads was there before the product launched ahead of it
  const unsigned char* sa;
  const unsigned char* sb;
  void* d;                  // [batch or splits][m][ldd]
  long long ldd;
};

// The work item `w`: tile corner, matrix (or split) and its range of blocks.
struct Tile {
  int m0, n0, z, begin, end;
};
__device__ __forceinline__ Tile tile_of(const Args& a, int w, int bn) {
  Tile t;
  const int per = a.tiles_m * a.tiles_n;
  t.z = w / per;
  const int r = w - t.z * per;
  const int i = a.m_first ? r % a.tiles_m : r / a.tiles_n;
  const int j = a.m_first ? r / a.tiles_m : r % a.tiles_n;
  t.m0 = i * 256;
  t.n0 = j * bn;
  t.begin = a.splits > 1 ? t.z * a.per_split : 0;
  t.end = a.splits > 1 ? min(a.total, t.begin + a.per_split) : a.total;
  return t;
}

__device__ __forceinline__ void umma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                            uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}

template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_mm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
           const __grid_constant__ CUtensorMap td, const Args a) {
  using C = Cfg<BN>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = px::align1024(smem_raw);
  unsigned char* stg = smem + C::kStages * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + kEpiWarps * kStageBuf);
  uint64_t* empty = full + C::kStages;
  uint64_t* sfull = empty + C::kStages;  // scales of a slot are in tensor memory (both CTAs')
  uint64_t* sempty = sfull + 2;
  uint64_t* tfull = sempty + 2;          // accumulator b is complete
  uint64_t* drained = tfull + 2;         // the readers have taken accumulator b, or the columns that it shares
  uint32_t* holder = reinterpret_cast<uint32_t*>(drained + 2);

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
      mbar_init(&sfull[b], 2 * kScaleWarps);
      mbar_init(&sempty[b], 1);
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
  if (!a.beside) {
    pdl_wait();
    pdl_release();
  }

  if (warp == kWarpTma) {
    const bool issuer = elect_one();
    // both CTAs' copies count on the first one's barrier
    const uint32_t bar0 = in_cta(smem_u32(full), 0), ring = smem_u32(smem);
    int s = 0, round = 0;
    for (int w = first; w < a.work && ok; w += stride) {
      const Tile t = tile_of(a, w, BN);
      const int m0 = t.m0 + (int)rank * 128, n0 = t.n0 + (int)rank * (BN / 2);
      int img = a.sum ? t.begin / a.nkb : t.z, kb = a.sum ? t.begin - img * a.nkb : t.begin;
      for (int f = t.begin; f < t.end; ++f) {
        if (round && !warp_wait(&empty[s], (round - 1) & 1, &g_fp8_error)) {
          ok = false;
          break;
        }
        if (issuer) {
          if (rank == 0) mbar_expect_tx(&full[s], 2 * C::kStage);
          const uint32_t sa = ring + s * C::kStage, bar = bar0 + s * 8;
          tma_load(sa, &ta, bar, kb * kBK, m0, a.a_shared ? 0 : img);
          tma_load(sa + C::kA, &tb, bar, kb * kBK, n0, a.b_shared ? 0 : img);
        }
        __syncwarp();
        if (++kb == a.nkb) kb = 0, ++img;
        if (++s == C::kStages) s = 0, ++round;
      }
    }
    if (!ok) let_copies_land();
  } else if (warp == kWarpMma) {
    if (rank == 0) {
      const bool issuer = elect_one();
      const uint32_t idesc0 = ((uint32_t)a.a_fmt << 7) | ((uint32_t)a.b_fmt << 10) | ((uint32_t)(BN >> 3) << 17) |
                              (1u << 23) | ((256u >> 4) << 24);
      const uint64_t desc0 = sdesc(smem_u32(smem), 16, 1024);
      int s = 0, round = 0, slot = 0, j = 0;  // stages, scale slots and runs so far
      uint32_t acc = tmem;
      for (int w = first; w < a.work && ok; w += stride) {
        const Tile t = tile_of(a, w, BN);
        int kb = a.sum ? t.begin % a.nkb : t.begin;
        int left = 0;  // blocks of the run
        for (int f = t.begin; f < t.end; ++f, --left) {
          const bool begins = left == 0;
          if (begins) {
            left = min(kRun, t.end - f);
            // accumulators apart: the run before last has been read; sharing
            // columns: these have been read of the last one (and the one before whole)
            const int before = j - (C::kShared ? 1 : 2);
            if (before >= 0 && !warp_wait(&drained[before & 1], (before >> 1) & 1, &g_fp8_error)) {
              ok = false;
              break;
            }
            acc = tmem + (j & 1) * C::kAcc1;
          }
          if (f == t.begin || (kb & 3) == 0) {
            if (!warp_wait(&sfull[slot & 1], (slot >> 1) & 1, &g_fp8_error)) {
              ok = false;
              break;
            }
          }
          if (!warp_wait(&full[s], round & 1, &g_fp8_error)) {
            ok = false;
            break;
          }
          tc_after();
          const uint64_t da = desc0 + (uint64_t)(s * (C::kStage >> 4)), db = da + (C::kA >> 4);
          const uint32_t scale = tmem + C::kScaleCol + (slot & 1) * C::kSlot;
          // the byte of each scale word that holds this block's exponent
          const uint32_t idesc = idesc0 | ((uint32_t)(kb & 3) << 4) | ((uint32_t)(kb & 3) << 29);
          const bool chunk_end = f + 1 == t.end || (kb & 3) == 3 || kb + 1 == a.nkb;
          if (issuer) {
#pragma unroll
            for (int k = 0; k < kBK / 32; ++k)
              umma_scaled(acc, da + 2 * k, db + 2 * k, idesc, scale, scale + 4, (!begins || k > 0) ? 1u : 0u);
            commit_both(&empty[s]);
            if (chunk_end) commit_both(&sempty[slot & 1]);
            if (left == 1) commit_both(&tfull[j & 1]);
          }
          __syncwarp();
          j += left == 1;
          slot += chunk_end;
          if (++kb == a.nkb) kb = 0;
          if (++s == C::kStages) s = 0, ++round;
        }
      }
    }
  } else if (warp >= kEpiWarps) {
    // scales: a word holds the exponents of four blocks of one row; row r of a
    // tile sits in lane r % 32 of column r / 32, the same in every quarter
    const int kc = (a.nkb + 3) / 4, ra = (a.m + 127) / 128, rb = (a.n + 127) / 128;
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    int slot = 0;
    for (int w = first; w < a.work && ok; w += stride) {
      const Tile t = tile_of(a, w, BN);
      for (int f = t.begin; f < t.end && ok; ++slot) {
        const int img = a.sum ? f / a.nkb : t.z, kb = a.sum ? f - img * a.nkb : f;
        const int ta0 = t.m0 / 128 + (int)rank, tb0 = t.n0 / 128;
        const uint4 none = make_uint4(0, 0, 0, 0);
        auto word = [&](const unsigned char* p, int i, int rows, int r) {
          return r < rows ? __ldcg(reinterpret_cast<const uint4*>(p + (((long long)i * rows + r) * kc + kb / 4) * 512) + lane)
                          : none;
        };
        const uint4 va = word(a.sa, a.a_shared ? 0 : img, ra, ta0);
        uint4 vb[BN / 128];
#pragma unroll
        for (int h = 0; h < BN / 128; ++h) vb[h] = word(a.sb, a.b_shared ? 0 : img, rb, tb0 + h);
        if (slot >= 2) {
          ok = warp_wait(&sempty[slot & 1], ((slot >> 1) - 1) & 1, &g_fp8_error);
          if (!ok) break;
          tc_after();
        }
        const uint32_t to = tmem + quarter + C::kScaleCol + (slot & 1) * C::kSlot;
        tmem_st4(to, va);
#pragma unroll
        for (int h = 0; h < BN / 128; ++h) tmem_st4(to + 4 + 4 * h, vb[h]);
        tmem_st_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) arrive_at(in_cta(smem_u32(&sfull[slot & 1]), 0));
        f += min(min(4 - (kb & 3), a.nkb - kb), t.end - f);
      }
    }
  } else {
    // results: this warp's 32 rows, half of the columns
    const int quad = warp & 3, half = warp >> 2;
    unsigned char* buf = stg + warp * kStageBuf;
    int j = 0, used = 0;
    for (int w = first, from = 0; w < a.work; ++j) {
      const Tile t = tile_of(a, w, BN);
      const bool adds = a.add_runs && from > 0;  // to what this warp's runs before have left
      ok = warp_wait(&tfull[j & 1], (j >> 1) & 1, &g_fp8_error);
      if (!ok) break;
      tc_after();
      if (adds && lane == 0) store_wait_all();
      const uint32_t acc = tmem + (j & 1) * C::kAcc1 + ((uint32_t)(quad * 32) << 16);
      const int row0 = t.m0 + (int)rank * 128 + quad * 32;
      constexpr int kChunks = BN / 64;  // of 32 columns, for each half
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        // the columns shared with the next accumulator first: the last 32 of
        // the first accumulator, the first 32 of the second
        int chunk = half * kChunks + c;
        if (C::kShared && (j & 1) == 0) chunk = half ? 2 * kChunks - 1 - c : c;
        uint32_t r[32];
        tmem_ld32(acc + chunk * 32, r);
        tmem_ld_wait();
        if (c == (C::kShared ? 0 : kChunks - 1)) {
          tc_before();
          __syncwarp();
          if (lane == 0) arrive_at(in_cta(smem_u32(&drained[j & 1]), 0));
        }
        const int col0 = t.n0 + chunk * 32;
        if (row0 >= a.m || col0 >= a.n) continue;
        unsigned char* b = buf + (a.out_f32 || !a.tma_out ? 0 : (used++ & 1) * (kStageBuf / 2));
        if (a.tma_out) {
          if (lane == 0) {
            if (a.out_f32)
              store_wait_read<0>();
            else
              store_wait_read<1>();
          }
          __syncwarp();
          if (a.out_f32) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              *reinterpret_cast<uint4*>(b + lane * 128 + ((v ^ (lane & 7)) << 4)) =
                  make_uint4(r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t p[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(r[v * 8 + 2 * e]),
                                                               __uint_as_float(r[v * 8 + 2 * e + 1]));
                p[e] = *reinterpret_cast<const uint32_t*>(&h);
              }
              // 64-byte lines: the swizzle's address bits 4-5 by bits 7-8
              *reinterpret_cast<uint4*>(b + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(p[0], p[1], p[2], p[3]);
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            if (adds)
              tma_add(&td, smem_u32(b), col0, row0, t.z);
            else
              tma_store(&td, smem_u32(b), col0, row0, t.z);
            store_commit();
          }
        } else {
          // through shared memory, so that a warp's store covers one row's 32 columns
          float* f = reinterpret_cast<float*>(b);
#pragma unroll
          for (int v = 0; v < 32; ++v) f[lane * 32 + (v ^ lane)] = __uint_as_float(r[v]);
          __syncwarp();
          const long long base = ((long long)t.z * a.m + row0) * a.ldd + col0;
          const int rows = min(32, a.m - row0);
          if (col0 + lane < a.n)
            for (int i = 0; i < rows; ++i) {
              const float v = f[i * 32 + (lane ^ i)];
              if (a.out_f32)
                static_cast<float*>(a.d)[base + i * a.ldd + lane] = v;
              else
                static_cast<__nv_bfloat16*>(a.d)[base + i * a.ldd + lane] = __float2bfloat16_rn(v);
            }
          __syncwarp();
        }
      }
      // the tile's next run, or the next tile
      from = t.end - t.begin - from > kRun ? from + kRun : 0;
      if (from == 0) w += stride;
    }
    if (lane == 0) store_wait_all();
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers and tensor memory are no longer used
  tc_after();
  if (warp == 0) tmem_free(tmem);
  // what follows this launch also follows the one before it, and starts no earlier
  // than this one's wait (it is released by this one's end)
  if (a.beside) pdl_wait();
}

// D = the splits' sums, in order (rows: those of all matrices).
__global__ void __launch_bounds__(256)
    fp8_mm_sum(const float* __restrict__ part, int splits, long long rows, int n, long long ldd, void* d, int out_f32) {
  pdl_wait();
  pdl_release();
  const long long total = rows * ldd / 4, stride = rows * ldd;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    float4 s = __ldcg(reinterpret_cast<const float4*>(part) + i);
#pragma unroll 8
    for (int k = 1; k < splits; ++k) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(part + k * stride) + i);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const long long r = 4 * i / ldd;
    const int c = (int)(4 * i - r * ldd);
    const float e[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < n) {
        if (out_f32)
          static_cast<float*>(d)[r * n + c + q] = e[q];
        else
          static_cast<__nv_bfloat16*>(d)[r * n + c + q] = __float2bfloat16_rn(e[q]);
      }
  }
}

// ---------------------------------------------------------------- host side

struct Plan {
  int bn, tiles_m, tiles_n, splits, per_split, total;
  bool add_runs;  // a tile's (or split's) reduction has more than kRun blocks
  bool sums;      // float32 sums in the workspace, by splits or runs
  long long ldd;  // theirs, or D's
};

Plan plan_of(const dc_fp8_product& p) {
  Plan q;
  const int nkb = (int)ceil_div_ll(p.k, kBK);
  q.total = p.sum ? p.batch * nkb : nkb;
  q.tiles_m = (int)ceil_div_ll(p.m, 256);
  const int z = p.sum ? 1 : p.batch;
  // Wide tiles read less of shared memory for each product, narrow ones fill the
  // pairs better: wide ones for three rounds of tiles or more (268800 x 256 x 256:
  // 34.8 against 40.3 us), for one round of a long reduction, and for a sum,
  // whose splits fill the pairs (2048 x 512 over 16800: 19.6 against 23.7 us);
  // narrow ones else (8 times 256 x 3136 x 256: 6.4 against 7.0 us).
  const long long wide = q.tiles_m * ceil_div_ll(p.n, 256) * z;
  q.bn = p.n > 128 && (p.sum ? wide >= 8 : wide >= 3 * kPairs || (wide >= kPairs && nkb >= 8)) ? 256 : 128;
  q.tiles_n = (int)ceil_div_ll(p.n, q.bn);
  // few tiles of a long reduction: split it over the pairs, eight blocks of
  // k or more each (a sum over matrices only: its length grows with the batch)
  const long long tiles = (long long)q.tiles_m * q.tiles_n;
  q.splits = 1;
  q.per_split = q.total;
  if (p.sum && tiles * 2 <= kPairs && q.total >= 16) {
    long long want = kPairs / tiles;
    if (want > q.total / 8) want = q.total / 8;
    q.per_split = (int)ceil_div_ll(q.total, want);
    q.splits = (int)ceil_div_ll(q.total, q.per_split);
  }
  q.add_runs = q.per_split > kRun;
  q.sums = q.splits > 1 || q.add_runs;
  q.ldd = q.sums ? (p.n + 3) / 4 * 4 : p.n;
  return q;
}

template <int BN>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& td, const Args& a, cudaStream_t s) {
  static std::atomic<bool> allowed[kOnceDevices];
  cudaError_t e = allow_smem_once(fp8_mm<BN>, Cfg<BN>::kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(a.work < kPairs ? a.work : kPairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<BN>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fp8_mm<BN>, ta, tb, td, a);
  note_launches(1);
  return e;
}

}  // namespace

size_t fp8_matmul_workspace_bytes(const dc_fp8_product& p) {
  if (p.k == 0 || p.batch == 0) return 0;
  const Plan q = plan_of(p);
  return q.sums ? (size_t)(p.sum ? q.splits : p.batch) * p.m * q.ldd * sizeof(float) : 0;
}

cudaError_t launch_fp8_matmul(const Fp8Product& t, cudaStream_t s) {
  const dc_fp8_product& p = t.p;
  const Plan q = plan_of(p);
  Args a{};
  a.m = p.m;
  a.n = p.n;
  a.sum = p.sum;
  a.a_shared = p.a_shared;
  a.b_shared = p.b_shared;
  a.nkb = (int)ceil_div_ll(p.k, kBK);
  a.a_fmt = p.a_format;
  a.b_fmt = p.b_format;
  a.tiles_m = q.tiles_m;
  a.tiles_n = q.tiles_n;
  a.splits = q.splits;
  a.per_split = q.per_split;
  a.total = q.total;
  const int z = p.sum ? q.splits : p.batch;
  const long long work = (long long)q.tiles_m * q.tiles_n * z;
  if (work > INT_MAX) return cudaErrorInvalidValue;
  a.work = (int)work;
  a.beside = p.beside;
  a.m_first = q.tiles_m <= q.tiles_n;
  a.sa = static_cast<const unsigned char*>(t.a_scales);
  a.sb = static_cast<const unsigned char*>(t.b_scales);
  a.add_runs = q.add_runs;
  // runs of one split are added up in D itself where TMA can write it (2048 x 2048
  // over 33600: 90 us in place of 97; ldd is n then)
  const bool sums = q.sums && !(q.splits == 1 && p.out == DC_F32 && q.ldd == p.n && (uintptr_t)t.d % 16 == 0);
  a.out_f32 = p.out == DC_F32 || sums;
  a.d = sums ? t.ws : t.d;
  a.ldd = q.ldd;
  const int size = a.out_f32 ? 4 : 2;
  a.tma_out = a.ldd * size % 16 == 0 && (uintptr_t)a.d % 16 == 0;

  const unsigned long long ld = (unsigned long long)a.nkb * kBK;
  CUtensorMap ta, tb, td;
  auto codes = [&](CUtensorMap* m, const void* base, int rows, int shared, unsigned box) {
    const unsigned long long dims[3] = {ld, (unsigned long long)rows, (unsigned long long)(shared ? 1 : p.batch)};
    const unsigned long long strides[2] = {ld, ld * rows};
    const unsigned b[3] = {kBK, box, 1};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 3, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  bool made = codes(&ta, t.a, p.m, p.a_shared, 128) && codes(&tb, t.b, p.n, p.b_shared, (unsigned)q.bn / 2);
  if (a.tma_out) {
    const unsigned long long dims[3] = {(unsigned long long)p.n, (unsigned long long)p.m, (unsigned long long)z};
    const unsigned long long strides[2] = {(unsigned long long)(a.ldd * size), (unsigned long long)(a.ldd * size * p.m)};
    const unsigned b[3] = {32, 32, 1};
    made = made && make_tmap(&td, a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.d,
                             3, dims, strides, b, a.out_f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
  } else {
    td = ta;
  }
  if (!made) return cudaErrorInvalidValue;
  cudaError_t e = q.bn == 256 ? launch<256>(ta, tb, td, a, s) : launch<128>(ta, tb, td, a, s);
  if (e != cudaSuccess || !sums) return e;
  const long long rows = (long long)(p.sum ? 1 : p.batch) * p.m, blocks = ceil_div_ll(rows * q.ldd / 4, 256);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fp8_mm_sum, static_cast<const float*>(t.ws), q.splits, rows, p.n, q.ldd, t.d,
                         (int)(p.out == DC_F32));
  note_launches(1);
  return e;
}

// This file's share of dc_device_error (2 = unreadable).
unsigned int fp8_read_error(int clear) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_fp8_error, sizeof(v)) != cudaSuccess) return 2u;
  if (clear && cudaMemcpyToSymbol(g_fp8_error, &zero, sizeof(zero)) != cudaSuccess) return 2u;
  return v;
}

}  // namespace dc
