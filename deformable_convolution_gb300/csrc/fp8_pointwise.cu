// A pointwise layer's forward pass in one launch: y = W x over the channels of
// every pixel, x quantised on its way into shared memory.
//
// The result is dc_fp8_quantize's codes of x and dc_fp8_matmul's product, bit
// for bit, without the codes' way to memory and back: 1 + 1 of 2 + 1 + 1 + 2
// bytes a value of x and y at c_in = c_out.  A tile is 128 pixels by all output
// channels (at most 256, so that x is read once).  What bounds it is memory:
// channels last, 16 x 100 x 168 pixels of 256 -> 256 channels, 275 MB, take 57 us
// (71 % of the copy bandwidth) in place of a quantiser's and a product's 75.
// Channels first the codes are transposed on the way and y leaves in lines of 64
// bytes: 92 us (the two launches: 80).
//
// Warps: 0-7 and 8-15 take every other block of 128 channels of the tile's x
// into registers and write its codes where the tensor cores read them (the
// 128-byte swizzle), their scales into tensor memory beside the weight's (one
// group of eight warps with a block ahead in registers took 4 us a block,
// waiting for its own chains); 16-23 store the results; 24 loads the weight's
// codes by TMA; 25 issues the MMAs.
// Persistent, three stages of 128 channels, two accumulators (of 256 columns,
// sharing 64, which their readers take first).
#include <cuda.h>

#include "fp8_codes.cuh"
#include "once.cuh"
#include "tc_pair.cuh"

namespace dc {

__device__ unsigned int g_pointwise_error;  // raised by this file's bounded waits

namespace {

using pair::elect_one;
using pair::fence_proxy_async;
using pair::mbar_expect_tx;
using pair::mbar_init;
using pair::mbar_wait;
using pair::sdesc;
using pair::smem_u32;
using pair::store_commit;
using pair::store_wait_all;
using pair::store_wait_read;
using pair::tc_after;
using pair::tc_before;
using pair::tma_store;
using pair::tmem_ld32;
using pair::tmem_ld_wait;
using pair::tmem_st4;
using pair::tmem_st_wait;
using pair::warp_wait;

constexpr int kTile = 128, kStages = 3;
constexpr int kACodes = kTile * 128, kBCodes = 256 * 128, kStage = kACodes + kBCodes;
constexpr int kGroup = 8, kProducers = 2 * kGroup, kEpiWarps = 8;  // kGroup: warps that make a block's codes
constexpr int kWarpTma = kProducers + kEpiWarps, kWarpMma = kWarpTma + 1, kThreads = (kWarpMma + 1) * 32;
constexpr int kBuf = 2048;             // a warp's 32 pixels by 32 channels of results, twice
constexpr int kAcc1 = 192;             // the second accumulator's first column
constexpr int kScaleCol = 448;         // of each stage: 4 columns for x, 8 for the weight
constexpr int kTops = (kGroup + 1) * 128 * 4;  // a group's largest magnitudes by warp and column, and the columns' factors
constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kEpiWarps * 2 * kBuf + 2 * kTops + kStages * 128 + 256;
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Args {
  int images, pixels, c_in, c_out;  // pixels of an image (channels last: one image of all)
  int n;                            // c_out rounded up to 16: the MMAs' width
  int nkb, tiles;                   // blocks of 128 channels; tiles of an image
  int vectors, tma_out, even;       // x by 16-byte pieces; y by TMA (channels last) or by two pixels
  const __nv_bfloat16* x;
  const unsigned char* w_scales;
  __nv_bfloat16* y;
};

__device__ __forceinline__ void commit_one(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                     uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void group_meets(int group) { asm volatile("bar.sync %0, 256;" ::"r"(1 + group) : "memory"); }
// As that; whether `ok` holds for all.
__device__ __forceinline__ bool group_all(int group, bool ok) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, 256, p;\n selp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)ok), "r"(1 + group)
      : "memory");
  return r != 0;
}

// A thread's eight values turned so that the k-th comes first.
__device__ __forceinline__ void turn(Eight<__nv_bfloat16>& x, int k) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = k & 2 ? x.w[(i + 1) & 3] : x.w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = k & 4 ? a[(i + 2) & 3] : a[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) x.w[i] = k & 1 ? __funnelshift_r(b[i], b[(i + 1) & 3], 16) : b[i];
}

// LAST: x [pixel][channel], else [channel][pixel] of each image.
template <bool LAST>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_pointwise(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap ty, const Args a) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = px::align1024(smem_raw);
  unsigned char* stg = smem + kStages * kStage;
  unsigned char* tops = stg + kEpiWarps * 2 * kBuf;
  unsigned char* bytes = tops + 2 * kTops;  // [stage][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(bytes + kStages * 128);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* drained = tfull + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(drained + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int work = a.images * a.tiles;
  const bool shared_cols = a.n > kAcc1;  // the accumulators share columns

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(holder)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], kGroup + 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&drained[b], kEpiWarps);
    }
    px::fence_mbar_init();
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *holder;
  bool ok = true;
  pdl_wait();
  pdl_release();

  if (warp < kProducers) {
    // a thread's eight rows by eight columns of the block in memory: 8 h .. and
    // 8 l ..; rows are pixels and columns channels (LAST), or the other way round
    const int group = warp / kGroup, gw = warp % kGroup, gt = tid % (kGroup * 32);
    const int l = lane & 15, h = 2 * gw + (lane >> 4);
    uint32_t(*part)[128] = reinterpret_cast<uint32_t(*)[128]>(tops + group * kTops);
    float* inverse = reinterpret_cast<float*>(part + kGroup);
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    const int kc = (a.nkb + 3) / 4, atoms = (a.c_out + 127) / 128;
    Eight<__nv_bfloat16> v[8];
    // the group's blocks: its first, and every second one after it
    int w = blockIdx.x, kb = 0, block = 0;
    auto advance = [&](int by) {
      block += by;
      for (kb += by; kb >= a.nkb; kb -= a.nkb) w += gridDim.x;
    };
    auto load = [&] {
      if (w >= work) return;
      const int img = w / a.tiles, p0 = (w - img * a.tiles) * kTile, k0 = kb * 128;
      const int rows = LAST ? a.pixels - p0 : a.c_in - k0, cols = LAST ? a.c_in - k0 : a.pixels - p0;
      const long long ld = LAST ? a.c_in : a.pixels;
      const __nv_bfloat16* x = a.x + (long long)img * a.c_in * a.pixels + (LAST ? p0 * ld + k0 : k0 * ld + p0) +
                               8 * h * ld + 8 * l;
      const int left = min(8, cols - 8 * l);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int some = 8 * h + r < rows ? left : 0;
        if (a.vectors && some > 0)
          v[r].load(x + r * ld);
        else
          v[r].load_some(x + r * ld, some);
      }
    };
    advance(group);
    load();
    while (w < work) {
      {
        const int s = block % kStages, round = block / kStages;
        uint4 ws[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};  // the weight's scales
        if (gw >= 4)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (t < atoms) ws[t] = __ldcg(reinterpret_cast<const uint4*>(a.w_scales + ((long long)t * kc + kb / 4) * 512) + lane);
        unsigned char* codes = smem + s * kStage;
        unsigned char* sb = bytes + s * 128;
        const bool free = round == 0 || warp_wait(&empty[s], (round - 1) & 1, &g_pointwise_error);
        tc_after();  // (scales are written over those that finished MMAs read)
        if (LAST) {
          // (all warps of the group go on or none: they meet at the barrier below)
#pragma unroll
          for (int r = 0; r < 8; r += 2) {
            uint32_t two = scale_byte<DC_E4M3>(v[r].top()) | (scale_byte<DC_E4M3>(v[r + 1].top()) << 16);
#pragma unroll
            for (int o = 8; o; o >>= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, o));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t byte = q ? two >> 16 : two & 0xffffu;
              const float f = inverse_scale(byte);
              const Eight<__nv_bfloat16>& x = v[r + q];
              uint2 c;
              c.x = codes2<DC_E4M3>(x.get(0) * f, x.get(1) * f) | (codes2<DC_E4M3>(x.get(2) * f, x.get(3) * f) << 16);
              c.y = codes2<DC_E4M3>(x.get(4) * f, x.get(5) * f) | (codes2<DC_E4M3>(x.get(6) * f, x.get(7) * f) << 16);
              const int row = 8 * h + r + q;
              if (free) {
                *reinterpret_cast<uint2*>(codes + row * 128 + (((l >> 1) ^ (row & 7)) << 4) + (l & 1) * 8) = c;
                if (l == r + q) sb[row] = (unsigned char)byte;
              }
            }
          }
        } else {
          uint32_t top[8];
          column_tops<__nv_bfloat16>(v, top);
          if (lane < 16) {
            *reinterpret_cast<uint4*>(&part[gw][8 * l]) = make_uint4(top[0], top[1], top[2], top[3]);
            *reinterpret_cast<uint4*>(&part[gw][8 * l + 4]) = make_uint4(top[4], top[5], top[6], top[7]);
          }
          group_meets(group);
          if (gt < 128) {
            uint32_t most = 0u;
#pragma unroll
            for (int q = 0; q < kGroup; ++q) most = max(most, part[q][gt]);
            const uint32_t byte = scale_byte<DC_E4M3>(most);
            inverse[gt] = inverse_scale(byte);
            if (free) sb[gt] = (unsigned char)byte;
          }
          group_meets(group);
          // lanes start at pixels of their own, so that two of them and not 16 write to a bank
#pragma unroll
          for (int r = 0; r < 8; ++r) turn(v[r], l & 7);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int in = (i + l) & 7, row = 8 * l + in;  // the pixel; its channels 8 h ..
            const float f = inverse[row];
            uint2 c;
            c.x = codes2<DC_E4M3>(v[0].get(i) * f, v[1].get(i) * f) | (codes2<DC_E4M3>(v[2].get(i) * f, v[3].get(i) * f) << 16);
            c.y = codes2<DC_E4M3>(v[4].get(i) * f, v[5].get(i) * f) | (codes2<DC_E4M3>(v[6].get(i) * f, v[7].get(i) * f) << 16);
            if (free) *reinterpret_cast<uint2*>(codes + row * 128 + (((h >> 1) ^ in) << 4) + (h & 1) * 8) = c;
          }
        }
        advance(2);
        load();  // while this block's codes settle and the stage after it is waited for
        fence_proxy_async();
        ok = group_all(group, free);  // the block's scale bytes are there
        if (!ok) break;
        const uint32_t to = tmem + quarter + kScaleCol + s * 12;
        if (gw < 4) {
          // row r's exponent in lane r % 32 of column r / 32, in the lowest byte
          tmem_st4(to, make_uint4(sb[lane], sb[lane + 32], sb[lane + 64], sb[lane + 96]));
        } else {
          tmem_st4(to + 4, ws[0]);
          if (atoms > 1) tmem_st4(to + 8, ws[1]);
        }
        tmem_st_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) arrive(&full[s]);
      }
    }
  } else if (warp == kWarpTma) {
    const bool issuer = elect_one();
    int s = 0, round = 0;
    for (int w = blockIdx.x; w < work && ok; w += gridDim.x)
      for (int kb = 0; kb < a.nkb; ++kb) {
        if (round && !warp_wait(&empty[s], (round - 1) & 1, &g_pointwise_error)) {
          ok = false;
          break;
        }
        if (issuer) {
          mbar_expect_tx(&full[s], (uint32_t)a.n * 128);
          asm volatile(
              "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                  smem_u32(smem + s * kStage + kACodes)),
              "l"(&tw), "r"(smem_u32(&full[s])), "r"(kb * 128), "r"(0)
              : "memory");
        }
        __syncwarp();
        if (++s == kStages) s = 0, ++round;
      }
    if (!ok) pair::let_copies_land();
  } else if (warp == kWarpMma) {
    const bool issuer = elect_one();
    const uint32_t idesc0 = ((uint32_t)(a.n >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
    const uint64_t desc0 = sdesc(smem_u32(smem), 16, 1024);
    int s = 0, round = 0, j = 0;
    for (int w = blockIdx.x; w < work && ok; w += gridDim.x, ++j) {
      const int before = j - (shared_cols ? 1 : 2);
      if (before >= 0 && !warp_wait(&drained[before & 1], (before >> 1) & 1, &g_pointwise_error)) {
        ok = false;
        break;
      }
      const uint32_t acc = tmem + (j & 1) * kAcc1;
      for (int kb = 0; kb < a.nkb; ++kb) {
        if (!warp_wait(&full[s], round & 1, &g_pointwise_error)) {
          ok = false;
          break;
        }
        tc_after();
        const uint64_t da = desc0 + (uint64_t)(s * (kStage >> 4)), db = da + (kACodes >> 4);
        const uint32_t scale = tmem + kScaleCol + s * 12;
        if (issuer) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma(acc, da + 2 * k, db + 2 * k, idesc0 | ((uint32_t)(kb & 3) << 4), scale, scale + 4, (kb > 0 || k > 0) ? 1u : 0u);
          commit_one(&empty[s]);
          if (kb + 1 == a.nkb) commit_one(&tfull[j & 1]);
        }
        __syncwarp();
        if (++s == kStages) s = 0, ++round;
      }
    }
  } else {
    const int quad = warp & 3, half = (warp - kProducers) >> 2;
    unsigned char* bufs = stg + (warp - kProducers) * 2 * kBuf;
    int used = 0;
    const int all = (a.n + 31) / 32, mine = shared_cols ? 4 : half ? all / 2 : (all + 1) / 2;
    const int begin = half ? all - mine : 0;
    int j = 0;
    for (int w = blockIdx.x; w < work; w += gridDim.x, ++j) {
      const int img = w / a.tiles, p0 = (w - img * a.tiles) * kTile + quad * 32;
      ok = warp_wait(&tfull[j & 1], (j >> 1) & 1, &g_pointwise_error);
      if (!ok) break;
      tc_after();
      const uint32_t acc = tmem + (j & 1) * kAcc1 + ((uint32_t)(quad * 32) << 16);
      const int px = p0 + lane;
      if (mine == 0 && lane == 0) arrive(&drained[j & 1]);
#pragma unroll 1
      for (int c = 0; c < mine; ++c) {
        // the columns shared with the next accumulator first: the last 64 of the
        // first accumulator, the first 64 of the second
        const int chunk = begin + (shared_cols && half && (j & 1) == 0 ? mine - 1 - c : c);
        uint32_t r[32];
        tmem_ld32(acc + chunk * 32, r);
        tmem_ld_wait();
        if (c == (shared_cols ? 1 : mine - 1)) {
          tc_before();
          __syncwarp();
          if (lane == 0) arrive(&drained[j & 1]);
        }
        const int c0 = chunk * 32;
        if (p0 >= a.pixels || c0 >= a.c_out) continue;
        uint32_t two[16];
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[2 * v]), __uint_as_float(r[2 * v + 1]));
          two[v] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if (LAST && a.tma_out) {
          unsigned char* buf = bufs + (used++ & 1) * kBuf;
          if (lane == 0) store_wait_read<1>();
          __syncwarp();
#pragma unroll
          for (int v = 0; v < 4; ++v)
            *reinterpret_cast<uint4*>(buf + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(two[4 * v], two[4 * v + 1], two[4 * v + 2], two[4 * v + 3]);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            tma_store(&ty, smem_u32(buf), c0, p0, 0);
            store_commit();
          }
        } else if (LAST) {
          if (px < a.pixels) {
            __nv_bfloat16* y = a.y + (long long)px * a.c_out + c0;
#pragma unroll
            for (int v = 0; v < 32; ++v)
              if (c0 + v < a.c_out) reinterpret_cast<unsigned short*>(y)[v] = (unsigned short)(v & 1 ? two[v >> 1] >> 16 : two[v >> 1]);
          }
        } else {
          // lanes are pixels: neighbours exchange, so that each stores two pixels of one channel
          __nv_bfloat16* y = a.y + ((long long)img * a.c_out + c0) * a.pixels;
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            if (a.even) {
              const uint32_t other = __shfl_xor_sync(0xffffffffu, two[v], 1);
              const uint32_t out = lane & 1 ? __byte_perm(other, two[v], 0x7632) : __byte_perm(two[v], other, 0x5410);
              const int ch = 2 * v + (lane & 1), at = px & ~1;
              if (at < a.pixels && c0 + ch < a.c_out) *reinterpret_cast<uint32_t*>(y + (long long)ch * a.pixels + at) = out;
            } else if (px < a.pixels) {
#pragma unroll
              for (int q = 0; q < 2; ++q)
                if (c0 + 2 * v + q < a.c_out)
                  reinterpret_cast<unsigned short*>(y)[(long long)(2 * v + q) * a.pixels + px] =
                      (unsigned short)(q ? two[v] >> 16 : two[v]);
            }
          }
        }
      }
    }
    if (lane == 0) store_wait_all();
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <bool LAST>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& ty, const Args& a, cudaStream_t s) {
  static std::atomic<bool> allowed[kOnceDevices];
  cudaError_t e = allow_smem_once(fp8_pointwise<LAST>, kSmem, allowed);
  if (e != cudaSuccess) return e;
  const long long work = (long long)a.images * a.tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(work < 152 ? work : 152));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, fp8_pointwise<LAST>, tw, ty, a);
  note_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_fp8_pointwise(const Fp8Pointwise& t, cudaStream_t s) {
  const dc_fp8_layer& p = t.p;
  const bool last = p.layout == DC_NHWC;
  Args a{};
  a.images = last ? 1 : p.n;
  a.pixels = last ? p.n * p.pixels : p.pixels;
  a.c_in = p.c_in;
  a.c_out = p.c_out;
  a.n = (p.c_out + 15) / 16 * 16;
  a.nkb = (p.c_in + 127) / 128;
  a.tiles = (a.pixels + kTile - 1) / kTile;
  a.vectors = (last ? p.c_in : a.pixels) % 8 == 0 && (uintptr_t)t.x % 16 == 0;
  a.tma_out = last && p.c_out % 8 == 0 && (uintptr_t)t.y % 16 == 0;
  a.even = a.pixels % 2 == 0 && (uintptr_t)t.y % 4 == 0;
  a.x = static_cast<const __nv_bfloat16*>(t.x);
  a.w_scales = static_cast<const unsigned char*>(t.w_scales);
  a.y = static_cast<__nv_bfloat16*>(t.y);
  CUtensorMap tw, ty;
  const unsigned long long ld = (unsigned long long)a.nkb * 128;
  const unsigned long long wd[2] = {ld, (unsigned long long)p.c_out}, wst[1] = {ld};
  const unsigned wbox[2] = {128, (unsigned)a.n};
  bool made = make_tmap(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, t.w_codes, 2, wd, wst, wbox, CU_TENSOR_MAP_SWIZZLE_128B);
  ty = tw;
  if (a.tma_out) {
    const unsigned long long row = 2ull * p.c_out;
    const unsigned long long yd[3] = {(unsigned long long)p.c_out, (unsigned long long)a.pixels, 1}, yst[2] = {row, row * a.pixels};
    const unsigned ybox[3] = {32, 32, 1};
    made = made && make_tmap(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, t.y, 3, yd, yst, ybox, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  if (!made) return cudaErrorInvalidValue;
  return last ? launch<true>(tw, ty, a, s) : launch<false>(tw, ty, a, s);
}

// This file's share of dc_device_error (2 = unreadable).
unsigned int pointwise_read_error(int clear) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_pointwise_error, sizeof(v)) != cudaSuccess) return 2u;
  if (clear && cudaMemcpyToSymbol(g_pointwise_error, &zero, sizeof(zero)) != cudaSuccess) return 2u;
  return v;
}

}  // namespace dc
