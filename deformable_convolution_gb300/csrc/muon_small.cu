// Orthogonalisation and the Muon step of matrices with a short side of at most
// 64 (the offset convolutions' weights): everything in one launch.
//
// A matrix belongs to a cluster of eight CTAs, each of which keeps its share of
// the long side in shared memory, as pairs of 16-bit floats times 2^12, from
// the first step to the last.  A step: every CTA multiplies its share (R and X
// as in muon_products.cu, but on mma.sync: 18 rows fill a seventh of a tcgen05
// tile's 128), the CTAs add up their grams by rows through distributed shared
// memory, in order, and hand every sum to all; the polynomial (64 x 64 at most)
// is computed by each for itself, and X updated in place.  Two cluster barriers
// a step take the place of four waits through global memory: 18 x 2304 takes
// 36 us in place of 125.
//
// Products are high high + high low + low high whatever the precision: they are
// not what a step spends its time on.
#include "dc_tma.cuh"
#include "muon.cuh"
#include "muon_values.cuh"

namespace dc {
namespace {

constexpr int kThreads = 512, kWarps = 16, kCtas = 8;

// Layout of a CTA's shared memory, in bytes.
struct Small {
  int sp, nc;        // the short side up to a multiple of 16; the columns of X that the CTA keeps
  int xs, ps;        // row strides of X and of R and P in halves (an odd number of 16-byte pieces)
  int ks;            // splits of the CTA's columns over warps in the gram
  int x, part, r, p, diag, bytes;
};
__host__ __device__ inline Small small_of(int side, int length) {
  Small s;
  s.sp = (side + 15) / 16 * 16;
  s.nc = ((length + kCtas - 1) / kCtas + 15) / 16 * 16;
  s.xs = s.nc + 8;
  s.ps = s.sp + 8;
  s.ks = s.sp == 16 ? 16 : s.sp == 32 ? 4 : 1;
  s.x = 0;                                     // [2][sp][xs] halves
  s.part = s.x + 4 * s.sp * s.xs;              // [ks][sp][sp + 4] float
  s.r = s.part + s.ks * s.sp * (s.sp + 4) * 4; // [2][sp][ps] halves
  s.p = s.r + 4 * s.sp * s.ps;
  s.diag = s.p + 4 * s.sp * s.ps;              // [2][sp] float: of the gram and of the polynomial; [16] sums of squares
  s.bytes = s.diag + 8 * s.sp + 64;
  return s;
}
constexpr int kMaxBytes = 224 * 1024;

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_remote(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_remote(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t addr, __half2 v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(*reinterpret_cast<const uint32_t*>(&v)) : "memory");
}
__device__ __forceinline__ float2 ld_remote2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void ldm4(uint32_t* r, uint32_t addr) { px::ldmatrix_x4(r, addr); }
__device__ __forceinline__ void ldm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// acc[2][4] += rows m0 .. + 15 of `a` by rows n0 .. + 15 of `b` over columns k0
// .. + 15 (pairs: the low parts stand `alow`, `blow` bytes on).  main: high
// high; cross: the others.
__device__ __forceinline__ void unit16(float (*acc)[4], float (*cross)[4], uint32_t a, uint32_t alow, uint32_t b,
                                       uint32_t blow) {
  uint32_t ah[4], al[4], bh[4], bl[4];
  ldm4(ah, a);
  ldm4(al, a + alow);
  ldm4(bh, b);
  ldm4(bl, b + blow);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    mma(acc[n], ah, bh + 2 * n);
    mma(cross[n], ah, bl + 2 * n);
    mma(cross[n], al, bh + 2 * n);
  }
}

__global__ void __launch_bounds__(kThreads, 1) muon_small(const __grid_constant__ MuonGroup g) {
  extern __shared__ __align__(16) unsigned char smem[];
  pdl_wait();
  pdl_release();
  const MuonMat t = g.mat[blockIdx.x / kCtas];  // (a copy: registers, where the table would be read again after every store)
  float scale;
  if (skipped(g, &scale)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cta_rank();
  const int side = t.side, length = t.tall ? t.rows : t.cols;
  const Small L = small_of(side, length);
  const int j0 = (int)rank * L.nc, here = max(0, min(L.nc, length - j0));  // its share of the long side
  __half* xh = reinterpret_cast<__half*>(smem + L.x);
  __half* xl = xh + L.sp * L.xs;
  float* part = reinterpret_cast<float*>(smem + L.part);
  __half* rh = reinterpret_cast<__half*>(smem + L.r);
  __half* ph = reinterpret_cast<__half*>(smem + L.p);
  float* gd = reinterpret_cast<float*>(smem + L.diag);
  float* pd = gd + L.sp;
  float* squares = pd + L.sp;
  const uint32_t base = px::smem_u32(smem);
  // Passes over the share's values in the order that memory has them, kBatch of
  // a thread's loaded before the first is used: short index i, long index j of
  // the share and place of each, or a place of -1.
  constexpr int kBatch = 8;
  const int inner = t.tall ? side : here, total = side * here;
  const int next_o = inner ? kThreads / inner : 0, next_n = kThreads - next_o * inner;
  struct Walk {
    int e, o, n;
  };
  Walk walk;
  auto start = [&] {
    walk.e = tid;
    walk.o = inner ? tid / inner : 0;
    walk.n = tid - walk.o * inner;
  };
  auto batch = [&](int* x, long long* at) {  // x: the value's place in shared memory
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      at[k] = -1;
      if (walk.e < total) {
        const int i = t.tall ? walk.n : walk.o, j = t.tall ? walk.o : walk.n;
        x[k] = i * L.xs + j;
        at[k] = t.tall ? (long long)(j0 + j) * side + i : (long long)i * length + j0 + j;
      }
      walk.e += kThreads;
      walk.o += next_o;
      walk.n += next_n;
      if (walk.n >= inner) walk.n -= inner, ++walk.o;
    }
  };
  int xs[kBatch];
  long long at[kBatch];

  // the momentum's update and the norm
  float sum = 0.f;
  for (start(); walk.e < total;) {
    float v[kBatch], m[kBatch];
    batch(xs, at);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      v[k] = at[k] < 0 ? 0.f : load_in(t.in, t.in_dtype, at[k]);
      m[k] = at[k] < 0 || !g.update ? 0.f : t.m[at[k]];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (g.update) {
        m[k] = m[k] * g.momentum + v[k] * scale * g.rest;
        if (at[k] >= 0) t.m[at[k]] = m[k];
      }
      const float u = direction(g, scale, v[k], m[k]);
      sum += u * u;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) squares[warp] = sum;
  for (int e = tid; e < 2 * L.sp * L.xs / 8; e += kThreads) reinterpret_cast<uint4*>(smem + L.x)[e] = make_uint4(0, 0, 0, 0);
  cluster_sync();
  // every warp adds the CTAs' sums in one order
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps * kCtas / 32; ++k) {
    const int w = lane + 32 * k;
    sum += ld_remote(in_cta(base + L.diag + 8 * L.sp + 4 * (w % kWarps), w / kWarps));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float norm = sqrtf(sum);
  const float f = norm <= 3.402823466e38f ? kOrthoScale / (norm + kOrthoEps) : __uint_as_float(0x7fffffffu);
  for (start(); walk.e < total;) {
    float v[kBatch], m[kBatch];
    batch(xs, at);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      v[k] = at[k] < 0 ? 0.f : load_in(t.in, t.in_dtype, at[k]);
      m[k] = at[k] < 0 || !g.update ? 0.f : t.m[at[k]];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (at[k] >= 0) {
        const float u = direction(g, scale, v[k], m[k]) * f;
        const __half h = __float2half_rn(u);
        xh[xs[k]] = h;
        xl[xs[k]] = __float2half_rn(u - __half2float(h));
      }
  }
  __syncthreads();

  const float unit = 1.f / kOrthoScale;
  const float lr = g.lr_device ? *g.lr_device : g.lr;
  const int blocks = L.sp / 16;
  const uint32_t xlow = 2u * L.sp * L.xs, plow = 2u * L.sp * L.ps;
  // ldmatrix's lanes: rows of an A unit (two 8 x 8 down, two across), of a B unit
  // (two across, two down), and of one that is transposed as it is read
  const int a_row = lane & 15, a_col = (lane >> 4) * 8;
  const int b_row = (lane & 7) + (lane >> 4) * 8, b_col = (lane >> 3 & 1) * 8;
  const int t_row = (lane & 7) + (lane >> 3 & 1) * 8, t_col = (lane >> 4) * 8;
  const int acc_row = lane >> 2, acc_col = 2 * (lane & 3);

  for (int step = 0; step < g.steps; ++step) {
    // gram: units of 16 x 16 and, where these are few, parts of the columns, over the warps
    const int tasks = blocks * blocks * L.ks, depth = L.nc / 16;
    for (int q = warp; q < tasks; q += kWarps) {
      const int k = q / (blocks * blocks), un = q - k * blocks * blocks, bi = un / blocks, bj = un - bi * blocks;
      // every 16 columns' sums added up by float32 additions: an accumulator that is
      // truncated after each product loses half a unit in the last place each time
      float total[2][4] = {};
      const uint32_t a = base + L.x + 2u * ((16 * bi + a_row) * L.xs + a_col);
      const uint32_t b = base + L.x + 2u * ((16 * bj + b_row) * L.xs + b_col);
      for (int c = k; c < depth; c += L.ks) {
        float acc[2][4] = {}, cross[2][4] = {};
        unit16(acc, cross, a + 32 * c, xlow, b + 32 * c, xlow);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) total[n][e] += acc[n][e] + cross[n][e];
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          part[(k * L.sp + 16 * bi + acc_row + 8 * (e >> 1)) * (L.sp + 4) + 16 * bj + 8 * n + acc_col + (e & 1)] =
              total[n][e];
    }
    cluster_sync();
    // this CTA's rows of the sum, handed to all
    for (int e = tid; e < L.sp * L.sp / kCtas / 2; e += kThreads) {
      const int i = (int)rank * (L.sp / kCtas) + 2 * e / L.sp, j = 2 * e % L.sp;
      float v0 = 0.f, v1 = 0.f;
      for (int k = 0; k < L.ks; ++k) {
        const uint32_t from = base + L.part + 4u * ((k * L.sp + i) * (L.sp + 4) + j);
        float2 w[kCtas];
#pragma unroll
        for (int c = 0; c < kCtas; ++c) w[c] = ld_remote2(in_cta(from, c));
#pragma unroll
        for (int c = 0; c < kCtas; ++c) v0 += w[c].x, v1 += w[c].y;
      }
      v0 *= unit, v1 *= unit;
      const float d = (i == j ? v0 : v1) * unit;
      const bool on = i == j || i == j + 1;
      if (i == j) v0 = 0.f;
      if (i == j + 1) v1 = 0.f;
      const __half2 h = __floats2half2_rn(v0, v1);
      const float2 back = __half22float2(h);
      const __half2 l = __floats2half2_rn(v0 - back.x, v1 - back.y);
#pragma unroll
      for (int c = 0; c < kCtas; ++c) {
        const uint32_t to = in_cta(base, c);
        st_remote(to + L.r + 2u * (i * L.ps + j), h);
        st_remote(to + L.r + plow + 2u * (i * L.ps + j), l);
        if (on) st_remote(to + L.diag + 4u * i, d);
      }
    }
    cluster_sync();
    // P = b R + c (R R + (d_i + d_j) R), its diagonal apart
    for (int q = warp; q < blocks * blocks; q += kWarps) {
      const int bi = q / blocks, bj = q - bi * blocks;
      float acc[2][4] = {}, cross[2][4] = {};
      const uint32_t a = base + L.r + 2u * ((16 * bi + a_row) * L.ps + a_col);
      const uint32_t b = base + L.r + 2u * ((16 * bj + b_row) * L.ps + b_col);
      for (int c = 0; c < blocks; ++c) unit16(acc, cross, a + 32 * c, plow, b + 32 * c, plow);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = 16 * bi + acc_row + 8 * r, j = 16 * bj + 8 * n + acc_col, o = i * L.ps + j;
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(rh + o));
          const float2 l = __half22float2(*reinterpret_cast<const __half2*>(rh + L.sp * L.ps + o));
          const float di = gd[i];
          const float2 dj = *reinterpret_cast<const float2*>(gd + j);
          const float sq0 = (acc[n][2 * r] + cross[n][2 * r]) * unit, sq1 = (acc[n][2 * r + 1] + cross[n][2 * r + 1]) * unit;
          float v0 = kOrthoB * (h.x + l.x) + kOrthoC * (sq0 + (di + dj.x) * (h.x + l.x));
          float v1 = kOrthoB * (h.y + l.y) + kOrthoC * (sq1 + (di + dj.y) * (h.y + l.y));
          const float on = kOrthoB * di + kOrthoC * di * di;
          if (i == j) pd[i] = on + kOrthoC * sq0 * unit, v0 = 0.f;
          if (i == j + 1) pd[i] = on + kOrthoC * sq1 * unit, v1 = 0.f;
          const __half2 w = __floats2half2_rn(v0, v1);
          const float2 back = __half22float2(w);
          *reinterpret_cast<__half2*>(ph + o) = w;
          *reinterpret_cast<__half2*>(ph + L.sp * L.ps + o) = __floats2half2_rn(v0 - back.x, v1 - back.y);
        }
    }
    __syncthreads();
    // X = (a + e) X + P X, 16 columns at a time: a warp has read them all before it writes
    for (int cb = warp; cb < L.nc / 16; cb += kWarps) {
      if (16 * cb >= here) break;
      uint32_t bh[4][4], bl[4][4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < blocks) {
          const uint32_t at = base + L.x + 2u * ((16 * c + t_row) * L.xs + 16 * cb + t_col);
          ldm4t(bh[c], at);
          ldm4t(bl[c], at + xlow);
        }
      __syncwarp();
      for (int bi = 0; bi < blocks; ++bi) {
        float acc[2][4] = {}, cross[2][4] = {};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < blocks) {
            uint32_t ah[4], al[4];
            const uint32_t at = base + L.p + 2u * ((16 * bi + a_row) * L.ps + 16 * c + a_col);
            ldm4(ah, at);
            ldm4(al, at + plow);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              mma(acc[n], ah, bh[c] + 2 * n);
              mma(cross[n], ah, bl[c] + 2 * n);
              mma(cross[n], al, bh[c] + 2 * n);
            }
          }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int i = 16 * bi + acc_row + 8 * r, j = 16 * cb + 8 * n + acc_col;
            __half2* hp = reinterpret_cast<__half2*>(xh + i * L.xs + j);
            __half2* lp = reinterpret_cast<__half2*>(xl + i * L.xs + j);
            const float2 h = __half22float2(*hp), l = __half22float2(*lp);
            const float e = kOrthoA + pd[i];
            const float v0 = (acc[n][2 * r] + cross[n][2 * r]) * unit + e * (h.x + l.x);
            const float v1 = (acc[n][2 * r + 1] + cross[n][2 * r + 1]) * unit + e * (h.y + l.y);
            const __half2 w = __floats2half2_rn(v0, v1);
            const float2 back = __half22float2(w);
            *hp = w;
            *lp = __floats2half2_rn(v0 - back.x, v1 - back.y);
          }
      }
    }
    __syncthreads();
  }
  // the result, in the order that memory has it
  for (start(); walk.e < total;) {
    float p[kBatch];
    batch(xs, at);
    if (g.update) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        p[k] = at[k] < 0 ? 0.f : t.master ? t.master[at[k]] : load_in(t.param, t.out_dtype, at[k]);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (at[k] >= 0) {
        const float v = (__half2float(xh[xs[k]]) + __half2float(xl[xs[k]])) * unit;
        write_one(g, t, lr, at[k], p[k], v);
      }
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

}  // namespace

bool muon_is_small(int rows, int cols) {
  const int side = rows < cols ? rows : cols, length = rows < cols ? cols : rows;
  return side <= 64 && length <= (1 << 20) && small_of(side, length).bytes <= kMaxBytes;
}

cudaError_t launch_muon_small(const MuonGroup& g, cudaStream_t s) {
  int most = 0;
  for (int i = 0; i < g.count; ++i) {
    const MuonMat& t = g.mat[i];
    const int b = small_of(t.side, t.tall ? t.rows : t.cols).bytes;
    if (b > most) most = b;
  }
  cudaError_t e = cudaFuncSetAttribute(muon_small, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kCtas * g.count));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)most;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, muon_small, g);
  note_launches(1);
  return e;
}

}  // namespace dc
