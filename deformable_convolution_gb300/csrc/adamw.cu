// AdamW over many tensors in one launch, its 8-bit states, and the global
// gradient norm (no counterpart on the explainer page; the definitions are in
// the ABI header).
//
// The tensors' table travels as the kernel's argument, so a call needs no
// device memory and no copy of its own.  Blocks walk chunks of kChunk
// consecutive elements; a chunk lies in one tensor, and holds whole blocks of
// the 8-bit states, one to a warp.
//
// Every operation is rounded by itself (no contraction): an 8-bit code is a
// rounded number, and a last-bit difference ahead of it would show as a whole
// step of the code.
#include <float.h>

#include "dc_common.cuh"

namespace dc {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;  // elements of a thread
constexpr int kChunk = kThreads * kPer;
static_assert(kChunk / (kThreads / 32) == DC_STATE_BLOCK, "a warp holds one 8-bit block");

struct Entry {
  void* param;
  float* master;
  const void* grad;
  void *m, *v;
  float *m_scale, *v_scale;
  long long count;
  float decay;
  bool p16, g16, q8;
};
template <int N>
struct Table {
  int count;
  unsigned first[N + 1];  // chunks before each tensor
  Entry t[N];
};

// The tensor that holds chunk c: the last one with first <= c (a tensor
// without elements has no chunk).
template <typename TB>
__device__ __forceinline__ int find(const TB& tb, unsigned c) {
  int lo = 0, hi = tb.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tb.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float warp_max(float v) {
  // non-negative floats order as their bits do; NaN comes above infinity
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// A block's scale and its reciprocal, 0 and 0 for a block that counts as zero
// (the reciprocal alone is 0 where the scale is not finite).
__device__ __forceinline__ void block_scale(float top, float* scale, float* inv) {
  *scale = top < FLT_MIN ? 0.f : top;
  *inv = *scale > 0.f ? __frcp_rn(*scale) : 0.f;
}

__device__ __forceinline__ float decode_m(signed char q, float s) {
  const float t = __fmul_rn((float)q, 1.f / 127.f);
  return __fmul_rn(__fmul_rn(t, fabsf(t)), s);
}
__device__ __forceinline__ float decode_root(unsigned char q, float s) {
  const float t = __fmul_rn((float)q, 1.f / 255.f);
  return __fmul_rn(__fmul_rn(t, t), s);
}
__device__ __forceinline__ signed char encode_m(float m, float inv) {
  const int q = __float2int_rn(__fmul_rn(__fsqrt_rn(__fmul_rn(fabsf(m), inv)), 127.f));
  return (signed char)(m < 0.f ? -q : q);
}
__device__ __forceinline__ unsigned char encode_v(float v, float root, float inv) {
  const int q = __float2int_rn(__fmul_rn(__fsqrt_rn(__fmul_rn(root, inv)), 255.f));
  return (unsigned char)(v > 0.f && q < 1 && inv > 0.f ? 1 : q);
}

template <typename TB>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ TB tb, const __grid_constant__ AdamScalars h) {
  pdl_wait();
  const float gs = h.grad_scale ? *h.grad_scale : 1.f;
  float lr = h.lr, root2 = h.root2, step = h.step;
  if (h.schedule) {
    lr = h.schedule[0];
    step = __fdiv_rn(lr, h.schedule[1]);
    root2 = __frcp_rn(__fsqrt_rn(h.schedule[2]));
  }
  const unsigned chunks = tb.first[tb.count];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (isfinite(gs))
    for (unsigned c = blockIdx.x; c < chunks; c += gridDim.x) {
      const Entry& t = tb.t[find(tb, c)];
      const long long base =
          (long long)(c - tb.first[&t - tb.t]) * kChunk + warp * DC_STATE_BLOCK;
      const long long left = t.count - base;
      if (left <= 0) continue;
      const float keep = __fsub_rn(1.f, __fmul_rn(lr, t.decay));
      float p[kPer], g[kPer], m[kPer], r[kPer], v[kPer];
      const long long blk = base / DC_STATE_BLOCK;
      float ms = 0.f, vs = 0.f;
      if (t.q8) ms = t.m_scale[blk], vs = t.v_scale[blk];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const long long i = base + lane + 32 * k;
        p[k] = g[k] = m[k] = v[k] = 0.f;
        if (lane + 32 * k >= left) continue;
        g[k] = t.g16 ? to_f(static_cast<const __nv_bfloat16*>(t.grad)[i])
                     : static_cast<const float*>(t.grad)[i];
        p[k] = t.master ? t.master[i]
               : t.p16  ? to_f(static_cast<const __nv_bfloat16*>(t.param)[i])
                        : static_cast<const float*>(t.param)[i];
        if (t.q8) {
          m[k] = decode_m(static_cast<const signed char*>(t.m)[i], ms);
          v[k] = decode_root(static_cast<const unsigned char*>(t.v)[i], vs);
          v[k] = __fmul_rn(v[k], v[k]);
        } else {
          m[k] = static_cast<const float*>(t.m)[i];
          v[k] = static_cast<const float*>(t.v)[i];
        }
      }
      float mtop = 0.f, rtop = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (h.grad_scale) g[k] = __fmul_rn(g[k], gs);
        m[k] = __fadd_rn(__fmul_rn(m[k], h.b1), __fmul_rn(g[k], h.omb1));
        v[k] = __fadd_rn(__fmul_rn(v[k], h.b2), __fmul_rn(__fmul_rn(g[k], g[k]), h.omb2));
        r[k] = __fsqrt_rn(v[k]);
        const float u = __fdiv_rn(m[k], __fadd_rn(__fmul_rn(r[k], root2), h.eps));
        p[k] = __fsub_rn(__fmul_rn(p[k], keep), __fmul_rn(u, step));
        mtop = __uint_as_float(umax(__float_as_uint(mtop), __float_as_uint(fabsf(m[k]))));
        rtop = __uint_as_float(umax(__float_as_uint(rtop), __float_as_uint(r[k])));
      }
      float inv_m = 0.f, inv_v = 0.f;
      if (t.q8) {
        block_scale(warp_max(mtop), &ms, &inv_m);
        block_scale(warp_max(rtop), &vs, &inv_v);
        if (lane == 0) t.m_scale[blk] = ms, t.v_scale[blk] = vs;
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const long long i = base + lane + 32 * k;
        if (lane + 32 * k >= left) continue;
        if (t.master) t.master[i] = p[k];
        if (t.p16)
          static_cast<__nv_bfloat16*>(t.param)[i] = __float2bfloat16_rn(p[k]);
        else
          static_cast<float*>(t.param)[i] = p[k];
        if (t.q8) {
          static_cast<signed char*>(t.m)[i] = encode_m(m[k], inv_m);
          static_cast<unsigned char*>(t.v)[i] = encode_v(v[k], r[k], inv_v);
        } else {
          static_cast<float*>(t.m)[i] = m[k];
          static_cast<float*>(t.v)[i] = v[k];
        }
      }
    }
  pdl_release();
}

// The states as float32: Entry::param receives m, Entry::master v (either null).
template <typename TB>
__global__ void __launch_bounds__(kThreads) values_kernel(const __grid_constant__ TB tb) {
  pdl_wait();
  const unsigned chunks = tb.first[tb.count];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (unsigned c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Entry& t = tb.t[find(tb, c)];
    const long long base = (long long)(c - tb.first[&t - tb.t]) * kChunk + warp * DC_STATE_BLOCK;
    const long long blk = base / DC_STATE_BLOCK;
    const long long left = t.count - base;
    if (left <= 0) continue;
    float* mo = static_cast<float*>(t.param);
    float ms = 0.f, vs = 0.f;
    if (t.q8) ms = t.m_scale[blk], vs = t.v_scale[blk];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const long long i = base + lane + 32 * k;
      if (lane + 32 * k >= left) continue;
      if (t.q8) {
        const float root = decode_root(static_cast<const unsigned char*>(t.v)[i], vs);
        if (mo) mo[i] = decode_m(static_cast<const signed char*>(t.m)[i], ms);
        if (t.master) t.master[i] = __fmul_rn(root, root);
      } else {
        if (mo) mo[i] = static_cast<const float*>(t.m)[i];
        if (t.master) t.master[i] = static_cast<const float*>(t.v)[i];
      }
    }
  }
  pdl_release();
}

// Sum over the block in a fixed order, in thread 0.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float sm[32];
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = threadIdx.x < blockDim.x / 32 ? sm[threadIdx.x] : 0.f;
  if (threadIdx.x < 32)
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// part[block] = sum of squares of the block's chunks.
template <typename TB>
__global__ void __launch_bounds__(kThreads)
    squares_kernel(const __grid_constant__ TB tb, float* part) {
  pdl_wait();
  const unsigned chunks = tb.first[tb.count];
  float sum = 0.f;
  for (unsigned c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Entry& t = tb.t[find(tb, c)];
    const long long base = (long long)(c - tb.first[&t - tb.t]) * kChunk + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const long long i = base + kThreads * k;
      if (i >= t.count) continue;
      const float g = t.g16 ? to_f(static_cast<const __nv_bfloat16*>(t.grad)[i])
                            : static_cast<const float*>(t.grad)[i];
      sum = fmaf(g, g, sum);
    }
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
  pdl_release();
}

__global__ void __launch_bounds__(1024)
    grad_norm_kernel(const float* part, long long parts, float max_norm, float* norm,
                     float* scale) {
  pdl_wait();
  float sum = 0.f;
  for (long long i = threadIdx.x; i < parts; i += 1024) sum += part[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    const float n = sqrtf(sum);
    if (norm) *norm = n;
    if (scale) {
      const float r = isinf(max_norm) ? 1.f : max_norm / (n + 1e-6f);
      *scale = isfinite(n) ? fminf(r, 1.f) : __uint_as_float(0x7fc00000u);
    }
  }
  pdl_release();
}

int sm_count() {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

template <typename K, typename... A>
cudaError_t launch(K kern, unsigned grid, int threads, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  note_launches(1);
  return e;
}

// The tensors of one launch; false if their chunks do not fit in 32 bits.
template <int N>
bool fill(Table<N>* tb, const dc_adamw_tensor* t, int count) {
  unsigned long long at = 0;
  tb->count = count;
  for (int i = 0; i < count; ++i) {
    tb->first[i] = (unsigned)at;
    at += (unsigned long long)ceil_div_ll(t[i].count, kChunk);
    if (at > UINT_MAX) return false;
    tb->t[i] = Entry{t[i].param,   t[i].master,  t[i].grad,
                     t[i].m,       t[i].v,       t[i].m_scale,
                     t[i].v_scale, t[i].count,   t[i].weight_decay,
                     t[i].param_dtype == DC_BF16, t[i].grad_dtype == DC_BF16,
                     t[i].state == DC_STATE_Q8};
  }
  tb->first[count] = (unsigned)at;
  return true;
}

constexpr int kFew = 40;  // a table that fits in the first 4 KB of a launch's arguments

// f(table) with a table of the tensors, a small one where they are few.
template <typename F>
cudaError_t with_table(const dc_adamw_tensor* t, int count, F&& f) {
  if (count <= kFew) {
    Table<kFew> tb;
    return fill(&tb, t, count) ? f(tb) : cudaErrorInvalidValue;
  }
  Table<kAdamTensors> tb;
  return fill(&tb, t, count) ? f(tb) : cudaErrorInvalidValue;
}

unsigned grid_of(unsigned chunks, int per_sm) {
  const int sms = sm_count();
  const unsigned most = (unsigned)((sms ? sms : 1) * per_sm);
  return chunks < most ? chunks : most;
}

}  // namespace

cudaError_t launch_adamw(const dc_adamw_tensor* t, int count, const AdamScalars& h,
                         cudaStream_t s) {
  return with_table(t, count, [&](const auto& tb) {
    const unsigned grid = grid_of(tb.first[tb.count], 8);
    if (!grid) return cudaSuccess;
    return launch(adamw_kernel<std::decay_t<decltype(tb)>>, grid, kThreads, s, tb, h);
  });
}

cudaError_t launch_adamw_values(const dc_adamw_tensor* t, int count, float* const* m,
                                float* const* v, cudaStream_t s) {
  return with_table(t, count, [&](auto& tb) {
    for (int i = 0; i < count; ++i) {
      tb.t[i].param = m ? m[i] : nullptr;
      tb.t[i].master = v ? v[i] : nullptr;
    }
    const unsigned grid = grid_of(tb.first[tb.count], 8);
    if (!grid) return cudaSuccess;
    return launch(values_kernel<std::decay_t<decltype(tb)>>, grid, kThreads, s, tb);
  });
}

// part: kNormParts floats, all written.
cudaError_t launch_grad_squares(const dc_adamw_tensor* t, int count, float* part,
                                cudaStream_t s) {
  return with_table(t, count, [&](const auto& tb) {
    return launch(squares_kernel<std::decay_t<decltype(tb)>>, (unsigned)kNormParts, kThreads, s,
                  tb, part);
  });
}

cudaError_t launch_grad_norm(const float* part, long long parts, float max_norm, float* norm,
                             float* scale, cudaStream_t s) {
  return launch(grad_norm_kernel, 1u, 1024, s, part, parts, max_norm, norm, scale);
}

}  // namespace dc
