// AdamW over many tensors in one launch, its 8-bit states, and the global
// gradient norm (no counterpart on the explainer page; the definitions are in
// the ABI header).
//
// The tensors' table travels as the kernel's argument, so a call needs no
// device memory and no copy of its own.  Blocks walk chunks of kChunk
// consecutive elements; a chunk lies in one tensor, and holds whole blocks of
// the 8-bit states, one to a warp.
//
// Every operation ahead of an 8-bit code is rounded by itself (no contraction):
// a code is a rounded number, and a last-bit difference ahead of it would show
// as a whole step.
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
  unsigned char lead;  // elements by which the first chunk starts ahead of the tensor
  bool vec;            // runs of four elements from `lead` ahead are aligned in every array
  bool p16, g16, q8;
};
template <int N>
struct Table {
  int count;
  unsigned first[N + 1];  // chunks before each tensor
  Entry t[N];
};

// The tensor that holds chunk c: the last one with first <= c (a tensor
// without elements has no chunk).  (A search by the whole warp at once, each
// lane at its own entries, measured up to five times slower: the table lies in
// the arguments, where a warp's lanes are served one after the other.)
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

// Codes to floats and back without the conversion instructions (a sixteenth of
// the multiplier's rate): a small integer added to 1.5 * 2^23 sits in the low
// bits of the sum, rounded to nearest even by the addition itself.
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
// byte e of a word of four codes, as the float 1.5 * 2^23 + byte (for signed
// codes the word's bytes come with their top bits flipped, 128 more)
__device__ __forceinline__ float code_bits(uint32_t w, int e) {
  return __uint_as_float(__byte_perm(w, 0x4b400000u, 0x7650 | e));
}

__device__ __forceinline__ float decode_m(float q, float s) {
  const float t = __fmul_rn(q, 1.f / 127.f);
  return __fmul_rn(__fmul_rn(t, fabsf(t)), s);
}
__device__ __forceinline__ float decode_root(float q, float s) {
  const float t = __fmul_rn(q, 1.f / 255.f);
  return __fmul_rn(__fmul_rn(t, t), s);
}
// The codes before rounding, from the root of m (or of r = sqrt(v)) over s.
__device__ __forceinline__ float level_m(float root, float m) {
  return copysignf(__fmul_rn(root, 127.f), m);
}
// At least `low` (1, or 0 in a block that counts as zero) where r > 0: a root
// of a float32 is 0 or at least 2^-75.
__device__ __forceinline__ float level_v(float root, float r, float low) {
  return fmaxf(__fmul_rn(root, 255.f), fminf(r * 0x1p127f, low));
}

// Two floats in one instruction.  A product that goes into a packed sum may be
// contracted with it: where that would matter the sum is taken apart.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 ra, rb, rd;\n mov.b64 ra, {%2,%3};\n mov.b64 rb, {%4,%5};\n"
      " mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0,%1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 ra, rb, rd;\n mov.b64 ra, {%2,%3};\n mov.b64 rb, {%4,%5};\n"
      " add.rn.f32x2 rd, ra, rb;\n mov.b64 {%0,%1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2,%3};\n mov.b64 rb, {%4,%5};\n"
      " mov.b64 rc, {%6,%7};\n fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0,%1}, rd;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// One instruction each; a subnormal argument counts as 0.
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- element access
// A lane's eight elements of a warp's block of 256: two runs of four
// consecutive ones (VEC: every array 16-byte aligned for float, 8 for bf16,
// 4 for codes), or every 32nd one.  A warp's access is whole 128-byte lines
// either way; the runs take a quarter of the instructions.

template <bool VEC>
__device__ __forceinline__ int place(int lane, int k) {
  return VEC ? (k >> 2) * 128 + lane * 4 + (k & 3) : lane + 32 * k;
}

template <bool VEC>
__device__ __forceinline__ void load8(const float* p, int lane, float* f) {
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = *reinterpret_cast<const float4*>(p + h * 128 + lane * 4);
      f[4 * h] = v.x, f[4 * h + 1] = v.y, f[4 * h + 2] = v.z, f[4 * h + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) f[k] = p[lane + 32 * k];
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int lane, float* f) {
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint2 v = *reinterpret_cast<const uint2*>(p + h * 128 + lane * 4);
      f[4 * h] = __uint_as_float(v.x << 16), f[4 * h + 1] = __uint_as_float(v.x & 0xffff0000u);
      f[4 * h + 2] = __uint_as_float(v.y << 16), f[4 * h + 3] = __uint_as_float(v.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) f[k] = to_f(p[lane + 32 * k]);
  }
}
// codes: four to a word
template <bool VEC>
__device__ __forceinline__ void load8(const unsigned char* p, int lane, uint32_t* w) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (VEC) {
      w[h] = *reinterpret_cast<const uint32_t*>(p + h * 128 + lane * 4);
    } else {
      w[h] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[h] |= (uint32_t)p[lane + 32 * (4 * h + e)] << (8 * e);
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(float* p, int lane, const float* f) {
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float4*>(p + h * 128 + lane * 4) =
          make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) p[lane + 32 * k] = f[k];
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int lane, const float* f) {
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(f[4 * h], f[4 * h + 1]);
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[4 * h + 2], f[4 * h + 3]);
      *reinterpret_cast<uint2*>(p + h * 128 + lane * 4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) p[lane + 32 * k] = __float2bfloat16_rn(f[k]);
  }
}
// codes in the low bytes of q
template <bool VEC>
__device__ __forceinline__ void store8(unsigned char* p, int lane, const uint32_t* q) {
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint32_t*>(p + h * 128 + lane * 4) =
          __byte_perm(__byte_perm(q[4 * h], q[4 * h + 1], 0x0040),
                      __byte_perm(q[4 * h + 2], q[4 * h + 3], 0x0040), 0x5410);
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) p[lane + 32 * k] = (unsigned char)q[k];
  }
}

// ---------------------------------------------------------------- the step

// The step's numbers, read once by each thread (gs and the schedule's from
// device memory).
struct Step {
  float gs, lr, root2, step;
};
__device__ __forceinline__ Step make_step(const AdamScalars& h) {
  Step st{1.f, h.lr, h.root2, h.step};
  if (h.grad_scale) st.gs = *h.grad_scale;
  if (h.schedule) {
    st.lr = h.schedule[0];
    st.step = __fdiv_rn(st.lr, h.schedule[1]);
    st.root2 = __frcp_rn(__fsqrt_rn(h.schedule[2]));
  }
  return st;
}

// Two elements: p, m, v in, out with r = sqrt(v).  The quotient (2 units in
// the last place) and the sum it goes into feed no code and need not be
// separately rounded ones.
__device__ __forceinline__ void update2(const AdamScalars& h, const Step& st, float keep, float2 g,
                                        float2& p, float2& m, float2& v, float2& r) {
  g = mul2(g, both(st.gs));
  const float2 mo = mul2(m, both(h.b1)), mg = mul2(g, both(h.omb1));
  const float2 vo = mul2(v, both(h.b2)), vg = mul2(mul2(g, g), both(h.omb2));
  m = make_float2(__fadd_rn(mo.x, mg.x), __fadd_rn(mo.y, mg.y));
  v = make_float2(__fadd_rn(vo.x, vg.x), __fadd_rn(vo.y, vg.y));
  r = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 d = add2(mul2(r, both(st.root2)), both(h.eps));
  const float2 u = mul2(m, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
  p = fma2(u, both(-st.step), mul2(p, both(keep)));
}

__device__ __forceinline__ float abs_max(float a, float b, float c) {  // NaN stays
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}

// The block's new scales (stored by lane 0) and their reciprocals.
__device__ __forceinline__ void new_scales(const Entry& t, long long blk, int lane,
                                           const float* m, const float* r, float* inv_m,
                                           float* inv_v) {
  float mt = 0.f, rt = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; k += 2) {
    mt = abs_max(mt, m[k], m[k + 1]);
    rt = abs_max(rt, r[k], r[k + 1]);
  }
  float ms, vs;
  block_scale(warp_max(mt), &ms, inv_m);
  block_scale(warp_max(rt), &vs, inv_v);
  if (lane == 0) t.m_scale[blk] = ms, t.v_scale[blk] = vs;
}

__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN is passed over
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A lane's codes, exactly the rounded ones: levels from the approximate
// root decide (its error is below 2^-22 of at most 255), unless one of the
// lane's is within 2.5e-4 of half way between two codes.
__device__ __forceinline__ void encode8(const float* m, const float* r, float inv_m, float inv_v,
                                        uint32_t* qm, uint32_t* qv) {
  const float low = inv_v > 0.f ? 1.f : 0.f;
  float off = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; k += 2) {
    const float2 am = mul2(make_float2(m[k], m[k + 1]), both(inv_m));
    const float2 av = mul2(make_float2(r[k], r[k + 1]), both(inv_v));
    const float2 lm = make_float2(level_m(sqrt_approx(fabsf(am.x)), m[k]),
                                  level_m(sqrt_approx(fabsf(am.y)), m[k + 1]));
    const float2 lv = make_float2(level_v(sqrt_approx(av.x), r[k], low),
                                  level_v(sqrt_approx(av.y), r[k + 1], low));
    const float2 cm = add2(lm, both(kMagic)), cv = add2(lv, both(kMagic));
    const float2 dm = fma2(both(-1.f), add2(cm, both(-kMagic)), lm);
    const float2 dv = fma2(both(-1.f), add2(cv, both(-kMagic)), lv);
    off = max3(off, fabsf(dm.x), fabsf(dm.y));
    off = max3(off, fabsf(dv.x), fabsf(dv.y));
    qm[k] = __float_as_uint(cm.x), qm[k + 1] = __float_as_uint(cm.y);
    qv[k] = __float_as_uint(cv.x), qv[k + 1] = __float_as_uint(cv.y);
  }
  if (off > 0.5f - 2.5e-4f) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const float lm = level_m(__fsqrt_rn(__fmul_rn(fabsf(m[k]), inv_m)), m[k]);
      const float lv = level_v(__fsqrt_rn(__fmul_rn(r[k], inv_v)), r[k], low);
      qm[k] = __float_as_uint(__fadd_rn(lm, kMagic));
      qv[k] = __float_as_uint(__fadd_rn(lv, kMagic));
    }
  }
}

// decode: the lane's m and v from its two words of codes each.
__device__ __forceinline__ void decode8(const uint32_t* cm, const uint32_t* cv, float ms, float vs,
                                        float* m, float* v) {
#pragma unroll
  for (int k = 0; k < kPer; k += 2) {
    const uint32_t wm = cm[k >> 2] ^ 0x80808080u, wv = cv[k >> 2];
    const int e = k & 3;
    float2 t = mul2(add2(make_float2(code_bits(wm, e), code_bits(wm, e + 1)), both(-(kMagic + 128.f))),
                    both(1.f / 127.f));
    t = mul2(make_float2(__fmul_rn(t.x, fabsf(t.x)), __fmul_rn(t.y, fabsf(t.y))), both(ms));
    m[k] = t.x, m[k + 1] = t.y;
    t = mul2(add2(make_float2(code_bits(wv, e), code_bits(wv, e + 1)), both(-kMagic)),
             both(1.f / 255.f));
    t = mul2(mul2(t, t), both(vs));
    t = mul2(t, t);
    v[k] = t.x, v[k + 1] = t.y;
  }
}

// A whole block of 256 elements from `base`.  PARAM: 0 float, 1 bf16 with a
// master, 2 bf16 alone.
template <int PARAM, bool G16, bool Q8, bool VEC>
__device__ __forceinline__ void whole_block(const Entry& t, long long base, int lane,
                                            const AdamScalars& h, const Step& st) {
  float p[kPer], g[kPer], m[kPer], v[kPer], r[kPer];
  uint32_t cm[2], cv[2];
  const long long blk = base / DC_STATE_BLOCK;
  float ms = 0.f, vs = 0.f;
  if (G16)
    load8<VEC>(static_cast<const __nv_bfloat16*>(t.grad) + base, lane, g);
  else
    load8<VEC>(static_cast<const float*>(t.grad) + base, lane, g);
  if (Q8) {
    load8<VEC>(static_cast<const unsigned char*>(t.m) + base, lane, cm);
    load8<VEC>(static_cast<const unsigned char*>(t.v) + base, lane, cv);
    ms = t.m_scale[blk], vs = t.v_scale[blk];
  } else {
    load8<VEC>(static_cast<const float*>(t.m) + base, lane, m);
    load8<VEC>(static_cast<const float*>(t.v) + base, lane, v);
  }
  if (PARAM == 1)
    load8<VEC>(t.master + base, lane, p);
  else if (PARAM == 2)
    load8<VEC>(static_cast<const __nv_bfloat16*>(t.param) + base, lane, p);
  else
    load8<VEC>(static_cast<const float*>(t.param) + base, lane, p);
  if (!isfinite(st.gs)) return;
  const float keep = __fsub_rn(1.f, __fmul_rn(st.lr, t.decay));
  if (Q8) decode8(cm, cv, ms, vs, m, v);
#pragma unroll
  for (int k = 0; k < kPer; k += 2) {
    float2 p2 = make_float2(p[k], p[k + 1]), m2 = make_float2(m[k], m[k + 1]);
    float2 v2 = make_float2(v[k], v[k + 1]), r2;
    update2(h, st, keep, make_float2(g[k], g[k + 1]), p2, m2, v2, r2);
    p[k] = p2.x, p[k + 1] = p2.y, m[k] = m2.x, m[k + 1] = m2.y;
    v[k] = v2.x, v[k + 1] = v2.y, r[k] = r2.x, r[k + 1] = r2.y;
  }
  if (PARAM == 0)
    store8<VEC>(static_cast<float*>(t.param) + base, lane, p);
  else
    store8<VEC>(static_cast<__nv_bfloat16*>(t.param) + base, lane, p);
  if (PARAM == 1) store8<VEC>(t.master + base, lane, p);
  if (Q8) {
    float inv_m, inv_v;
    new_scales(t, blk, lane, m, r, &inv_m, &inv_v);
    uint32_t qm[kPer], qv[kPer];
    encode8(m, r, inv_m, inv_v, qm, qv);
    store8<VEC>(static_cast<unsigned char*>(t.m) + base, lane, qm);
    store8<VEC>(static_cast<unsigned char*>(t.v) + base, lane, qv);
  } else {
    store8<VEC>(static_cast<float*>(t.m) + base, lane, m);
    store8<VEC>(static_cast<float*>(t.v) + base, lane, v);
  }
}

// A block that hangs over an end of its tensor (base < 0 where the tensor's
// start is not on the vectors' grid), any kind.
__device__ __noinline__ void part_block(const Entry& t, long long base, int lane,
                                        const AdamScalars& h, const Step& st) {
  if (!isfinite(st.gs)) return;
  const long long blk = base / DC_STATE_BLOCK;
  float ms = 0.f, vs = 0.f, m[kPer], r[kPer], v[kPer];
  if (t.q8) ms = t.m_scale[blk], vs = t.v_scale[blk];
  const float keep = __fsub_rn(1.f, __fmul_rn(st.lr, t.decay));
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const long long i = base + lane + 32 * k;
    m[k] = v[k] = r[k] = 0.f;
    if (i < 0 || i >= t.count) continue;
    const float g = t.g16 ? to_f(static_cast<const __nv_bfloat16*>(t.grad)[i])
                          : static_cast<const float*>(t.grad)[i];
    float p = t.master ? t.master[i]
              : t.p16  ? to_f(static_cast<const __nv_bfloat16*>(t.param)[i])
                       : static_cast<const float*>(t.param)[i];
    if (t.q8) {
      m[k] = decode_m((float)static_cast<const signed char*>(t.m)[i], ms);
      v[k] = decode_root((float)static_cast<const unsigned char*>(t.v)[i], vs);
      v[k] = __fmul_rn(v[k], v[k]);
    } else {
      m[k] = static_cast<const float*>(t.m)[i];
      v[k] = static_cast<const float*>(t.v)[i];
    }
    float2 p2 = both(p), m2 = both(m[k]), v2 = both(v[k]), r2;
    update2(h, st, keep, both(g), p2, m2, v2, r2);
    p = p2.x, m[k] = m2.x, v[k] = v2.x, r[k] = r2.x;
    if (t.master) t.master[i] = p;
    if (t.p16)
      static_cast<__nv_bfloat16*>(t.param)[i] = __float2bfloat16_rn(p);
    else
      static_cast<float*>(t.param)[i] = p;
    if (!t.q8) {
      static_cast<float*>(t.m)[i] = m[k];
      static_cast<float*>(t.v)[i] = v[k];
    }
  }
  if (!t.q8) return;
  __syncwarp();  // every lane has read the old scales
  float inv_m, inv_v;
  new_scales(t, blk, lane, m, r, &inv_m, &inv_v);
  uint32_t qm[kPer], qv[kPer];
  encode8(m, r, inv_m, inv_v, qm, qv);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const long long i = base + lane + 32 * k;
    if (i >= t.count) continue;
    static_cast<unsigned char*>(t.m)[i] = (unsigned char)qm[k];
    static_cast<unsigned char*>(t.v)[i] = (unsigned char)qv[k];
  }
}

template <bool G16, bool Q8, bool VEC>
__device__ __forceinline__ void by_param(const Entry& t, long long base, int lane,
                                         const AdamScalars& h, const Step& st) {
  if (!t.p16)
    whole_block<0, G16, Q8, VEC>(t, base, lane, h, st);
  else if (t.master)
    whole_block<1, G16, Q8, VEC>(t, base, lane, h, st);
  else
    whole_block<2, G16, Q8, VEC>(t, base, lane, h, st);
}

// Float32 with 32-bit states, 60 M elements: 277 us, 6.05 TB/s, memory's rate
// for three streams read and written (28 bytes an element).  8-bit states with
// bf16 parameters and float32 masters, 64 M elements: 229 us, where the 16
// bytes an element take 152; bound by the chain of a warp's 80 instructions an
// element at 27 warps an SM (2.4 of 4 a cycle).  64 registers and four blocks
// to an SM: 48 took 255 us there, 72 276.  Consecutive chunks for a block
// instead of strided ones took 364 us on the float32 tensors (blocks then stay
// equally far apart in memory).
template <typename TB>
__global__ void __launch_bounds__(kThreads, 4)
    adamw_kernel(const __grid_constant__ TB tb, const __grid_constant__ AdamScalars h) {
  pdl_wait();
  pdl_release();
  const Step st = make_step(h);
  const unsigned chunks = tb.first[tb.count];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (unsigned c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int ti = find(tb, c);
    const Entry& t = tb.t[ti];
    const long long base =
        (long long)(c - tb.first[ti]) * kChunk + warp * DC_STATE_BLOCK - t.lead;
    if (base >= t.count) continue;
    if (base < 0 || base + DC_STATE_BLOCK > t.count) {
      part_block(t, base, lane, h, st);
      continue;
    }
    switch ((t.g16 ? 4 : 0) | (t.q8 ? 2 : 0) | (t.vec ? 1 : 0)) {
      case 0: by_param<false, false, false>(t, base, lane, h, st); break;
      case 1: by_param<false, false, true>(t, base, lane, h, st); break;
      case 2: by_param<false, true, false>(t, base, lane, h, st); break;
      case 3: by_param<false, true, true>(t, base, lane, h, st); break;
      case 4: by_param<true, false, false>(t, base, lane, h, st); break;
      case 5: by_param<true, false, true>(t, base, lane, h, st); break;
      case 6: by_param<true, true, false>(t, base, lane, h, st); break;
      case 7: by_param<true, true, true>(t, base, lane, h, st); break;
    }
  }
}

// The states as float32: Entry::param receives m, Entry::master v (either null).
template <bool Q8, bool VEC>
__device__ __forceinline__ void whole_values(const Entry& t, long long base, int lane) {
  float* mo = static_cast<float*>(t.param);
  float m[kPer], v[kPer];
  if (Q8) {
    uint32_t cm[2], cv[2];
    load8<VEC>(static_cast<const unsigned char*>(t.m) + base, lane, cm);
    load8<VEC>(static_cast<const unsigned char*>(t.v) + base, lane, cv);
    const float ms = t.m_scale[base / DC_STATE_BLOCK], vs = t.v_scale[base / DC_STATE_BLOCK];
    decode8(cm, cv, ms, vs, m, v);
  } else {
    load8<VEC>(static_cast<const float*>(t.m) + base, lane, m);
    load8<VEC>(static_cast<const float*>(t.v) + base, lane, v);
  }
  if (mo) store8<VEC>(mo + base, lane, m);
  if (t.master) store8<VEC>(t.master + base, lane, v);
}

// 64 M elements of 8-bit states: 118 us, 5.4 TB/s of which four fifths are
// written; bound by memory's rate for writes.
template <typename TB>
__global__ void __launch_bounds__(kThreads) values_kernel(const __grid_constant__ TB tb) {
  pdl_wait();
  pdl_release();
  const unsigned chunks = tb.first[tb.count];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (unsigned c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int ti = find(tb, c);
    const Entry& t = tb.t[ti];
    const long long base =
        (long long)(c - tb.first[ti]) * kChunk + warp * DC_STATE_BLOCK - t.lead;
    if (base >= t.count) continue;
    if (base >= 0 && base + DC_STATE_BLOCK <= t.count) {
      if (t.q8)
        t.vec ? whole_values<true, true>(t, base, lane) : whole_values<true, false>(t, base, lane);
      else
        t.vec ? whole_values<false, true>(t, base, lane) : whole_values<false, false>(t, base, lane);
      continue;
    }
    float* mo = static_cast<float*>(t.param);
    float ms = 0.f, vs = 0.f;
    if (t.q8) ms = t.m_scale[base / DC_STATE_BLOCK], vs = t.v_scale[base / DC_STATE_BLOCK];
    for (int k = 0; k < kPer; ++k) {
      const long long i = base + lane + 32 * k;
      if (i < 0 || i >= t.count) continue;
      if (t.q8) {
        const float root = decode_root((float)static_cast<const unsigned char*>(t.v)[i], vs);
        if (mo) mo[i] = decode_m((float)static_cast<const signed char*>(t.m)[i], ms);
        if (t.master) t.master[i] = __fmul_rn(root, root);
      } else {
        if (mo) mo[i] = static_cast<const float*>(t.m)[i];
        if (t.master) t.master[i] = static_cast<const float*>(t.v)[i];
      }
    }
  }
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

// part[block] = sum of squares of the block's chunks.  A chunk is B vectors of
// 16 bytes for every thread, all under way before the first is used; chunks
// start `lead` elements ahead of their tensor, on a boundary of 16 bytes.
template <typename T, int B>
__device__ __forceinline__ void add_squares(const Entry& t, long long chunk, float (&sum)[8]) {
  constexpr int V = 16 / sizeof(T);
  const T* grad = static_cast<const T*>(t.grad);
  const long long base = chunk * (B * kThreads * V) - t.lead + threadIdx.x * V;
  uint4 w[B];
  if ((chunk > 0 || t.lead == 0) && base - threadIdx.x * V + B * kThreads * V <= t.count) {
#pragma unroll
    for (int b = 0; b < B; ++b)
      w[b] = *reinterpret_cast<const uint4*>(grad + base + b * kThreads * V);
  } else {  // an end of the tensor lies in the chunk
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const long long at = base + b * kThreads * V;
      w[b] = make_uint4(0u, 0u, 0u, 0u);
      if (at >= 0 && at + V <= t.count) {
        w[b] = *reinterpret_cast<const uint4*>(grad + at);
      } else {
        uint32_t* u = reinterpret_cast<uint32_t*>(&w[b]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          if (at + e < 0 || at + e >= t.count) continue;
          if (sizeof(T) == 4)
            u[e] = reinterpret_cast<const uint32_t*>(grad)[at + e];
          else
            u[e >> 1] |= (uint32_t) reinterpret_cast<const unsigned short*>(grad)[at + e]
                         << (16 * (e & 1));
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&w[b]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (sizeof(T) == 4) {
        const float f = __uint_as_float(u[e]);
        sum[e + 4 * (b & 1)] = fmaf(f, f, sum[e + 4 * (b & 1)]);
      } else {
        const float lo = __uint_as_float(u[e] << 16), hi = __uint_as_float(u[e] & 0xffff0000u);
        sum[e] = fmaf(lo, lo, sum[e]);
        sum[4 + e] = fmaf(hi, hi, sum[4 + e]);
      }
    }
  }
}

// Blocks' sums go to memory and a second launch adds them in a fixed order (no
// atomics).  60 M bf16 gradients: 21 us for both, 5.7 TB/s, bound by memory;
// 2.5 M float32 ones: 3.9 us, the latency of two launches.
template <int B, typename TB>
__global__ void __launch_bounds__(kThreads)
    squares_kernel(const __grid_constant__ TB tb, float* part) {
  pdl_wait();
  pdl_release();
  const unsigned chunks = tb.first[tb.count];
  float sum[8] = {};
  for (unsigned c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int ti = find(tb, c);
    const Entry& t = tb.t[ti];
    if (t.g16)
      add_squares<__nv_bfloat16, B>(t, c - tb.first[ti], sum);
    else
      add_squares<float, B>(t, c - tb.first[ti], sum);
  }
  const float all = block_sum(((sum[0] + sum[1]) + (sum[2] + sum[3])) +
                              ((sum[4] + sum[5]) + (sum[6] + sum[7])));
  if (threadIdx.x == 0) part[blockIdx.x] = all;
}

__global__ void __launch_bounds__(1024)
    grad_norm_kernel(const float* part, long long parts, float max_norm, float* norm,
                     float* scale) {
  pdl_wait();
  pdl_release();
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

// Elements from an address back to the last boundary of four of them.
int lead_of(const void* p, int size) { return (int)((uintptr_t)p / size % 4); }

// lead and vec of a tensor whose arrays are the given ones (null: not read):
// arrays that all sit the same distance past a boundary of four elements are
// read from there (vec); 8-bit blocks start with the tensor, so they need it at 0.
struct Array {
  const void* p;
  int size;
};
template <int N>
void set_grid(Entry* e, const Array (&arrays)[N]) {
  int lead = -1;
  bool same = true;
  for (const Array& a : arrays) {
    if (!a.p) continue;
    const int l = lead_of(a.p, a.size);
    if (lead < 0) lead = l;
    same &= l == lead;
  }
  e->vec = same && (!e->q8 || lead <= 0);
  e->lead = (unsigned char)(e->vec && lead > 0 ? lead : 0);
}

enum class Use { kStep, kValues, kGrad };

// The tensors of one launch; false if their chunks do not fit in 32 bits.
// chunk: elements of one, or (kGrad) its 16-byte vectors.  Values go to m[i]
// and v[i].
template <int N>
bool fill(Table<N>* tb, const dc_adamw_tensor* t, int count, int chunk, Use use,
          float* const* m, float* const* v) {
  unsigned long long at = 0;
  tb->count = count;
  for (int i = 0; i < count; ++i) {
    Entry& e = tb->t[i];
    e = Entry{t[i].param, t[i].master, t[i].grad, t[i].m, t[i].v, t[i].m_scale, t[i].v_scale,
              t[i].count, t[i].weight_decay};
    e.p16 = t[i].param_dtype == DC_BF16;
    e.g16 = t[i].grad_dtype == DC_BF16;
    e.q8 = use != Use::kGrad && t[i].state == DC_STATE_Q8;
    const int st = e.q8 ? 1 : 4, gr = e.g16 ? 2 : 4;
    if (use == Use::kValues) {
      e.param = m ? m[i] : nullptr;
      e.master = v ? v[i] : nullptr;
      set_grid(&e, {{e.m, st}, {e.v, st}, {e.param, 4}, {e.master, 4}});
    } else if (use == Use::kGrad) {
      e.lead = (unsigned char)((uintptr_t)e.grad % 16 / gr);
    } else {
      set_grid(&e, {{e.param, e.p16 ? 2 : 4}, {e.master, 4}, {e.grad, gr}, {e.m, st}, {e.v, st}});
    }
    tb->first[i] = (unsigned)at;
    if (e.count)
      at += (unsigned long long)ceil_div_ll(e.count + e.lead,
                                            use == Use::kGrad ? chunk * 16 / gr : chunk);
    if (at > UINT_MAX / 2) return false;
  }
  tb->first[count] = (unsigned)at;
  return true;
}

constexpr int kFew = 40;  // a table that fits in the first 4 KB of a launch's arguments

// f(table) with a table of the tensors, a small one where they are few.
template <typename F>
cudaError_t with_table(const dc_adamw_tensor* t, int count, int chunk, Use use, float* const* m,
                       float* const* v, F&& f) {
  if (count <= kFew) {
    Table<kFew> tb;
    return fill(&tb, t, count, chunk, use, m, v) ? f(tb) : cudaErrorInvalidValue;
  }
  Table<kAdamTensors> tb;
  return fill(&tb, t, count, chunk, use, m, v) ? f(tb) : cudaErrorInvalidValue;
}

unsigned grid_of(unsigned chunks, int per_sm) {
  const int sms = sm_count();
  const unsigned most = (unsigned)((sms ? sms : 1) * per_sm);
  return chunks < most ? chunks : most;
}

}  // namespace

cudaError_t launch_adamw(const dc_adamw_tensor* t, int count, const AdamScalars& h,
                         cudaStream_t s) {
  return with_table(t, count, kChunk, Use::kStep, nullptr, nullptr, [&](const auto& tb) {
    const unsigned grid = grid_of(tb.first[tb.count], 8);
    if (!grid) return cudaSuccess;
    return launch(adamw_kernel<std::decay_t<decltype(tb)>>, grid, kThreads, s, tb, h);
  });
}

cudaError_t launch_adamw_values(const dc_adamw_tensor* t, int count, float* const* m,
                                float* const* v, cudaStream_t s) {
  return with_table(t, count, kChunk, Use::kValues, m, v, [&](const auto& tb) {
    const unsigned grid = grid_of(tb.first[tb.count], 8);
    if (!grid) return cudaSuccess;
    return launch(values_kernel<std::decay_t<decltype(tb)>>, grid, kThreads, s, tb);
  });
}

// part: kNormParts floats, all written.  Eight vectors a thread keep enough
// loads in flight; few elements are spread over the blocks two at a time.
cudaError_t launch_grad_squares(const dc_adamw_tensor* t, int count, float* part,
                                cudaStream_t s) {
  double bytes = 0;
  for (int i = 0; i < count; ++i) bytes += (double)t[i].count * (t[i].grad_dtype == DC_BF16 ? 2 : 4);
  const bool large = bytes > 8.0 * kThreads * 16 * kNormParts;
  return with_table(t, count, (large ? 8 : 2) * kThreads, Use::kGrad, nullptr, nullptr,
                    [&](const auto& tb) {
    using TB = std::decay_t<decltype(tb)>;
    if (large)
      return launch(squares_kernel<8, TB>, (unsigned)kNormParts, kThreads, s, tb, part);
    return launch(squares_kernel<2, TB>, (unsigned)kNormParts, kThreads, s, tb, part);
  });
}

cudaError_t launch_grad_norm(const float* part, long long parts, float max_norm, float* norm,
                             float* scale, cudaStream_t s) {
  return launch(grad_norm_kernel, 1u, 1024, s, part, parts, max_norm, norm, scale);
}

}  // namespace dc
