// The optimizer step: global gradient norm and AdamW over many tensors at
// once, each in one pass over its arrays.
//
//  g = grad coef; m = b1 m + (1-b1) g; v = b2 v + (1-b2) g^2
//  w = w (1 - lr wd) - (lr / (1-b1^t)) m / (sqrt(v) / sqrt(1-b2^t) + eps)
//
// Work is cut into chunks of 2048 elements of one tensor; a CTA takes a run of
// consecutive chunks, finds its first tensor by bisection on first_chunk and
// walks on from there, so hundreds of small tensors cost no launch each (a launch
// per combination of types, mostly one).  An element's update depends on that
// element alone (8-bit states: on its block of 128), whatever the grid.
//
// FP32 states (22 to 30 bytes a weight) are bound by HBM: 714 M weights, bf16 with
// an FP32 master, 3.56 ms with the norm, 6.8 TB/s of the bytes that it asks for.
// 8-bit states (8 to 16 bytes) by instructions: 714 M bf16 weights 1.53 ms with
// stochastic rounding, 4.7 TB/s; about 72 instructions a weight issue at 81% of the
// rate, of which the two hashes are 14 and the roundings 10.  3.5 M weights 20 us
// (16 us of HBM time), 300 ragged tensors 21 us: the latency of the norm's partials,
// their total, and a search and a first load per CTA.
#include <algorithm>
#include <vector>

#include "common.cuh"

namespace biv {
namespace {

constexpr int kOT = 256;            // threads of a CTA
constexpr int kEPT = 8;             // consecutive elements per thread
constexpr int kChunk = kOT * kEPT;  // elements per chunk
constexpr int kBlk = 128;           // elements per scale of an 8-bit state
constexpr int kNormChunks = 4;      // chunks per partial sum of the norm
constexpr int kNT = 1024;           // threads that add the norm's partials up
constexpr int64_t kUnitsHere = 8192;  // partials that the norm's last CTA adds up itself
constexpr uint64_t kDrainNs = 100000000;   // what a wait for copies behind a failed one takes at most
constexpr float kMinAmax = 7.888609052210118e-31f;  // 2^-100

enum VecBits { kVec16 = 1, kVec32 = 2, kVecBulk = 4 };   // biv_opt_tensor.vec
enum ParamKind { kParamF32 = 0, kParamBf16 = 1, kParamMaster = 2 };

// the tensor that holds chunk c: the last one with first_chunk <= c, found by a
// warp that looks at 32 at once
__device__ __forceinline__ int find_tensor(const biv_opt_tensor* t, int n, int64_t c) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, i = lo + int(threadIdx.x & 31) * step;
    const int below = __popc(__ballot_sync(0xffffffffu, i < hi && t[i].first_chunk <= c));
    lo += max(below - 1, 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// two FP32 operations in one instruction
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// a + b, by single additions: a product before them keeps its own rounding (an
// addition of pairs is merged with it into one)
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  float a0, a1, b0, b1;
  unpack2(a, a0, a1);
  unpack2(b, b0, b1);
  return pack2(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// min that gives NaN where one of them is
__device__ __forceinline__ float fmin3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 8 consecutive elements of an array, as its bytes: raw words of F32 (8), BF16
// (4) or e4m3 (2)
template <int W>
struct Raw {
  uint32_t w[W];
};
// (wide: FP32 arrays keep 32 bytes' alignment, one 256-bit access)
template <int W>
__device__ __forceinline__ void load_raw(const void* p, bool wide, Raw<W>& r) {
  const uint8_t* q = static_cast<const uint8_t*>(p);
  if (W == 8 && wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1 % W]), "=r"(r.w[2 % W]), "=r"(r.w[3 % W]), "=r"(r.w[4 % W]),
                   "=r"(r.w[5 % W]), "=r"(r.w[6 % W]), "=r"(r.w[7 % W])
                 : "l"(q)
                 : "memory");
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(q);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(q + i * 4);
      r.w[i] = v.x; r.w[i + 1] = v.y; r.w[i + 2] = v.z; r.w[i + 3] = v.w;
    }
  }
}
// the same element by element; those past n read as 0
template <int W>
__device__ __forceinline__ void load_raw_slow(const void* p, int64_t e, int64_t n, Raw<W>& r) {
#pragma unroll
  for (int i = 0; i < W; ++i) r.w[i] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e + i >= n) continue;
    if constexpr (W == 8) r.w[i] = static_cast<const uint32_t*>(p)[e + i];
    else if constexpr (W == 4) r.w[i >> 1] |= uint32_t(static_cast<const uint16_t*>(p)[e + i]) << (16 * (i & 1));
    else r.w[i >> 2] |= uint32_t(static_cast<const uint8_t*>(p)[e + i]) << (8 * (i & 3));
  }
}
template <int W>
__device__ __forceinline__ void store_raw(void* p, bool wide, const Raw<W>& r) {
  uint8_t* q = static_cast<uint8_t*>(p);
  if (W == 8 && wide) {
    st_global_v8(q, r.w);
  } else if constexpr (W == 2) {
    *reinterpret_cast<uint2*>(q) = make_uint2(r.w[0], r.w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4)
      *reinterpret_cast<uint4*>(q + i * 4) = make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]);
  }
}
template <int W>
__device__ __forceinline__ void store_raw_slow(void* p, int64_t e, int64_t n, const Raw<W>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (e + i >= n) continue;
    if constexpr (W == 8) static_cast<uint32_t*>(p)[e + i] = r.w[i];
    else if constexpr (W == 4) static_cast<uint16_t*>(p)[e + i] = uint16_t(r.w[i >> 1] >> (16 * (i & 1)));
    else static_cast<uint8_t*>(p)[e + i] = uint8_t(r.w[i >> 2] >> (8 * (i & 3)));
  }
}
// as four pairs of FP32
template <int W>
__device__ __forceinline__ void to_pairs(const Raw<W>& r, uint64_t (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (W == 8) {
      f[i] = pack2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    } else if constexpr (W == 4) {
      f[i] = pack2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
    } else {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          __nv_fp8x2_storage_t(r.w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
      const float2 v = __half22float2(__half2(h));
      f[i] = pack2(v.x, v.y);
    }
  }
}

// 32-bit hash, a bijection: xor-shifts and two odd multipliers (Wellons,
// "Prospecting for hash functions", 2018)
__device__ __forceinline__ uint32_t mix32_tail(uint32_t x) {   // after the first xor-shift, before the last
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  return x * 0x846CA68Bu;
}
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = mix32_tail(x ^ (x >> 16));
  return x ^ (x >> 16);
}
// The random bits of elements id .. id + 7 (id a multiple of 8): the hash of
// (low half ^ key) + a multiple of the high half.  Here without its last
// xor-shift (x ^= x >> 16), which is undone by the first one of a second hash:
// element: low and high 16 bits of hashed(x); weight: second_hash(x).
__device__ __forceinline__ void hash8(uint64_t id, uint32_t key, uint32_t (&x)[8]) {
  const uint32_t a = uint32_t(id) ^ key, hi = uint32_t(id >> 32) * 0x85EBCA6Bu;
  if (hi == 0) {          // (a warp's elements differ here at most once in 2^32)
    const uint32_t b = a ^ (a >> 16);        // a ^ i has the same upper half for all eight
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = mix32_tail(b ^ uint32_t(i));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t y = (a ^ uint32_t(i)) + hi;
      x[i] = mix32_tail(y ^ (y >> 16));
    }
  }
}
// mix32(h ^ G) for h = x ^ (x >> 16): its first xor-shift gives x ^ G ^ (G >> 16)
__device__ __forceinline__ uint32_t second_hash(uint32_t x) {
  constexpr uint32_t G = 0x9E3779B9u;
  const uint32_t y = mix32_tail(x ^ (G ^ (G >> 16)));
  return y ^ (y >> 16);
}

// The bits of y + rnd, rnd in the digits that a rounding cuts off.  Arithmetic's NaN
// is 0x7FFFFFFF, which the sum would carry into a zero: the larger of the sum and y,
// as signed integers, keeps it and is the sum otherwise, for either sign of y (one
// instruction, as the sum alone).
// 714 M bf16 weights with 8-bit states take 1527 us, 1517 without the care for NaN
// here and below; by cvt.rs.bf16x2, which has the same bits, 1554.
__device__ __forceinline__ uint32_t add_below(float y, uint32_t rnd) {
  const int b = __float_as_int(y);
  return uint32_t(__viaddmax_s32(b, int(rnd), b));
}
// |y| <= 448 to the e4m3 grid, up with a chance of the part cut off (16 random
// bits): normal numbers keep 3 fraction bits, so 20 bits of the float fall
// away; below 2^-6 the grid is 2^-9 apart
constexpr float kE4m3Normal = 0.015625f;   // 2^-6
__device__ __forceinline__ float stochastic_normal(float y, uint32_t rnd16) {   // not NaN
  uint32_t u;   // (a multiply-add: the adders are the busier unit)
  asm("mad.lo.u32 %0, %1, 16, %2;" : "=r"(u) : "r"(rnd16), "r"(__float_as_uint(y)));
  return __uint_as_float(u & 0xFFF00000u);
}
__device__ __forceinline__ float stochastic_any(float y, uint32_t rnd16) {
  const float a = fabsf(y);
  const float small = floorf(fmaf(float(rnd16), 1.0f / 65536.0f, a * 512.0f)) * (1.0f / 512.0f);
  return a < kE4m3Normal ? copysignf(small, y) : __uint_as_float(add_below(y, rnd16 << 4) & 0xFFF00000u);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}
// Eight square roots, rounded to nearest but where two floats all but tie: from an
// approximate reciprocal root y one Newton step on x^2 = v, r = v y + (v - (v y)^2) y / 2,
// its residual exact by FMA (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990).  Zeros, the smallest values and infinities
// take sqrtf.  Returns whether none is infinite.
__device__ __forceinline__ bool sqrt8(const uint64_t (&v)[4], float (&r)[8]) {
  float f[8], x[8];
  uint64_t y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y0, y1;
    unpack2(v[i], f[2 * i], f[2 * i + 1]);
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(f[2 * i]));
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(f[2 * i + 1]));
    y[i] = pack2(y0, y1);
    unpack2(mul2(v[i], y[i]), x[2 * i], x[2 * i + 1]);
  }
  // (v y is NaN for 0 and infinity)
  float lo = fmin3_nan(x[0], x[1], x[2]);
  lo = fmin3_nan(lo, x[3], x[4]);
  lo = fmin3_nan(fmin3_nan(lo, x[5], x[6]), x[7], x[7]);
  if (lo >= 1e-15f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t e = pack2(__fmaf_rn(-x[2 * i], x[2 * i], f[2 * i]),
                               __fmaf_rn(-x[2 * i + 1], x[2 * i + 1], f[2 * i + 1]));
      unpack2(fma2(e, mul2(y[i], pack2(0.5f, 0.5f)), pack2(x[2 * i], x[2 * i + 1])), r[2 * i], r[2 * i + 1]);
    }
    return true;
  }
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[i] = sqrtf(f[i]);
    finite = finite && f[i] != INFINITY;
  }
  return finite;
}
// reciprocal to about 1 ulp
__device__ __forceinline__ float recip_near(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max over the 16 lanes that hold a block of 128
__device__ __forceinline__ float block_amax(const float (&x)[8]) {
  float a = fmaxf(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
  for (int i = 2; i < 8; i += 2) a = fmax3(a, fabsf(x[i]), fabsf(x[i + 1]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return fmaxf(a, kMinAmax);
}

// 8 values as e4m3 codes of x inv, inv = 448 (1 / amax).  ROOT: x
// are roots of second moments: a positive one that would round to 0 takes the
// smallest code, since a later m / (0 + eps) would throw the weight far off (so
// does an infinite one, where inv is 0: times its infinite scale it stays infinite).
// NaN, and an infinite first moment, become the code NaN.
template <bool SR, bool ROOT>
__device__ __forceinline__ Raw<2> encode8(const float (&x)[8], float inv, const uint32_t (&h)[8]) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) unpack2(mul2(pack2(x[i], x[i + 1]), pack2(inv, inv)), y[i], y[i + 1]);
  auto rnd = [&](int i) { return ROOT ? h[i] >> 16 : (h[i] ^ (h[i] >> 16)) & 0xFFFFu; };
  if (SR || ROOT) {
    float low = fmin3_nan(fabsf(y[0]), fabsf(y[1]), fabsf(y[2]));
    low = fmin3_nan(low, fabsf(y[3]), fabsf(y[4]));
    low = fmin3_nan(fmin3_nan(low, fabsf(y[5]), fabsf(y[6])), fabsf(y[7]), fabsf(y[7]));
    if (low >= kE4m3Normal) {          // nearly always: no NaN, and none on the grid's subnormal part
      if constexpr (SR) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = stochastic_normal(y[i], rnd(i));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (SR) y[i] = stochastic_any(y[i], rnd(i));
        if (ROOT && x[i] > 0.f) y[i] = fmaxf(y[i], 0.001953125f);
      }
    }
  }
  Raw<2> r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.w[i] = e4m3x2(y[4 * i], y[4 * i + 1]) | (e4m3x2(y[4 * i + 2], y[4 * i + 3]) << 16);
  return r;
}

struct AdamArgs {
  const biv_opt_tensor* t;
  int n;
  int64_t chunks;
  const float* lr;
  const float* clip;
  int32_t* step;
  double b1d, b2d;
  float b1, c1, b2, c2, eps;   // c1 = 1 - b1, c2 = 1 - b2
  uint32_t seed_lo, seed_hi;
  int* err;
};

struct StepScalars {
  float coef, rbc2, lr, lr_bc1;
  uint32_t key;
};

__device__ __forceinline__ double pow_int(double b, uint32_t t) {
  double r = 1.0;
  while (t) {
    if (t & 1) r *= b;
    b *= b;
    t >>= 1;
  }
  return r;
}

// What a chunk is made of: PK the weight's kind, GB bf16 gradients, E8 8-bit
// states, SR stochastic rounding.
template <int PK, bool GB, bool E8, bool SR>
struct Kind {
  static constexpr int GW = GB ? 4 : 8, PW = PK == kParamBf16 ? 4 : 8, SW = E8 ? 2 : 8;
  Raw<GW> g;
  Raw<PW> w;
  Raw<SW> m, v;
  float sm, sv;           // scales of m, v (8-bit states)
  Raw<4> w16;             // a master's bf16 copy
};

struct TensorScalars {
  float keep, rate;       // 1 - lr wd; lr / (1 - b1^t)
};

// The update of a thread's 8 elements, in place; id: the first one's number for
// the random bits.
template <int PK, bool GB, bool E8, bool SR>
__device__ __forceinline__ void adam_math(Kind<PK, GB, E8, SR>& d, const AdamArgs& a,
                                          const StepScalars& s, const TensorScalars& ts, uint64_t id) {
  uint64_t g[4], w[4], m[4], v[4];
  to_pairs(d.g, g);
  to_pairs(d.w, w);
  to_pairs(d.m, m);
  to_pairs(d.v, v);
  float mf[8], rf[8], wf[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E8) {
      m[i] = mul2(m[i], pack2(d.sm, d.sm));
      v[i] = mul2(v[i], pack2(d.sv, d.sv));
      v[i] = mul2(v[i], v[i]);
    }
    const uint64_t gi = mul2(g[i], pack2(s.coef, s.coef));
    m[i] = add2(mul2(pack2(a.b1, a.b1), m[i]), mul2(pack2(a.c1, a.c1), gi));
    v[i] = add2(mul2(pack2(a.b2, a.b2), v[i]), mul2(mul2(pack2(a.c2, a.c2), gi), gi));
    unpack2(m[i], mf[2 * i], mf[2 * i + 1]);
  }
  const bool finite = sqrt8(v, rf);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (rate m) / (r rbc2 + eps), rounded to nearest as the roots are, by one correction
    // of the quotient with its exact remainder (Markstein, as above)
    float d[2], q[2], n[2];
    unpack2(mul2(pack2(rf[2 * i], rf[2 * i + 1]), pack2(s.rbc2, s.rbc2)), d[0], d[1]);
    const uint64_t num = mul2(pack2(ts.rate, ts.rate), m[i]);
    unpack2(num, n[0], n[1]);
    d[0] = __fadd_rn(d[0], a.eps);
    d[1] = __fadd_rn(d[1], a.eps);
    const uint64_t rc = pack2(recip_near(d[0]), recip_near(d[1])), q0 = mul2(num, rc);
    unpack2(q0, q[0], q[1]);
    unpack2(fma2(pack2(__fmaf_rn(-q[0], d[0], n[0]), __fmaf_rn(-q[1], d[1], n[1])), rc, q0), q[0], q[1]);
    float w0, w1;
    unpack2(mul2(w[i], pack2(ts.keep, ts.keep)), w0, w1);
    wf[2 * i] = __fsub_rn(w0, q[0]);
    wf[2 * i + 1] = __fsub_rn(w1, q[1]);
  }
  if (!finite) {           // an infinite second moment moves its weight no more
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[2], y[2];
      unpack2(w[i >> 1], x[0], x[1]);
      unpack2(m[i >> 1], y[0], y[1]);
      const float d = __fadd_rn(__fmul_rn(rf[i], s.rbc2), a.eps);
      wf[i] = __fsub_rn(__fmul_rn(x[i & 1], ts.keep), __fdiv_rn(__fmul_rn(ts.rate, y[i & 1]), d));
    }
  }
  uint32_t h[8];
  if constexpr (SR && (E8 || PK == kParamBf16)) hash8(id, s.key, h);
  if constexpr (PK != kParamBf16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) d.w.w[i] = __float_as_uint(wf[i]);
  }
  if constexpr (PK != kParamF32) {
    Raw<4> b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (SR && PK == kParamBf16) {
        const uint32_t lo = add_below(wf[2 * i], second_hash(h[2 * i]) & 0xFFFFu);
        const uint32_t hi = add_below(wf[2 * i + 1], second_hash(h[2 * i + 1]) & 0xFFFFu);
        b.w[i] = __byte_perm(lo, hi, 0x7632);
      } else {
        const __nv_bfloat162 c = __floats2bfloat162_rn(wf[2 * i], wf[2 * i + 1]);
        b.w[i] = *reinterpret_cast<const uint32_t*>(&c);
      }
    }
    if constexpr (PK == kParamBf16) d.w = b; else d.w16 = b;
  }
  if constexpr (E8) {
    const float am = block_amax(mf), ar = block_amax(rf);
    // both reciprocals by one instruction sequence, half of the lanes each
    const float inv = __fmul_rn(448.0f, __frcp_rn(threadIdx.x & 1 ? ar : am));
    const int first = threadIdx.x & 30;            // (a lane of the same block)
    d.m = encode8<SR, false>(mf, __shfl_sync(0xffffffffu, inv, first), h);
    d.v = encode8<SR, true>(rf, __shfl_sync(0xffffffffu, inv, first + 1), h);
    d.sm = __fmul_rn(am, 1.0f / 448.0f);
    d.sv = __fmul_rn(ar, 1.0f / 448.0f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) d.m.w[i] = __float_as_uint(mf[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v0, v1;
      unpack2(v[i], v0, v1);
      d.v.w[2 * i] = __float_as_uint(v0);
      d.v.w[2 * i + 1] = __float_as_uint(v1);
    }
  }
}

// Staging (8-bit states): one thread copies a chunk's arrays to shared memory by
// bulk copies that complete on the stage's mbarrier, a few chunks ahead; each
// thread reads its own 8 elements back.  An array's area holds the chunk's bytes
// in order.
template <int W>
__device__ __forceinline__ void from_stage(const uint8_t* slot, Raw<W>& r) {
  const uint8_t* q = slot + threadIdx.x * (W * 4);
  if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(q);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(q + i * 4);
      r.w[i] = v.x; r.w[i + 1] = v.y; r.w[i + 2] = v.z; r.w[i + 3] = v.w;
    }
  }
}
template <int GW, int PW>
struct StageLayout {   // a stage: gradient, weight, codes, scales
  static constexpr int W = kOT * GW * 4, M = W + kOT * PW * 4, V = M + kOT * 8, MS = V + kOT * 8,
                       VS = MS + kChunk / kBlk * 4, BYTES = VS + kChunk / kBlk * 4;
  static constexpr int STAGES = (50 << 10) / BYTES;    // four CTAs per SM
};
struct Ring {          // where the next chunk of a CTA is staged, over its tensors
  uint8_t* bufs;
  uint64_t* bars;
  uint32_t* read;      // warps that have read the stage
  int stage;
  uint32_t phase;
  int* err;
  bool dead;           // a wait ran out: this warp does no more
};

// `count` consecutive chunks of one tensor, the first one number `chunk` of it.
// Full chunks of aligned arrays take the fast way.  With 8-bit states a chunk is
// few bytes and much arithmetic: its arrays are copied to shared memory ahead, so
// that loads are in flight while a warp computes, at no register's cost and a
// few instructions of one thread.
template <int PK, bool GB, bool E8, bool SR>
__device__ __forceinline__ void adam_run(const biv_opt_tensor& t, int64_t chunk, int64_t count,
                                         const AdamArgs& a, const StepScalars& s, Ring& ring) {
  using K = Kind<PK, GB, E8, SR>;
  using L = StageLayout<K::GW, K::PW>;
  constexpr int kGB = kChunk * K::GW / 2, kPB = kChunk * K::PW / 2, kSB = kChunk * K::SW / 2,
                kScales = kChunk / kBlk;
  const int64_t n = t.numel, e0 = chunk * kChunk + threadIdx.x * kEPT;
  TensorScalars ts;
  ts.rate = __fmul_rn(s.lr_bc1, t.lr_scale);
  ts.keep = __fsub_rn(1.0f, __fmul_rn(__fmul_rn(s.lr, t.lr_scale), t.weight_decay));
  void* weight = PK == kParamMaster ? static_cast<void*>(t.master) : t.param;
  const int64_t full = t.vec ? min(count, max(int64_t(0), n / kChunk - chunk)) : 0;
  const uint64_t id0 = uint64_t(t.rng_base + e0);
  const bool wide = (t.vec & kVec32) != 0, staged = E8 && (t.vec & kVecBulk);
  {
    const uint8_t* pg = static_cast<const uint8_t*>(t.grad) + e0 * (K::GW / 2);
    uint8_t* pw = static_cast<uint8_t*>(weight) + e0 * (K::PW / 2);
    uint8_t* pc = static_cast<uint8_t*>(t.param) + e0 * 2;
    uint8_t* pm = static_cast<uint8_t*>(t.m) + e0 * (K::SW / 2);
    uint8_t* pv = static_cast<uint8_t*>(t.v) + e0 * (K::SW / 2);
    float* pms = t.m_scale + (e0 >> 7);
    float* pvs = t.v_scale + (e0 >> 7);
    auto copy_ahead = [&](int64_t k, int stage) {     // chunk k of the run, by one thread
      const uint32_t bar = smem_u32(ring.bars + stage), st = smem_u32(ring.bufs) + stage * L::BYTES;
      const int64_t c = chunk + k;
      mbar_expect_tx(bar, kGB + kPB + 2 * kSB + 2 * kScales * 4);
      bulk_load(st, static_cast<const uint8_t*>(t.grad) + c * kGB, kGB, bar);
      bulk_load(st + L::W, static_cast<const uint8_t*>(weight) + c * kPB, kPB, bar);
      bulk_load(st + L::M, static_cast<const uint8_t*>(t.m) + c * kSB, kSB, bar);
      bulk_load(st + L::V, static_cast<const uint8_t*>(t.v) + c * kSB, kSB, bar);
      bulk_load(st + L::MS, t.m_scale + c * kScales, kScales * 4, bar);
      bulk_load(st + L::VS, t.v_scale + c * kScales, kScales * 4, bar);
    };
    if (staged) __syncthreads();           // the tensor before: its last stages are read
    if (ring.dead) return;
    if (staged && threadIdx.x == 0) {
      for (int k = 0; k < L::STAGES && k < full; ++k) {
        const int st = ring.stage + k;
        copy_ahead(k, st < L::STAGES ? st : st - L::STAGES);
      }
    }
    for (int64_t k = 0; k < full; ++k) {
      K d;
      if (staged) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(ring.bars + ring.stage), ring.phase, ring.err))) {
          // given up: nothing is written from here on, and copies in flight get some
          // time to land
          ring.dead = true;
          for (int i = 0; i < L::STAGES; ++i)
            mbar_wait(smem_u32(ring.bars + i), i < ring.stage ? ring.phase ^ 1u : ring.phase, ring.err, kDrainNs);
          return;
        }
        const uint8_t* st = ring.bufs + ring.stage * L::BYTES;
        from_stage(st, d.g);
        from_stage(st + L::W, d.w);
        from_stage(st + L::M, d.m);
        from_stage(st + L::V, d.v);
        d.sm = reinterpret_cast<const float*>(st + L::MS)[threadIdx.x >> 4];
        d.sv = reinterpret_cast<const float*>(st + L::VS)[threadIdx.x >> 4];
        // the warp that reads a stage last fills it again: none waits for another
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
          __threadfence_block();
          if (atomicInc(ring.read + ring.stage, kOT / 32 - 1) == kOT / 32 - 1 && k + L::STAGES < full)
            copy_ahead(k + L::STAGES, ring.stage);
        }
        if (++ring.stage == L::STAGES) {
          ring.stage = 0;
          ring.phase ^= 1;
        }
      } else {
        load_raw(pg, wide, d.g);
        load_raw(pw, wide, d.w);
        load_raw(pm, wide, d.m);
        load_raw(pv, wide, d.v);
        if (E8) {
          d.sm = *pms;
          d.sv = *pvs;
        }
      }
      adam_math(d, a, s, ts, id0 + uint64_t(k) * kChunk);
      store_raw(pw, wide, d.w);
      if constexpr (PK == kParamMaster) store_raw(pc, wide, d.w16);
      store_raw(pm, wide, d.m);
      store_raw(pv, wide, d.v);
      if constexpr (E8) {
        if ((threadIdx.x & 15) == 0) {
          *pms = d.sm;
          *pvs = d.sv;
        }
        pms += kScales; pvs += kScales;
      }
      pg += kGB; pw += kPB; pc += kChunk * 2; pm += kSB; pv += kSB;
    }
  }
  // the tensor's last chunk, and tensors of any alignment
  for (int64_t k = full; k < count; ++k) {
    const int64_t x = e0 + k * kChunk, blk = x >> 7;
    static_assert(kBlk == 128, "x >> 7");
    K d;
    load_raw_slow(t.grad, x, n, d.g);
    load_raw_slow(weight, x, n, d.w);
    load_raw_slow(t.m, x, n, d.m);
    load_raw_slow(t.v, x, n, d.v);
    d.sm = d.sv = 0.f;
    if (E8 && x < n) {
      d.sm = t.m_scale[blk];
      d.sv = t.v_scale[blk];
    }
    adam_math(d, a, s, ts, id0 + uint64_t(k) * kChunk);
    store_raw_slow(weight, x, n, d.w);
    if constexpr (PK == kParamMaster) store_raw_slow(t.param, x, n, d.w16);
    store_raw_slow(t.m, x, n, d.m);
    store_raw_slow(t.v, x, n, d.v);
    if (E8 && (threadIdx.x & 15) == 0 && x < n) {
      t.m_scale[blk] = d.sm;
      t.v_scale[blk] = d.sv;
    }
  }
}

__host__ __device__ inline int kind_of(const biv_opt_tensor& t) {
  const int pk = t.param_dtype == BIV_F32 ? kParamF32 : t.master ? kParamMaster : kParamBf16;
  return pk * 4 + (t.grad_dtype == BIV_BF16 ? 2 : 0) + (t.state_dtype == BIV_E4M3 ? 1 : 0);
}

// The tensors of one kind (others are passed over); `last`: the call's last
// launch, which counts the step.  8-bit states want many warps: four CTAs per SM
// (64 registers) 1594 us where three take 1684 and five, which spill, 1866 (714 M
// weights, before the ring's last change); FP32 states are the same to 1% with two
// to four.
template <int PK, bool GB, bool E8, bool SR>
__global__ void __launch_bounds__(kOT, E8 ? 4 : 3) adamw_kernel(const __grid_constant__ AdamArgs a, int last) {
  constexpr int kKind = PK * 4 + (GB ? 2 : 0) + (E8 ? 1 : 0);
  using L = StageLayout<GB ? 4 : 8, PK == kParamBf16 ? 4 : 8>;
  __shared__ float s_bc[2];
  __shared__ __align__(8) uint64_t s_bars[L::STAGES];
  __shared__ uint32_t s_read[L::STAGES];
  extern __shared__ __align__(128) uint8_t stages[];
  if (E8 && threadIdx.x == 0) {
    for (int i = 0; i < L::STAGES; ++i) {
      mbar_init(smem_u32(s_bars + i), 1);
      s_read[i] = 0;
    }
    fence_barrier_init();
  }
  Ring ring = {stages, s_bars, s_read, 0, 0u, a.err, false};
  const int64_t c0 = a.chunks * blockIdx.x / gridDim.x;
  const int64_t c1 = a.chunks * (int64_t(blockIdx.x) + 1) / gridDim.x;
  int ti = find_tensor(a.t, a.n, c0);   // (the table is the host's: no kernel writes it)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const uint32_t step = uint32_t(a.step[0]) + 1u;
  StepScalars s;
  s.coef = 1.0f;
  if (a.clip) {
    if (!isfinite(a.clip[0])) return;   // the same answer in every CTA: nothing changes
    s.coef = a.clip[1];
  }
  if (tid == 0) s_bc[0] = float(1.0 - pow_int(a.b1d, step));
  if (tid == 32) s_bc[1] = float(1.0 / sqrt(1.0 - pow_int(a.b2d, step)));
  __syncthreads();   // also: every thread of the CTA has read the step
  s.lr = a.lr[0];
  s.lr_bc1 = __fdiv_rn(s.lr, s_bc[0]);
  s.rbc2 = s_bc[1];
  s.key = mix32(a.seed_lo + step * 0x9E3779B9u) ^ (a.seed_hi * 0x9E3779B1u);
  for (int64_t c = c0; c < c1;) {
    while (ti + 1 < a.n && a.t[ti + 1].first_chunk <= c) ++ti;
    const biv_opt_tensor& t = a.t[ti];
    const int64_t end = ti + 1 < a.n ? min(c1, a.t[ti + 1].first_chunk) : c1;
    if (kind_of(t) == kKind) adam_run<PK, GB, E8, SR>(t, c - t.first_chunk, end - c, a, s, ring);
    c = end;
  }
  // the last CTA to get here stores the new step: every CTA has read the old one
  if (last && tid == 0) {
    __threadfence();
    if (atomicAdd(a.step + 1, 1) == int(gridDim.x) - 1) {
      a.step[0] = int32_t(step);
      a.step[1] = 0;
    }
  }
}

// ------------------------------------------------------------------ norm --
// sums as (value, what its rounding lost)
struct Sum2 {
  float hi, lo;
};
__device__ __forceinline__ Sum2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ Sum2 add_sums(Sum2 a, Sum2 b) {
  Sum2 r = two_sum(a.hi, b.hi);
  r.lo = __fadd_rn(r.lo, __fadd_rn(a.lo, b.lo));
  return r;
}
// over the warp, by a xor tree
__device__ __forceinline__ Sum2 warp_sum2(Sum2 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add_sums(v, {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

// the squares of a thread's 8 values of `n` chunks, all loads first
template <int W, int N>
__device__ __forceinline__ void add_squares(const uint8_t* p, bool wide, uint64_t (&q)[4]) {
  Raw<W> r[N];
#pragma unroll
  for (int k = 0; k < N; ++k) load_raw(p + int64_t(k) * kChunk * (W / 2), wide, r[k]);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint64_t f[4];
    to_pairs(r[k], f);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = fma2(f[i], f[i], q[i]);
  }
}
template <int W>
__device__ __forceinline__ void add_squares_slow(const biv_opt_tensor& t, int64_t e, uint64_t (&q)[4]) {
  Raw<W> r;
  load_raw_slow(t.grad, e, t.numel, r);
  uint64_t f[4];
  to_pairs(r, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = fma2(f[i], f[i], q[i]);
}

// All partials: thread i of 1024 takes i, i + 1024, ... in order, then a xor tree
// over its warp and one over the 32 warps.  By NT threads, each in the place of 1024 / NT.
template <int NT>
__device__ __forceinline__ void norm_total(const float2* part, int64_t units, float max_norm, float* out,
                                           Sum2 (&red)[kNT / 32]) {
  constexpr int R = kNT / NT;
  const int tid = threadIdx.x;
  Sum2 v[R];
#pragma unroll
  for (int k = 0; k < R; ++k) v[k] = {0.f, 0.f};
#pragma unroll 2
  for (int64_t i = tid; i < units; i += kNT) {
    float2 p[R];
#pragma unroll
    for (int k = 0; k < R; ++k) p[k] = i + k * NT < units ? __ldcg(part + i + k * NT) : make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] = add_sums(v[k], {p[k].x, p[k].y});
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < R; ++k) {
    v[k] = warp_sum2(v[k]);
    if ((tid & 31) == 0) red[(k * NT + tid) >> 5] = v[k];
  }
  __syncthreads();
  if (tid < 32) {
    const Sum2 tot = warp_sum2(red[tid]);
    if (tid == 0) {
      const float norm = float(sqrt(double(tot.hi) + double(tot.lo)));
      out[0] = norm;
      out[1] = max_norm > 0.f ? fminf(1.0f, __fmul_rn(max_norm, __frcp_rn(__fadd_rn(norm, 1e-6f)))) : 1.0f;
    }
  }
}

// partial u: the squares of chunks [4u, 4u + 4): eight sums per thread, over the
// chunks in order, then all of them with the rounding errors kept: the thread's
// in order, a warp xor tree, the warps in order.  `here`: the last CTA to be done
// adds the partials up too (few of them), counted in out[2].
__global__ void __launch_bounds__(kOT) grad_norm_kernel(const biv_opt_tensor* __restrict__ tens,
                                                        int n, int64_t chunks, int64_t units,
                                                        float2* __restrict__ part, int here,
                                                        float max_norm, float* out) {
  __shared__ Sum2 red[2][kOT / 32], total[kNT / 32];
  __shared__ bool s_last;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (int64_t(blockIdx.x) + 1) / gridDim.x;
  int ti = find_tensor(tens, n, u0 * kNormChunks);   // (the table is the host's: no kernel writes it)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  for (int64_t u = u0; u < u1; ++u) {
    uint64_t q[4] = {0, 0, 0, 0};
    const int64_t c0 = u * kNormChunks;
    while (ti + 1 < n && tens[ti + 1].first_chunk <= c0) ++ti;
    const biv_opt_tensor& t = tens[ti];
    const int64_t in = c0 - t.first_chunk;     // chunk of the tensor
    if (t.vec && (in + kNormChunks) * kChunk <= t.numel) {
      const int64_t e = in * kChunk + tid * kEPT;
      const uint8_t* g = static_cast<const uint8_t*>(t.grad);
      if (t.grad_dtype == BIV_BF16) add_squares<4, kNormChunks>(g + e * 2, false, q);
      else add_squares<8, kNormChunks>(g + e * 4, (t.vec & kVec32) != 0, q);
    } else {
      for (int64_t c = c0; c < min(c0 + kNormChunks, chunks); ++c) {
        while (ti + 1 < n && tens[ti + 1].first_chunk <= c) ++ti;
        const biv_opt_tensor& x = tens[ti];
        const int64_t e = (c - x.first_chunk) * kChunk + tid * kEPT;
        const uint8_t* g = static_cast<const uint8_t*>(x.grad);
        const bool bf = x.grad_dtype == BIV_BF16;
        if (x.vec && (c - x.first_chunk + 1) * kChunk <= x.numel) {
          if (bf) add_squares<4, 1>(g + e * 2, false, q);
          else add_squares<8, 1>(g + e * 4, (x.vec & kVec32) != 0, q);
        } else {
          if (bf) add_squares_slow<4>(x, e, q);
          else add_squares_slow<8>(x, e, q);
        }
      }
    }
    Sum2 v = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unpack2(q[i], a, b);
      v = add_sums(v, two_sum(a, b));
    }
    v = warp_sum2(v);
    // two rows of partials in turn: one barrier per unit
    Sum2* row = red[u & 1];
    if ((tid & 31) == 0) row[tid >> 5] = v;
    __syncthreads();
    if (tid == 0) {
      Sum2 tot = row[0];
#pragma unroll
      for (int i = 1; i < kOT / 32; ++i) tot = add_sums(tot, row[i]);
      part[u] = make_float2(tot.hi, tot.lo);
    }
  }
  if (!here) return;
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(reinterpret_cast<unsigned*>(out) + 2, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (s_last) {
    __threadfence();
    norm_total<kOT>(part, units, max_norm, out, total);
    if (tid == 0) reinterpret_cast<unsigned*>(out)[2] = 0;
  }
}

__global__ void __launch_bounds__(kNT) grad_norm_final_kernel(const float2* __restrict__ part,
                                                              int64_t units, float max_norm,
                                                              float* __restrict__ out) {
  __shared__ Sum2 red[kNT / 32];
  pdl_wait();
  pdl_trigger();
  norm_total<kNT>(part, units, max_norm, out, red);
}

int64_t norm_units(int64_t chunks) { return (chunks + kNormChunks - 1) / kNormChunks; }

constexpr int kKinds = 12;

template <int PK, bool GB, bool E8, bool SR>
biv_status launch_adamw(const AdamArgs& a, bool last, cudaStream_t s) {
  using L = StageLayout<GB ? 4 : 8, PK == kParamBf16 ? 4 : 8>;
  constexpr int kSmem = E8 ? L::STAGES * L::BYTES : 0;
  auto kern = adamw_kernel<PK, GB, E8, SR>;
  if (kSmem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return set_error(BIV_ERR_CUDA, "adamw: cannot set the shared memory size: %s",
                     cudaGetErrorString(cudaGetLastError()));
  const int sms = sm_count() > 0 ? sm_count() : 148;
  // six chunks a CTA at least, where there are enough for two CTAs per SM (3.5 M
  // weights, FP32 states: 20 us; with one or two chunks a CTA, on up to six per SM,
  // 25 us) or, with 8-bit states, for the four that run at once (300 ragged tensors:
  // 21 us against 24.5 us for two and 24 us for six); and 16 CTAs per SM at most, so
  // that the faster SMs take more (714 M weights with 8-bit states: 1.5 ms against
  // 1.8 ms for two long CTAs per SM)
  const int64_t most = std::max<int64_t>((E8 ? 4 : 2) * sms, a.chunks / 6);
  const unsigned grid = unsigned(std::min(a.chunks, std::min<int64_t>(most, int64_t(sms) * 16)));
  launch_pdl(kern, grid, kOT, kSmem, s, a, int(last));
  return check_launch("adamw");
}
template <bool SR>
biv_status launch_kind(int kind, const AdamArgs& a, bool last, cudaStream_t s) {
  switch (kind) {
    case 0: return launch_adamw<0, false, false, SR>(a, last, s);
    case 1: return launch_adamw<0, false, true, SR>(a, last, s);
    case 2: return launch_adamw<0, true, false, SR>(a, last, s);
    case 3: return launch_adamw<0, true, true, SR>(a, last, s);
    case 4: return launch_adamw<1, false, false, SR>(a, last, s);
    case 5: return launch_adamw<1, false, true, SR>(a, last, s);
    case 6: return launch_adamw<1, true, false, SR>(a, last, s);
    case 7: return launch_adamw<1, true, true, SR>(a, last, s);
    case 8: return launch_adamw<2, false, false, SR>(a, last, s);
    case 9: return launch_adamw<2, false, true, SR>(a, last, s);
    case 10: return launch_adamw<2, true, false, SR>(a, last, s);
    default: return launch_adamw<2, true, true, SR>(a, last, s);
  }
}

struct Range {
  uintptr_t lo, hi;
  int tensor;
};

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" {

biv_status biv_opt_plan(biv_opt_tensor* t, int n, int64_t* chunks, int* kinds) {
  BIV_REQUIRE(n >= 0 && chunks && kinds && (t || n == 0), "opt_plan: null pointer or negative count");
  int64_t c = 0, base = 0;
  int seen = 0;
  try {
    std::vector<Range> written;
    written.reserve(size_t(n) * 6);
    for (int i = 0; i < n; ++i) {
      biv_opt_tensor& x = t[i];
      BIV_REQUIRE(x.numel >= 0 && x.numel <= (int64_t(1) << 40), "opt_plan: tensor %d: bad numel", i);
      BIV_REQUIRE(x.param_dtype == BIV_F32 || x.param_dtype == BIV_BF16,
                  "opt_plan: tensor %d: param must be f32 or bf16", i);
      BIV_REQUIRE(x.grad_dtype == BIV_F32 || x.grad_dtype == BIV_BF16,
                  "opt_plan: tensor %d: grad must be f32 or bf16", i);
      BIV_REQUIRE(x.state_dtype == BIV_F32 || x.state_dtype == BIV_E4M3,
                  "opt_plan: tensor %d: states must be f32 or e4m3", i);
      BIV_REQUIRE(!(x.param_dtype == BIV_F32 && x.master),
                  "opt_plan: tensor %d: an f32 param takes no master", i);
      x.first_chunk = c;
      x.rng_base = base;
      x.vec = 0;
      if (x.numel == 0) continue;
      const bool e8 = x.state_dtype == BIV_E4M3;
      BIV_REQUIRE(x.param && x.grad && x.m && x.v && (!e8 || (x.m_scale && x.v_scale)),
                  "opt_plan: tensor %d: null pointer", i);
      const size_t pb = x.param_dtype == BIV_F32 ? 4 : 2, gb = x.grad_dtype == BIV_F32 ? 4 : 2;
      const size_t sb = e8 ? 1 : 4;
      auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
      BIV_REQUIRE(at(x.param) % pb == 0 && at(x.grad) % gb == 0 && at(x.m) % sb == 0 &&
                      at(x.v) % sb == 0 && at(x.master) % 4 == 0 &&
                      (!e8 || (at(x.m_scale) % 4 == 0 && at(x.v_scale) % 4 == 0)),
                  "opt_plan: tensor %d: a pointer is not aligned to its elements", i);
      // 16-byte accesses of 8 (bf16), 4 (f32) or 8-byte ones of 8 (e4m3) elements
      const size_t sa = e8 ? 8 : 16;
      x.vec = at(x.param) % 16 == 0 && at(x.grad) % 16 == 0 && at(x.master) % 16 == 0 &&
              at(x.m) % sa == 0 && at(x.v) % sa == 0;
      // 32-byte ones of 8 (f32) elements
      const bool f32_32 = (x.param_dtype != BIV_F32 || at(x.param) % 32 == 0) && at(x.master) % 32 == 0 &&
                          (x.grad_dtype != BIV_F32 || at(x.grad) % 32 == 0) &&
                          (e8 || (at(x.m) % 32 == 0 && at(x.v) % 32 == 0));
      // bulk copies of whole chunks (8-bit states)
      const bool bulk = e8 && at(x.m) % 16 == 0 && at(x.v) % 16 == 0 && at(x.m_scale) % 16 == 0 &&
                        at(x.v_scale) % 16 == 0;
      if (x.vec) x.vec = kVec16 | (f32_32 ? kVec32 : 0) | (bulk ? kVecBulk : 0);
      c += (x.numel + kChunk - 1) / kChunk;
      seen |= 1 << kind_of(x);
      const int64_t blocks = (x.numel + kBlk - 1) / kBlk;
      base += blocks * kBlk;
      const size_t ne = size_t(x.numel);
      written.push_back({at(x.param), at(x.param) + ne * pb, i});
      if (x.master) written.push_back({at(x.master), at(x.master) + ne * 4, i});
      written.push_back({at(x.m), at(x.m) + ne * sb, i});
      written.push_back({at(x.v), at(x.v) + ne * sb, i});
      if (e8) {
        written.push_back({at(x.m_scale), at(x.m_scale) + size_t(blocks) * 4, i});
        written.push_back({at(x.v_scale), at(x.v_scale) + size_t(blocks) * 4, i});
      }
    }
    std::sort(written.begin(), written.end(),
              [](const Range& p, const Range& q) { return p.lo < q.lo; });
    for (size_t i = 1; i < written.size(); ++i)
      BIV_REQUIRE(written[i].lo >= written[i - 1].hi, "opt_plan: tensors %d and %d write the same memory",
                  written[i - 1].tensor, written[i].tensor);
    // a gradient inside a written range would be read after it changed
    for (int i = 0; i < n; ++i) {
      if (t[i].numel == 0) continue;
      const uintptr_t lo = reinterpret_cast<uintptr_t>(t[i].grad);
      const uintptr_t hi = lo + size_t(t[i].numel) * (t[i].grad_dtype == BIV_F32 ? 4 : 2);
      const auto r = std::lower_bound(written.begin(), written.end(), lo,
                                      [](const Range& p, uintptr_t v) { return p.hi <= v; });
      BIV_REQUIRE(r == written.end() || r->lo >= hi,
                  "opt_plan: the gradient of tensor %d overlaps what tensor %d writes", i, r->tensor);
    }
  } catch (...) {
    return set_error(BIV_ERR_INVALID, "opt_plan: out of host memory");
  }
  *chunks = c;
  *kinds = seen;
  return BIV_OK;
}

biv_status biv_grad_norm_workspace(int64_t chunks, size_t* bytes) {
  BIV_REQUIRE(chunks >= 0 && bytes, "grad_norm_workspace: bad arguments");
  *bytes = size_t(std::max<int64_t>(1, norm_units(chunks))) * sizeof(float2);
  return BIV_OK;
}

biv_status biv_grad_norm(const biv_opt_tensor* tensors, int n, int64_t chunks, float max_norm,
                         float* out, void* workspace, size_t workspace_bytes, biv_stream_t stream) {
  BIV_REQUIRE(n >= 0 && chunks >= 0 && (n > 0 || chunks == 0), "grad_norm: bad sizes");
  BIV_REQUIRE(max_norm >= 0.f, "grad_norm: max_norm must not be negative");
  BIV_REQUIRE(out && (tensors || chunks == 0), "grad_norm: null pointer");
  const int64_t units = norm_units(chunks);
  const size_t need = size_t(std::max<int64_t>(1, units)) * sizeof(float2);
  if (!workspace || workspace_bytes < need)
    return set_error(BIV_ERR_WORKSPACE, "grad_norm: workspace of %zu bytes needed", need);
  BIV_REQUIRE(aligned16(workspace), "grad_norm: workspace must be 16-byte aligned");
  cudaStream_t s = as_cuda(stream);
  float2* part = static_cast<float2*>(workspace);
  const bool here = units > 0 && units <= kUnitsHere;
  if (units > 0) {
    const int sms = sm_count() > 0 ? sm_count() : 148;
    const unsigned grid = unsigned(std::min<int64_t>(units, int64_t(sms) * 8));
    launch_pdl(grad_norm_kernel, grid, kOT, 0, s, tensors, n, chunks, units, part, int(here), max_norm, out);
    biv_status st = check_launch("grad_norm");
    if (st != BIV_OK || here) return st;
  }
  launch_pdl(grad_norm_final_kernel, 1, kNT, 0, s, static_cast<const float2*>(part), units, max_norm, out);
  return check_launch("grad_norm_final");
}

biv_status biv_adamw(const biv_adamw_desc* d, biv_stream_t stream) {
  BIV_REQUIRE(d, "adamw: null descriptor");
  BIV_REQUIRE(d->n >= 0 && d->chunks >= 0 && (d->n > 0 || d->chunks == 0), "adamw: bad sizes");
  BIV_REQUIRE(d->beta1 >= 0.0 && d->beta1 < 1.0 && d->beta2 >= 0.0 && d->beta2 < 1.0,
              "adamw: betas must lie in [0, 1)");
  BIV_REQUIRE(d->eps >= 1e-30f, "adamw: eps must be at least 1e-30");
  BIV_REQUIRE(d->rounding == BIV_ROUND_NEAREST || d->rounding == BIV_ROUND_STOCHASTIC,
              "adamw: unknown rounding");
  if (d->chunks == 0) return BIV_OK;
  BIV_REQUIRE(d->kinds > 0 && d->kinds < (1 << kKinds), "adamw: kinds is not what biv_opt_plan gave");
  BIV_REQUIRE(d->tensors && d->lr && d->step, "adamw: null pointer");
  AdamArgs a;
  a.t = d->tensors; a.n = d->n; a.chunks = d->chunks;
  a.lr = d->lr; a.clip = d->clip; a.step = d->step;
  a.b1d = d->beta1; a.b2d = d->beta2;
  a.b1 = float(d->beta1); a.c1 = float(1.0 - d->beta1);
  a.b2 = float(d->beta2); a.c2 = float(1.0 - d->beta2);
  a.eps = d->eps;
  a.err = device_error_word();
  a.seed_lo = uint32_t(d->seed); a.seed_hi = uint32_t(d->seed >> 32);
  int left = d->kinds;
  cudaStream_t s = as_cuda(stream);
  for (int k = 0; k < kKinds; ++k) {
    if (!((left >> k) & 1)) continue;
    left &= ~(1 << k);
    const biv_status st = d->rounding == BIV_ROUND_STOCHASTIC ? launch_kind<true>(k, a, left == 0, s)
                                                              : launch_kind<false>(k, a, left == 0, s);
    if (st != BIV_OK) return st;
  }
  return BIV_OK;
}

}  // extern "C"
