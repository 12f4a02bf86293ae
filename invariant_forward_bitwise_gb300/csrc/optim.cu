// The optimizer step: global gradient norm and AdamW over many tensors at
// once, each in one pass over its arrays.
//
//  g = grad coef; m = b1 m + (1-b1) g; v = b2 v + (1-b2) g^2
//  w = w (1 - lr wd) - (lr / (1-b1^t)) m / (sqrt(v) / sqrt(1-b2^t) + eps)
//
// Work is cut into chunks of 2048 elements of one tensor; a CTA takes a run of
// consecutive chunks, finds its first tensor by bisection on first_chunk and
// walks on from there, so hundreds of small tensors cost no launch each.  An
// element's update depends on that element alone (8-bit states: on its block
// of 128), whatever the grid.
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
constexpr int kNT = 1024;           // threads of the norm's second kernel
constexpr float kMinAmax = 7.888609052210118e-31f;  // 2^-100

enum ParamKind { kParamF32 = 0, kParamBf16 = 1, kParamMaster = 2 };

// the tensor that holds chunk c: the last one with first_chunk <= c
__device__ __forceinline__ int find_tensor(const biv_opt_tensor* t, int n, int64_t c) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t[mid].first_chunk <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// 8 consecutive values from element e on; those past n read as 0
template <bool BF>
__device__ __forceinline__ void load8(const void* p, int64_t e, int64_t n, bool vec, float (&f)[8]) {
  if (vec && e + 8 <= n) {
    if constexpr (BF) {
      const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
      const float4 a = q[0], b = q[1];
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = 0.f;
    if (e + i < n)
      f[i] = BF ? bf2f(static_cast<const uint16_t*>(p)[e + i]) : static_cast<const float*>(p)[e + i];
  }
}
__device__ __forceinline__ void store8_f32(float* p, int64_t e, int64_t n, bool vec,
                                           const float (&f)[8]) {
  if (vec && e + 8 <= n) {
    float4* q = reinterpret_cast<float4*>(p + e);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i < n) p[e + i] = f[i];
}
__device__ __forceinline__ void store8_bf16(uint16_t* p, int64_t e, int64_t n, bool vec,
                                            const uint32_t (&b)[8]) {
  if (vec && e + 8 <= n) {
    *reinterpret_cast<uint4*>(p + e) = make_uint4(b[0] | (b[1] << 16), b[2] | (b[3] << 16),
                                                  b[4] | (b[5] << 16), b[6] | (b[7] << 16));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i < n) p[e + i] = uint16_t(b[i]);
}
__device__ __forceinline__ void load8_codes(const uint8_t* p, int64_t e, int64_t n, bool vec,
                                            uint32_t (&c)[2]) {
  if (vec && e + 8 <= n) {
    const uint2 r = *reinterpret_cast<const uint2*>(p + e);
    c[0] = r.x; c[1] = r.y;
    return;
  }
  c[0] = c[1] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i < n) c[i >> 2] |= uint32_t(p[e + i]) << (8 * (i & 3));
}
__device__ __forceinline__ void store8_codes(uint8_t* p, int64_t e, int64_t n, bool vec,
                                             const uint32_t (&c)[2]) {
  if (vec && e + 8 <= n) {
    *reinterpret_cast<uint2*>(p + e) = make_uint2(c[0], c[1]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (e + i < n) p[e + i] = uint8_t(c[i >> 2] >> (8 * (i & 3)));
}

// 32-bit hash: xor-shifts and two odd multipliers (a bijection)
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

// y in [0, 448] to the e4m3 grid, up with a chance of the part cut off (16
// random bits): normal numbers keep 3 fraction bits, so 20 bits of the float
// fall away; below 2^-6 the grid is 2^-9 apart
__device__ __forceinline__ float stochastic_e4m3(float y, uint32_t rnd16) {
  const float big = __uint_as_float((__float_as_uint(y) + (rnd16 << 4)) & 0xFFF00000u);
  const float small = floorf(fmaf(float(rnd16), 1.0f / 65536.0f, y * 512.0f)) * (1.0f / 512.0f);
  return y < 0.015625f ? small : big;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ void decode8(const uint32_t (&c)[2], float s, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        __nv_fp8x2_storage_t(c[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * i] = v.x * s;
    f[2 * i + 1] = v.y * s;
  }
}
// max over the 16 lanes that hold a block of 128
__device__ __forceinline__ float block_amax(const float (&x)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return fmaxf(a, kMinAmax);
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

template <int PK, bool GB, bool E8, bool SR>
__device__ __forceinline__ void adam_chunk(const biv_opt_tensor& t, int64_t e, const AdamArgs& a,
                                           const StepScalars& s) {
  const int64_t n = t.numel;
  const bool vec = t.vec != 0;
  float g[8], w[8], m[8], v[8];
  load8<GB>(t.grad, e, n, vec, g);
  load8<PK == kParamBf16>(PK == kParamMaster ? t.master : t.param, e, n, vec, w);
  const int64_t blk = e / kBlk;
  if constexpr (E8) {
    uint32_t cm[2], cv[2];
    load8_codes(static_cast<const uint8_t*>(t.m), e, n, vec, cm);
    load8_codes(static_cast<const uint8_t*>(t.v), e, n, vec, cv);
    const float sm = e < n ? t.m_scale[blk] : 0.f, sv = e < n ? t.v_scale[blk] : 0.f;
    decode8(cm, sm, m);
    decode8(cv, sv, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= v[i];
  } else {
    load8<false>(t.m, e, n, vec, m);
    load8<false>(t.v, e, n, vec, v);
  }
  const float keep = 1.0f - s.lr * t.lr_scale * t.weight_decay;
  const float rate = s.lr_bc1 * t.lr_scale;
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = g[i] * s.coef;
    m[i] = fmaf(a.b1, m[i], a.c1 * gi);
    v[i] = fmaf(a.b2, v[i], a.c2 * gi * gi);
    r[i] = sqrtf(v[i]);
    w[i] = w[i] * keep - rate * (m[i] / fmaf(r[i], s.rbc2, a.eps));
  }
  uint32_t h[8];
  if constexpr (SR && (E8 || PK == kParamBf16)) {
    const uint64_t i0 = uint64_t(t.rng_base + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t id = i0 + i;
      h[i] = mix32((uint32_t(id) ^ s.key) + uint32_t(id >> 32) * 0x85EBCA6Bu);
    }
  }
  if constexpr (PK == kParamF32) {
    store8_f32(static_cast<float*>(t.param), e, n, vec, w);
  } else {
    uint32_t b[8];
    if constexpr (PK == kParamMaster) store8_f32(t.master, e, n, vec, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (SR && PK == kParamBf16)
        b[i] = (__float_as_uint(w[i]) + (mix32(h[i] ^ 0x9E3779B9u) & 0xFFFFu)) >> 16;
      else
        b[i] = f2bf(w[i]);
    }
    store8_bf16(static_cast<uint16_t*>(t.param), e, n, vec, b);
  }
  if constexpr (E8) {
    const float am = block_amax(m), ar = block_amax(r);
    const float im = 448.0f / am, ir = 448.0f / ar;
    uint32_t cm[2] = {0, 0}, cr[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float ym[2], yr[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        ym[j] = m[i + j] * im;
        yr[j] = r[i + j] * ir;
        if constexpr (SR) {
          ym[j] = copysignf(stochastic_e4m3(fabsf(ym[j]), h[i + j] & 0xFFFFu), ym[j]);
          yr[j] = stochastic_e4m3(yr[j], h[i + j] >> 16);
        }
        // a positive root that would round to 0 takes the smallest code:
        // a later m / (0 + eps) would throw the weight far off
        if (r[i + j] > 0.f) yr[j] = fmaxf(yr[j], 0.001953125f);
      }
      cm[i >> 2] |= e4m3x2(ym[0], ym[1]) << (8 * (i & 3));
      cr[i >> 2] |= e4m3x2(yr[0], yr[1]) << (8 * (i & 3));
    }
    store8_codes(static_cast<uint8_t*>(t.m), e, n, vec, cm);
    store8_codes(static_cast<uint8_t*>(t.v), e, n, vec, cr);
    if ((threadIdx.x & 15) == 0 && e < n) {
      t.m_scale[blk] = am / 448.0f;
      t.v_scale[blk] = ar / 448.0f;
    }
  } else {
    store8_f32(static_cast<float*>(t.m), e, n, vec, m);
    store8_f32(static_cast<float*>(t.v), e, n, vec, v);
  }
}

template <int PK, bool SR>
__device__ __forceinline__ void adam_chunk_by_type(const biv_opt_tensor& t, int64_t e,
                                                   const AdamArgs& a, const StepScalars& s) {
  const bool gb = t.grad_dtype == BIV_BF16, e8 = t.state_dtype == BIV_E4M3;
  if (gb) {
    if (e8) adam_chunk<PK, true, true, SR>(t, e, a, s);
    else adam_chunk<PK, true, false, SR>(t, e, a, s);
  } else {
    if (e8) adam_chunk<PK, false, true, SR>(t, e, a, s);
    else adam_chunk<PK, false, false, SR>(t, e, a, s);
  }
}

template <bool SR>
__global__ void __launch_bounds__(kOT) adamw_kernel(const __grid_constant__ AdamArgs a) {
  __shared__ float s_bc[2];
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
  s.lr_bc1 = s.lr / s_bc[0];
  s.rbc2 = s_bc[1];
  s.key = mix32(a.seed_lo + step * 0x9E3779B9u) ^ (a.seed_hi * 0x9E3779B1u);
  const int64_t c0 = a.chunks * blockIdx.x / gridDim.x;
  const int64_t c1 = a.chunks * (int64_t(blockIdx.x) + 1) / gridDim.x;
  if (c0 < c1) {
    int ti = find_tensor(a.t, a.n, c0);
    for (int64_t c = c0; c < c1; ++c) {
      while (ti + 1 < a.n && a.t[ti + 1].first_chunk <= c) ++ti;
      const biv_opt_tensor& t = a.t[ti];
      const int64_t e = (c - t.first_chunk) * kChunk + tid * kEPT;
      if (t.param_dtype == BIV_F32) adam_chunk_by_type<kParamF32, SR>(t, e, a, s);
      else if (t.master) adam_chunk_by_type<kParamMaster, SR>(t, e, a, s);
      else adam_chunk_by_type<kParamBf16, SR>(t, e, a, s);
    }
  }
  // the last CTA to get here stores the new step: every CTA has read the old one
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(a.step + 1, 1) == int(gridDim.x) - 1) {
      a.step[0] = int32_t(step);
      a.step[1] = 0;
    }
  }
}

// ------------------------------------------------------------------ norm --
__device__ __forceinline__ float warp_sum_x(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// partial u: the squares of chunks [4u, 4u + 4), per thread in chunk order,
// then a warp xor tree and the warps in order
__global__ void __launch_bounds__(kOT) grad_norm_kernel(const biv_opt_tensor* __restrict__ tens,
                                                        int n, int64_t chunks, int64_t units,
                                                        float* __restrict__ part) {
  __shared__ float red[kOT / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (int64_t(blockIdx.x) + 1) / gridDim.x;
  if (u0 >= u1) return;
  int ti = find_tensor(tens, n, u0 * kNormChunks);
  for (int64_t u = u0; u < u1; ++u) {
    float f[kNormChunks][8];
#pragma unroll
    for (int k = 0; k < kNormChunks; ++k) {
      const int64_t c = u * kNormChunks + k;
      if (c < chunks) {
        while (ti + 1 < n && tens[ti + 1].first_chunk <= c) ++ti;
        const biv_opt_tensor& t = tens[ti];
        const int64_t e = (c - t.first_chunk) * kChunk + tid * kEPT;
        if (t.grad_dtype == BIV_BF16) load8<true>(t.grad, e, t.numel, t.vec != 0, f[k]);
        else load8<false>(t.grad, e, t.numel, t.vec != 0, f[k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[k][i] = 0.f;
      }
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < kNormChunks; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) q = fmaf(f[k][i], f[k][i], q);
    q = warp_sum_x(q);
    __syncthreads();   // red is free again
    if ((tid & 31) == 0) red[tid >> 5] = q;
    __syncthreads();
    if (tid == 0) {
      float tot = 0.f;
#pragma unroll
      for (int i = 0; i < kOT / 32; ++i) tot += red[i];
      part[u] = tot;
    }
  }
}

// all partials: thread i takes i, i + 1024, ... ascending with the rounding
// errors carried along, then a warp xor tree and the warps in order
__global__ void __launch_bounds__(kNT) grad_norm_final_kernel(const float* __restrict__ part,
                                                              int64_t units, float max_norm,
                                                              float* __restrict__ out) {
  __shared__ float red[kNT / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  float s = 0.f, lost = 0.f;
#pragma unroll 8
  for (int64_t i = tid; i < units; i += kNT) {
    const float x = part[i], y = s + x, b = y - s;
    lost += (s - (y - b)) + (x - b);
    s = y;
  }
  if (isfinite(s)) s += lost;
  s = warp_sum_x(s);
  if ((tid & 31) == 0) red[tid >> 5] = s;
  __syncthreads();
  if (tid == 0) {
    float tot = 0.f;
    for (int i = 0; i < kNT / 32; ++i) tot += red[i];
    const float norm = sqrtf(tot);
    out[0] = norm;
    out[1] = max_norm > 0.f ? fminf(1.0f, max_norm / (norm + 1e-6f)) : 1.0f;
  }
}

int64_t norm_units(int64_t chunks) { return (chunks + kNormChunks - 1) / kNormChunks; }

struct Range {
  uintptr_t lo, hi;
  int tensor;
};

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" {

biv_status biv_opt_plan(biv_opt_tensor* t, int n, int64_t* chunks) {
  BIV_REQUIRE(n >= 0 && chunks && (t || n == 0), "opt_plan: null pointer or negative count");
  int64_t c = 0, base = 0;
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
      c += (x.numel + kChunk - 1) / kChunk;
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
  return BIV_OK;
}

biv_status biv_grad_norm_workspace(int64_t chunks, size_t* bytes) {
  BIV_REQUIRE(chunks >= 0 && bytes, "grad_norm_workspace: bad arguments");
  *bytes = size_t(std::max<int64_t>(1, norm_units(chunks))) * sizeof(float);
  return BIV_OK;
}

biv_status biv_grad_norm(const biv_opt_tensor* tensors, int n, int64_t chunks, float max_norm,
                         float* out, void* workspace, size_t workspace_bytes, biv_stream_t stream) {
  BIV_REQUIRE(n >= 0 && chunks >= 0 && (n > 0 || chunks == 0), "grad_norm: bad sizes");
  BIV_REQUIRE(max_norm >= 0.f, "grad_norm: max_norm must not be negative");
  BIV_REQUIRE(out && (tensors || chunks == 0), "grad_norm: null pointer");
  const int64_t units = norm_units(chunks);
  const size_t need = size_t(std::max<int64_t>(1, units)) * sizeof(float);
  if (!workspace || workspace_bytes < need)
    return set_error(BIV_ERR_WORKSPACE, "grad_norm: workspace of %zu bytes needed", need);
  BIV_REQUIRE(aligned16(workspace), "grad_norm: workspace must be 16-byte aligned");
  cudaStream_t s = as_cuda(stream);
  float* part = static_cast<float*>(workspace);
  if (units > 0) {
    const int sms = sm_count() > 0 ? sm_count() : 148;
    const unsigned grid = unsigned(std::min<int64_t>(units, int64_t(sms) * 8));
    launch_pdl(grad_norm_kernel, grid, kOT, 0, s, tensors, n, chunks, units, part);
    biv_status st = check_launch("grad_norm");
    if (st != BIV_OK) return st;
  }
  launch_pdl(grad_norm_final_kernel, 1, kNT, 0, s, static_cast<const float*>(part), units, max_norm, out);
  return check_launch("grad_norm_final");
}

biv_status biv_adamw(const biv_adamw_desc* d, biv_stream_t stream) {
  BIV_REQUIRE(d, "adamw: null descriptor");
  BIV_REQUIRE(d->n >= 0 && d->chunks >= 0 && (d->n > 0 || d->chunks == 0), "adamw: bad sizes");
  BIV_REQUIRE(d->beta1 >= 0.0 && d->beta1 < 1.0 && d->beta2 >= 0.0 && d->beta2 < 1.0,
              "adamw: betas must lie in [0, 1)");
  BIV_REQUIRE(d->eps > 0.f, "adamw: eps must be positive");
  BIV_REQUIRE(d->rounding == BIV_ROUND_NEAREST || d->rounding == BIV_ROUND_STOCHASTIC,
              "adamw: unknown rounding");
  if (d->chunks == 0) return BIV_OK;
  BIV_REQUIRE(d->tensors && d->lr && d->step, "adamw: null pointer");
  AdamArgs a;
  a.t = d->tensors; a.n = d->n; a.chunks = d->chunks;
  a.lr = d->lr; a.clip = d->clip; a.step = d->step;
  a.b1d = d->beta1; a.b2d = d->beta2;
  a.b1 = float(d->beta1); a.c1 = float(1.0 - d->beta1);
  a.b2 = float(d->beta2); a.c2 = float(1.0 - d->beta2);
  a.eps = d->eps;
  a.seed_lo = uint32_t(d->seed); a.seed_hi = uint32_t(d->seed >> 32);
  const int sms = sm_count() > 0 ? sm_count() : 148;
  const unsigned grid = unsigned(std::min<int64_t>(d->chunks, int64_t(sms) * 8));
  cudaStream_t s = as_cuda(stream);
  if (d->rounding == BIV_ROUND_STOCHASTIC) launch_pdl(adamw_kernel<true>, grid, kOT, 0, s, a);
  else launch_pdl(adamw_kernel<false>, grid, kOT, 0, s, a);
  return check_launch("adamw");
}

}  // extern "C"
