// Rows in 8 bits: RMSNorm with the residual's addition and 8-bit outputs, and
// the activations that a trainer keeps in 8 bits with the backward passes that
// read them.  All rows are quantised alike: per 128 consecutive elements s =
// amax / 448 (1 when amax is 0), code = e4m3_rne_satfinite(v / s), as
// biv_act_quant_fp8 does.  Memory-bound: one pass over the inputs, 16-byte
// accesses, sums in FP32 in an order fixed by the row length.
#include <algorithm>

#include "common.cuh"

namespace biv {
namespace {

// two FP32 values in one register pair: an instruction for both (these kernels
// issue as much as they load)
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void split(f32x2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

// a * b + c where the caller wants an exact zero to be -0 (rounding down; the
// other sums it forms are exact)
__device__ __forceinline__ f32x2 fma2_down(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 v;
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(bf2(f[0], f[1]), bf2(f[2], f[3]), bf2(f[4], f[5]), bf2(f[6], f[7]));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// 1 / v within 1 ulp, for v and 1 / v that are not subnormal
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// two e4m3 codes, the first in the low byte
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// the values of four codes
__device__ __forceinline__ void values4(uint32_t c, float s, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> (16 * i)), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    split(mul2(pair(v.x, v.y), pair(s, s)), f[2 * i], f[2 * i + 1]);
  }
}

// The codes of a lane's 8 values of a group that 16 lanes share, and its scale
// from the group's largest magnitude.
// Scale and quotients are those of IEEE divisions: with r the correctly rounded
// reciprocal of the divisor, Markstein's correction q + (v - q s) r of q = v r
// gives them in three operations where nothing under- or overflows; one Newton
// step from within 1 ulp gives that r, unless the divisor's mantissa is all ones
// (Markstein).  Groups of such a scale, or of one far from 1, divide.
// A remainder of zero is formed as -0: times r it leaves q's sign, that of -0 / s
// among them (+0 would make it +0).
__device__ __forceinline__ uint2 quant8(const float (&v)[8], float amax, float& s) {
  float q[8];
  constexpr float r448 = 1.0f / 448.0f;
  s = amax * r448;
  s = fmaf(fmaf(-s, 448.0f, amax), r448, s);
  if (amax > 0x1p-60f && amax < 0x1p60f && (__float_as_uint(s) & 0x7FFFFFu) != 0x7FFFFFu) {
    float r1 = rcp_approx(s);
    r1 = fmaf(fmaf(-s, r1, 1.0f), r1, r1);
    const f32x2 r = pair(r1, r1), minus_s = pair(-s, -s);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const f32x2 v2 = pair(v[i], v[i + 1]), q0 = mul2(v2, r);
      split(fma2(fma2_down(q0, minus_s, v2), r, q0), q[i], q[i + 1]);
    }
  } else {
    s = amax == 0.f ? 1.0f : amax / 448.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] / s;
  }
  return make_uint2(codes2(q[0], q[1]) | (codes2(q[2], q[3]) << 16),
                    codes2(q[4], q[5]) | (codes2(q[6], q[7]) << 16));
}

// (every lane of the warp calls this; lanes behind the row hold zeros)
__device__ __forceinline__ uint2 quant8(const float (&v)[8], float& s) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  return quant8(v, half_warp_max(amax), s);
}

// ---------------------------------------------------- add + RMSNorm, FP8 ----
// A team of W warps per row (W = ceil(d / 256), at most 8), 8 / W rows per CTA (of
// 8 / W W warps: idle ones would cost as much as the others).
// Thread t of a team owns the 8-element chunks t, t + 256, ...: the sums run
// in biv_add_rmsnorm's order (its warps without chunks add zeros), so inv and
// y have its bits.  Half a warp holds a 128-element group.
struct NormArgs {
  const uint16_t* x; int64_t xs;
  const uint16_t* res; int64_t rs;
  uint16_t* res_out; int64_t ros;
  const uint16_t* w;
  uint16_t* y; int64_t ys;
  uint8_t* codes; float* scales;
  uint8_t* keep; float* keep_scales;
  float* inv;
  int rows, d, team;      // warps per row
  float eps;
};

// r' is held as bf16 and its kept codes are written before the row's sum is
// waited for: fewer registers, so more rows in flight (16384 x 4096 with all
// outputs 107 us, 94% of the copy rate; six CTAs per SM spilled, 120 us; rows of
// one chunk a thread, 32768 x 1536: eight 95 us, five 106).
template <int CPT>
__global__ void __launch_bounds__(256, CPT == 1 ? 8 : CPT == 2 ? 5 : 4)
    add_rmsnorm_fp8_kernel(const __grid_constant__ NormArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float warp_ss[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (blockDim.x >> 5) / a.team, mine = warp / a.team;        // rows per CTA, this warp's
  const int64_t row = int64_t(blockIdx.x) * per + mine;
  const bool on = row < a.rows;
  const int t = (warp - mine * a.team) * 32 + lane;        // thread of the team
  const int chunks = a.d / 8, groups = (a.d + 127) / 128;
  uint4 rp[CPT], wq[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * 256;
    rp[i] = wq[i] = make_uint4(0u, 0u, 0u, 0u);
    if (on && c < chunks) {
      rp[i] = __ldg(reinterpret_cast<const uint4*>(a.x + row * a.xs) + c);
      wq[i] = __ldg(reinterpret_cast<const uint4*>(a.w) + c);
    }
  }
  if (a.res) {
    uint4 rv[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * 256;
      rv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (on && c < chunks) rv[i] = reinterpret_cast<const uint4*>(a.res + row * a.rs)[c];
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * 256;
      float x[8], r[8];
      unpack8(rp[i], x);
      unpack8(rv[i], r);
#pragma unroll
      for (int j = 0; j < 8; j += 2) split(add2(pair(x[j], x[j + 1]), pair(r[j], r[j + 1])), x[j], x[j + 1]);
      rp[i] = pack8(x);
      if (on && c < chunks) reinterpret_cast<uint4*>(a.res_out + row * a.ros)[c] = rp[i];
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    float v[8];
    unpack8(rp[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
  }
  ss = warp_sum(ss);
  if (a.team > 1 && lane == 0) warp_ss[warp] = ss;
  if (a.keep) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = t + i * 256;
      if (c - lane >= chunks) break;           // (the whole warp)
      float v[8], s;
      unpack8(rp[i], v);
      const uint2 k = quant8(v, s);
      if (on && c < chunks) {
        reinterpret_cast<uint2*>(a.keep + row * a.d)[c] = k;
        if ((lane & 15) == 0) a.keep_scales[row * groups + c / 16] = s;
      }
    }
  }
  float tot = ss;
  if (a.team > 1) {
    __syncthreads();
    tot = 0.f;
    if (on)
      for (int i = 0; i < a.team; ++i) tot += warp_ss[mine * a.team + i];
  }
  const float inv = 1.0f / sqrtf(tot / float(a.d) + a.eps);
  if (on && t == 0 && a.inv) a.inv[row] = inv;
  const f32x2 inv2 = pair(inv, inv);
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = t + i * 256;
    if (c - lane >= chunks) break;
    const bool live = on && c < chunks;
    float v[8], wv[8];
    unpack8(rp[i], v);
    unpack8(wq[i], wv);
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      split(mul2(mul2(pair(v[j], v[j + 1]), inv2), pair(wv[j], wv[j + 1])), v[j], v[j + 1]);
    if (a.y && live) reinterpret_cast<uint4*>(a.y + row * a.ys)[c] = pack8(v);
    if (a.codes) {
      if (!live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
      }
      float s;
      const uint2 k = quant8(v, s);
      if (live) {
        reinterpret_cast<uint2*>(a.codes + row * a.d)[c] = k;
        if ((lane & 15) == 0) a.scales[row * groups + c / 16] = s;
      }
    }
  }
}

// ------------------------------------------------------ RMSNorm backward ----
// A CTA of W warps (W = ceil(d / 512), at most 16) walks rows r0, r0 + grid, ...;
// lane l of warp w owns the chunks (w * 2 + i) * 32 + l, i = 0, 1, of 8 elements
// and keeps their dw sums over the CTA's rows, which a second kernel adds up.
// With the normed row x' = code * (s inv): dx = inv (w dy - x' mean(w dy x')),
// dw = sum dy x'.  No power of inv is formed: the cube of a large row's is below
// FP32's range, and the projection would be lost.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t e, float (&f)[8]) {
  if (F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    const float4 a = s[0], b = s[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e), f);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t e, const float (&f)[8]) {
  if (F32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
    d[0] = make_float4(f[0], f[1], f[2], f[3]);
    d[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e) = pack8(f);
  }
}

struct NormBackArgs {
  const uint8_t* keep; const float* scales; const float* inv;
  const uint16_t* w;
  const void* dy; int64_t dys;
  const void* dres; int64_t drs;
  void* dx; int64_t dxs;
  float* parts;          // [grid][d]
  int rows, d;
};

constexpr int kBackChunks = 2;

// 8 values of a row as they lie in memory
template <bool F32>
struct Raw8 {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + e * (F32 ? 4 : 2));
    v[0] = s[0];
    if (F32) v[F32 ? 1 : 0] = s[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if (F32) {
      const uint4 a = v[0], b = v[F32 ? 1 : 0];
      f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
      f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
      f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
      f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    } else {
      unpack8(v[0], f);
    }
  }
};

// What a lane reads of one row.  It stays as it lies in memory (as floats the
// row's two passes over it took 181 to 231 registers a thread, 158 us for
// 16384 x 2048, now 43, 80% of the copy rate), and the next row's is loaded
// before this one is reduced.
template <bool DYF, bool DXF, bool RES>
struct BackRow {
  uint2 k[kBackChunks];
  float s[kBackChunks];
  Raw8<DYF> dy[kBackChunks];
  Raw8<DXF> res[RES ? kBackChunks : 1];
  float inv;
  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t row, int c0, int chunks, int groups) {
    inv = __ldg(a.inv + row);
#pragma unroll
    for (int i = 0; i < kBackChunks; ++i) {
      const int c = c0 + i * 32;
      if (c < chunks) {
        k[i] = __ldg(reinterpret_cast<const uint2*>(a.keep + row * a.d) + c);
        s[i] = __ldg(a.scales + row * groups + c / 16);
        dy[i].load(a.dy, row * a.dys + c * 8);
        if (RES) res[RES ? i : 0].load(a.dres, row * a.drs + c * 8);
      }
    }
  }
};

template <bool DYF, bool DXF, bool RES>
__global__ void __launch_bounds__(512) rmsnorm_bwd_fp8_kernel(const __grid_constant__ NormBackArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[2][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = a.d / 8, groups = (a.d + 127) / 128;
  const int c0 = warp * kBackChunks * 32 + lane;
  f32x2 dw[kBackChunks][4];
  uint4 wq[kBackChunks];
#pragma unroll
  for (int i = 0; i < kBackChunks; ++i) {
    const int c = c0 + i * 32;
    wq[i] = c < chunks ? __ldg(reinterpret_cast<const uint4*>(a.w) + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = 0;
  }
  BackRow<DYF, DXF, RES> next;
  next.load(a, blockIdx.x, c0, chunks, groups);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const BackRow<DYF, DXF, RES> r = next;
    if (row + gridDim.x < a.rows) next.load(a, row + gridDim.x, c0, chunks, groups);
    f32x2 sum2 = 0;
    const f32x2 inv2 = pair(r.inv, r.inv);
#pragma unroll
    for (int i = 0; i < kBackChunks; ++i) {
      if (c0 + i * 32 >= chunks) continue;
      float x[8], g[8], wv[8];
      values4(r.k[i].x, r.s[i] * r.inv, x);
      values4(r.k[i].y, r.s[i] * r.inv, x + 4);
      r.dy[i].get(g);
      unpack8(wq[i], wv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 g2 = pair(g[2 * j], g[2 * j + 1]), x2 = pair(x[2 * j], x[2 * j + 1]);
        sum2 = fma2(mul2(g2, pair(wv[2 * j], wv[2 * j + 1])), x2, sum2);
        dw[i][j] = fma2(g2, x2, dw[i][j]);
      }
    }
    float even, odd;
    split(sum2, even, odd);
    float sum = warp_sum(even + odd);
    if (warps > 1) {      // (two buffers: one barrier per row)
      if (lane == 0) red[turn][warp] = sum;
      __syncthreads();
      sum = 0.f;
      for (int i = 0; i < warps; ++i) sum += red[turn][i];
    }
    const float mean = sum / float(a.d);
    const f32x2 minus_mean = pair(-mean, -mean);
#pragma unroll
    for (int i = 0; i < kBackChunks; ++i) {
      const int c = c0 + i * 32;
      if (c >= chunks) continue;
      float x[8], g[8], wv[8], o[8];
      values4(r.k[i].x, r.s[i] * r.inv, x);
      values4(r.k[i].y, r.s[i] * r.inv, x + 4);
      r.dy[i].get(g);
      unpack8(wq[i], wv);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const f32x2 gw = mul2(pair(g[j], g[j + 1]), pair(wv[j], wv[j + 1]));
        split(mul2(inv2, fma2(pair(x[j], x[j + 1]), minus_mean, gw)), o[j], o[j + 1]);
      }
      if (RES) {
        float t[8];
        r.res[RES ? i : 0].get(t);
#pragma unroll
        for (int j = 0; j < 8; j += 2) split(add2(pair(o[j], o[j + 1]), pair(t[j], t[j + 1])), o[j], o[j + 1]);
      }
      store8<DXF>(a.dx, row * a.dxs + c * 8, o);
    }
  }
#pragma unroll
  for (int i = 0; i < kBackChunks; ++i) {
    const int c = c0 + i * 32;
    float o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) split(dw[i][j], o[2 * j], o[2 * j + 1]);
    if (c < chunks) store8<true>(a.parts, int64_t(blockIdx.x) * a.d + c * 8, o);
  }
}

template <bool DYF, bool DXF>
void launch_back(const NormBackArgs& a, int grid, int threads, cudaStream_t s) {
  launch_pdl(a.dres ? rmsnorm_bwd_fp8_kernel<DYF, DXF, true> : rmsnorm_bwd_fp8_kernel<DYF, DXF, false>,
             grid, threads, 0, s, a);
}

// dw[c] = the CTAs' partial sums: 32 warps take partials w, w + 32, ... in order
// of 32 columns, and their sums are added in warp order
__global__ void __launch_bounds__(1024) dw_sum_kernel(const float* __restrict__ parts, int n, int d,
                                                     float* __restrict__ dw, int accumulate) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sums[32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d)
#pragma unroll 8
    for (int i = warp; i < n; i += 32) s += parts[int64_t(i) * d + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
#pragma unroll
    for (int w = 1; w < 32; ++w) s += sums[w][lane];
    dw[c] = accumulate ? dw[c] + s : s;
  }
}

int back_warps(int d) { return (d + 511) / 512; }
// CTAs of the backward: fixed by the row count and length and by the types, so
// that dw's order is.  As many as run at once (16384 x 4096: 87 us, 124 with a
// quarter more): with bf16 gradients 20 warps per
// SM (16384 x 2048: 44 us, with 16 49, with 24 56), with FP32 ones 16 (20: 85 us, 16 68).
int back_grid(int rows, int d, bool bf16) {
  return std::min(rows, 152 * std::max(1, (bf16 ? 20 : 16) / back_warps(d)));
}

// --------------------------------------------------------------- SiLU-mul ----
// Half a warp per (row, 128-wide group of gate and of up), 8 values a lane.
// Issue-bound as much as memory-bound: group indexes are 32-bit, and a row is
// found by a multiplication (with 64-bit divisions biv_silu_mul_keep_fp8 of
// 8192 x 6144 issued 56 instructions a column and took 94 us).

// n / d for n < 2^31 as (mulhi(n, m) + n) >> s (Granlund and Montgomery)
struct Divider {
  uint32_t m, d;
  int s;
};
Divider divider(uint32_t d) {
  int s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return {uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1), d, s};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divider& v) {
  return (__umulhi(n, v.m) + n) >> v.s;
}

// magnitudes of 8 gates and 8 ups: the largest of one half of a's words below,
// of b's above (`halves` picks the low or the high ones)
__device__ __forceinline__ __nv_bfloat162 largest(const uint4& a, const uint4& b, uint32_t halves) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
  __nv_bfloat162 p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = __byte_perm(u[i], v[i], halves);
    p[i] = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  }
  return __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
}

// (48 warps per SM: 75 us for 8192 x 6144; 40 took a tenth more; CTAs of 2 warps 100 us)
__global__ void __launch_bounds__(128, 12) silu_mul_keep_kernel(
    const uint16_t* __restrict__ gu, int64_t gs, uint32_t items, Divider by_groups, int I,
    uint8_t* __restrict__ keep, float* __restrict__ scales, uint16_t* __restrict__ y, int64_t ys) {
  pdl_wait();
  pdl_trigger();
  const int groups = int(by_groups.d);
  const uint32_t hw = blockIdx.x * 8u + (threadIdx.x >> 4);
  const int lane = threadIdx.x & 31;
  const bool on = hw < items;
  const uint32_t r = divide(on ? hw : 0, by_groups);
  const int64_t row = r;
  const int g = on ? int(hw - r * by_groups.d) : 0, c0 = g * 128 + (lane & 15) * 8;
  const bool live = on && c0 < I;
  float gv[8], uv[8];
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  if (live) {
    a = __ldg(reinterpret_cast<const uint4*>(gu + row * gs + c0));
    b = __ldg(reinterpret_cast<const uint4*>(gu + row * gs + I + c0));
  }
  unpack8(a, gv);
  unpack8(b, uv);
  // the largest magnitudes of gate and of up, bf16 as they are, in one register
  __nv_bfloat162 m = __hmax2(largest(a, b, 0x5410u), largest(a, b, 0x7632u));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
  // (a group of NaN alone has no largest value: 0, so that its scale is 1)
  m = __hmax2(m, __nv_bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)));
  const float most = __low2float(m);
  float sg, su;
  const uint2 kg = quant8(gv, most, sg), ku = quant8(uv, __high2float(m), su);
  if (!live) return;
  *reinterpret_cast<uint2*>(keep + row * 2 * I + c0) = kg;
  *reinterpret_cast<uint2*>(keep + row * 2 * I + I + c0) = ku;
  if ((lane & 15) == 0) {
    scales[row * 2 * groups + g] = sg;
    scales[row * 2 * groups + groups + g] = su;
  }
  if (y) {
    // gate / (1 + exp(-gate)): the divisor is at most exp(80), and Newton's step
    // for the reciprocal and Markstein's for the quotient give the division's
    // bits (for every bf16 gate; tested); groups with larger gates divide.
    float o[8];
    if (most < 80.0f) {
      const f32x2 one = pair(1.0f, 1.0f);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        // (with -1 / d and -gate the remainder's zero leaves the quotient's sign)
        const f32x2 g2 = pair(-gv[j], -gv[j + 1]), d = add2(one, pair(expf(-gv[j]), expf(-gv[j + 1])));
        float d0, d1;
        split(d, d0, d1);
        f32x2 r = pair(-rcp_approx(d0), -rcp_approx(d1));
        r = fma2(fma2(d, r, one), r, r);
        const f32x2 q = mul2(g2, r);
        split(mul2(fma2(fma2(d, q, g2), r, q), pair(uv[j], uv[j + 1])), o[j], o[j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = (gv[j] / (1.0f + expf(-gv[j]))) * uv[j];
    }
    *reinterpret_cast<uint4*>(y + row * ys + c0) = pack8(o);
  }
}

template <bool DYF, bool DGF>
__global__ void __launch_bounds__(128, 12) silu_mul_bwd_fp8_kernel(
    const uint8_t* __restrict__ keep, const float* __restrict__ scales, const void* __restrict__ dy,
    int64_t dys, uint32_t items, Divider by_groups, int I, void* __restrict__ dgu, int64_t dgs,
    uint16_t* __restrict__ y, int64_t ys) {
  pdl_wait();
  pdl_trigger();
  const int groups = int(by_groups.d);
  const uint32_t hw = blockIdx.x * 8u + (threadIdx.x >> 4);
  if (hw >= items) return;
  const uint32_t r = divide(hw, by_groups);
  const int64_t row = r;
  const int gi = int(hw - r * by_groups.d), c0 = gi * 128 + (threadIdx.x & 15) * 8;
  if (c0 >= I) return;
  const uint2 kg = __ldg(reinterpret_cast<const uint2*>(keep + row * 2 * I + c0));
  const uint2 ku = __ldg(reinterpret_cast<const uint2*>(keep + row * 2 * I + I + c0));
  const float sg = __ldg(scales + row * 2 * groups + gi);
  const float su = __ldg(scales + row * 2 * groups + groups + gi);
  float g[8], u[8], d[8], dg[8], du[8], o[8];
  load8<DYF>(dy, row * dys + c0, d);
  values4(kg.x, sg, g);
  values4(kg.y, sg, g + 4);
  values4(ku.x, su, u);
  values4(ku.y, su, u + 4);
  const f32x2 one = pair(1.0f, 1.0f), minus = pair(-1.0f, -1.0f);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const f32x2 g2 = pair(g[j], g[j + 1]), u2 = pair(u[j], u[j + 1]), d2 = pair(d[j], d[j + 1]);
    // FP32 gradients: biv_silu_mul_backward's division (at the copy rate with it).  bf16
    // ones: a sigmoid within 1 ulp, and 0 where it is below 2^-126 (gates below -87.3);
    // with divisions 8192 x 6144 took 78 us, now 73.
    const float d0 = 1.0f + expf(-g[j]), d1 = 1.0f + expf(-g[j + 1]);
    const f32x2 s = DGF ? pair(1.0f / d0, 1.0f / d1) : pair(rcp_approx(d0), rcp_approx(d1));
    const f32x2 a = mul2(g2, s);
    split(mul2(mul2(d2, u2), mul2(s, fma2(g2, fma2(s, minus, one), one))), dg[j], dg[j + 1]);
    split(mul2(d2, a), du[j], du[j + 1]);
    split(mul2(a, u2), o[j], o[j + 1]);
  }
  store8<DGF>(dgu, row * dgs + c0, dg);
  store8<DGF>(dgu, row * dgs + I + c0, du);
  if (y) *reinterpret_cast<uint4*>(y + row * ys + c0) = pack8(o);
}

bool row_ok(const void* p, int64_t stride, int64_t width, int size) {
  return p && aligned16(p) && stride >= width && stride * size % 16 == 0;
}
bool float_type(int t) { return t == BIV_F32 || t == BIV_BF16; }
int size_of(int t) { return t == BIV_F32 ? 4 : 2; }

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" {

biv_status biv_add_rmsnorm_fp8(const biv_norm_fp8_desc* d, biv_stream_t stream) {
  BIV_REQUIRE(d, "add_rmsnorm_fp8: null descriptor");
  BIV_REQUIRE(d->rows >= 0 && d->d > 0 && d->d % 16 == 0 && d->d <= 8192,
              "add_rmsnorm_fp8: rows=%d d=%d (d a multiple of 16, at most 8192)", d->rows, d->d);
  if (d->rows == 0) return BIV_OK;
  BIV_REQUIRE(row_ok(d->x, d->x_stride, d->d, 2) && d->w && aligned16(d->w),
              "add_rmsnorm_fp8: x or w null or misaligned");
  uint16_t* out = d->residual_out ? d->residual_out : const_cast<uint16_t*>(d->residual);
  const int64_t os = d->residual_out ? d->ro_stride : d->r_stride;
  BIV_REQUIRE(!d->residual || (row_ok(d->residual, d->r_stride, d->d, 2) && row_ok(out, os, d->d, 2)),
              "add_rmsnorm_fp8: residual misaligned");
  BIV_REQUIRE(d->residual || !d->residual_out, "add_rmsnorm_fp8: residual_out without a residual");
  BIV_REQUIRE(!d->y || row_ok(d->y, d->y_stride, d->d, 2), "add_rmsnorm_fp8: y misaligned");
  BIV_REQUIRE((d->codes == nullptr) == (d->scales == nullptr) && aligned16(d->codes),
              "add_rmsnorm_fp8: codes and scales go together, codes 16-byte aligned");
  BIV_REQUIRE((d->keep == nullptr) == (d->keep_scales == nullptr) && aligned16(d->keep),
              "add_rmsnorm_fp8: keep and keep_scales go together, keep 16-byte aligned");
  BIV_REQUIRE(d->y || d->codes, "add_rmsnorm_fp8: no output");
  NormArgs a;
  a.x = d->x; a.xs = d->x_stride;
  a.res = d->residual; a.rs = d->r_stride;
  a.res_out = out; a.ros = os;
  a.w = d->w;
  a.y = d->y; a.ys = d->y_stride;
  a.codes = d->codes; a.scales = d->scales;
  a.keep = d->keep; a.keep_scales = d->keep_scales;
  a.inv = d->inv;
  a.rows = d->rows; a.d = d->d; a.eps = d->eps;
  a.team = std::min(8, (d->d + 255) / 256);
  const int per = 8 / a.team;
  const unsigned grid = unsigned((d->rows + per - 1) / per);
  cudaStream_t s = as_cuda(stream);
  const int cpt = (d->d / 8 + 255) / 256;
  launch_pdl(cpt == 1   ? add_rmsnorm_fp8_kernel<1>
             : cpt == 2 ? add_rmsnorm_fp8_kernel<2>
             : cpt == 3 ? add_rmsnorm_fp8_kernel<3>
                        : add_rmsnorm_fp8_kernel<4>,
             grid, 32 * a.team * per, 0, s, a);
  return check_launch("add_rmsnorm_fp8");
}

biv_status biv_rmsnorm_backward_fp8_workspace(int rows, int d, size_t* bytes) {
  BIV_REQUIRE(bytes && rows >= 0 && d > 0 && d <= 8192, "rmsnorm_backward_fp8_workspace: bad arguments");
  *bytes = size_t(back_grid(rows, d, true)) * d * 4;
  return BIV_OK;
}

biv_status biv_rmsnorm_backward_fp8(const biv_norm_bwd_fp8_desc* d, biv_stream_t stream) {
  BIV_REQUIRE(d, "rmsnorm_backward_fp8: null descriptor");
  BIV_REQUIRE(d->rows >= 0 && d->d > 0 && d->d % 16 == 0 && d->d <= 8192,
              "rmsnorm_backward_fp8: rows=%d d=%d (d a multiple of 16, at most 8192)", d->rows, d->d);
  BIV_REQUIRE(float_type(d->dy_dtype) && float_type(d->dx_dtype),
              "rmsnorm_backward_fp8: gradients are bf16 or f32");
  BIV_REQUIRE(d->accumulate == 0 || d->accumulate == 1, "rmsnorm_backward_fp8: accumulate is 0 or 1");
  BIV_REQUIRE(d->dw, "rmsnorm_backward_fp8: null dw");
  const int grid = back_grid(d->rows, d->d, d->dy_dtype == BIV_BF16 && d->dx_dtype == BIV_BF16);
  cudaStream_t s = as_cuda(stream);
  if (d->rows > 0) {
    BIV_REQUIRE(d->keep && aligned16(d->keep) && d->keep_scales && d->inv && d->w && aligned16(d->w),
                "rmsnorm_backward_fp8: keep, scales, inv or w null or misaligned");
    BIV_REQUIRE(row_ok(d->dy, d->dy_stride, d->d, size_of(d->dy_dtype)) &&
                    row_ok(d->dx, d->dx_stride, d->d, size_of(d->dx_dtype)) &&
                    (!d->dres || row_ok(d->dres, d->dres_stride, d->d, size_of(d->dx_dtype))),
                "rmsnorm_backward_fp8: dy, dx and dres need 16-byte aligned rows");
    const size_t need = size_t(back_grid(d->rows, d->d, true)) * d->d * 4;
    if (!d->workspace || d->workspace_bytes < need)
      return set_error(BIV_ERR_WORKSPACE, "rmsnorm_backward_fp8: workspace of %zu bytes needed", need);
    BIV_REQUIRE(aligned16(d->workspace), "rmsnorm_backward_fp8: workspace must be 16-byte aligned");
    NormBackArgs a;
    a.keep = d->keep; a.scales = d->keep_scales; a.inv = d->inv; a.w = d->w;
    a.dy = d->dy; a.dys = d->dy_stride;
    a.dres = d->dres; a.drs = d->dres_stride;
    a.dx = d->dx; a.dxs = d->dx_stride;
    a.parts = static_cast<float*>(d->workspace);
    a.rows = d->rows; a.d = d->d;
    const bool yf = d->dy_dtype == BIV_F32, xf = d->dx_dtype == BIV_F32;
    const int threads = 32 * back_warps(d->d);
    if (yf)
      xf ? launch_back<true, true>(a, grid, threads, s) : launch_back<true, false>(a, grid, threads, s);
    else
      xf ? launch_back<false, true>(a, grid, threads, s) : launch_back<false, false>(a, grid, threads, s);
    biv_status st = check_launch("rmsnorm_backward_fp8");
    if (st != BIV_OK) return st;
  }
  launch_pdl(dw_sum_kernel, (d->d + 31) / 32, 1024, 0, s, static_cast<const float*>(d->workspace),
             d->rows > 0 ? grid : 0, d->d, d->dw, d->accumulate);
  return check_launch("rmsnorm_backward_fp8 dw");
}

biv_status biv_silu_mul_keep_fp8(const uint16_t* gate_up, int64_t gu_stride, uint16_t* y,
                                 int64_t y_stride, uint8_t* keep, float* keep_scales, int rows, int I,
                                 biv_stream_t stream) {
  BIV_REQUIRE(rows >= 0 && I > 0 && I % 16 == 0 && I <= (1 << 24), "silu_mul_keep_fp8: rows=%d I=%d (I %% 16)", rows, I);
  if (rows == 0) return BIV_OK;
  BIV_REQUIRE(row_ok(gate_up, gu_stride, int64_t(2) * I, 2) && (!y || row_ok(y, y_stride, I, 2)) && keep &&
                  aligned16(keep) && keep_scales,
              "silu_mul_keep_fp8: null or misaligned pointer");
  const Divider groups = divider(uint32_t((I + 127) / 128));
  const int64_t items = int64_t(rows) * groups.d;
  BIV_REQUIRE(items < (int64_t(1) << 31), "silu_mul_keep_fp8: 2^31 groups of 128 or more");
  launch_pdl(silu_mul_keep_kernel, unsigned((items + 7) / 8), 128, 0, as_cuda(stream), gate_up, gu_stride,
             uint32_t(items), groups, I, keep, keep_scales, y, y_stride);
  return check_launch("silu_mul_keep_fp8");
}

biv_status biv_silu_mul_backward_fp8(const uint8_t* keep, const float* keep_scales, const void* dy,
                                     int64_t dy_stride, int dy_dtype, void* dgate_up,
                                     int64_t dgate_up_stride, int dgate_up_dtype, uint16_t* y,
                                     int64_t y_stride, int rows, int I, biv_stream_t stream) {
  BIV_REQUIRE(rows >= 0 && I > 0 && I % 16 == 0 && I <= (1 << 24), "silu_mul_backward_fp8: rows=%d I=%d (I %% 16)", rows, I);
  BIV_REQUIRE(float_type(dy_dtype) && float_type(dgate_up_dtype),
              "silu_mul_backward_fp8: gradients are bf16 or f32");
  if (rows == 0) return BIV_OK;
  BIV_REQUIRE(keep && aligned16(keep) && keep_scales && row_ok(dy, dy_stride, I, size_of(dy_dtype)) &&
                  row_ok(dgate_up, dgate_up_stride, int64_t(2) * I, size_of(dgate_up_dtype)) &&
                  (!y || row_ok(y, y_stride, I, 2)),
              "silu_mul_backward_fp8: null or misaligned pointer");
  const Divider groups = divider(uint32_t((I + 127) / 128));
  const int64_t items = int64_t(rows) * groups.d;
  BIV_REQUIRE(items < (int64_t(1) << 31), "silu_mul_backward_fp8: 2^31 groups of 128 or more");
  const bool yf = dy_dtype == BIV_F32, gf = dgate_up_dtype == BIV_F32;
  launch_pdl(yf ? (gf ? silu_mul_bwd_fp8_kernel<true, true> : silu_mul_bwd_fp8_kernel<true, false>)
                : (gf ? silu_mul_bwd_fp8_kernel<false, true> : silu_mul_bwd_fp8_kernel<false, false>),
             unsigned((items + 7) / 8), 128, 0, as_cuda(stream), keep, keep_scales, dy, dy_stride,
             uint32_t(items), groups, I, dgate_up, dgate_up_stride, y, y_stride);
  return check_launch("silu_mul_backward_fp8");
}

}  // extern "C"
