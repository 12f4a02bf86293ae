// Clipped policy loss with a KL term, forward and backward in one call, from
// per-token logprobs or from the logits.
//
// Per token (w its weight, A its advantage):
//   r = exp(lp - old), pg = max(-A r, -A clip(r)), kl = exp(ref - lp) - (ref - lp) - 1
//   loss = sum w (pg + beta kl - gamma H), dlp = w (taken ? -A r : 0 + beta (1 - exp(ref - lp)))
// From logits (x = z / temperature, p = softmax x):
//   dz_v = (dlp ([v = target] - p_v) + w gamma p_v (log p_v + H)) / temperature
//
// Launches: policy_prep_kernel (one cluster) counts the rows of each sequence
// and turns them into a weight and an advantage per row; the logits kernel
// writes lp, H and dz row by row; policy_token_kernel sums the loss (and, when
// it starts from logprobs, writes dlp), its last block adding the blocks up.
#include <algorithm>
#include <mutex>

#include "common.cuh"

namespace biv {
namespace {

constexpr int kPrepThreads = 1024;
constexpr int kPrepCtas = 8;       // one cluster
constexpr int kTB = 256;           // threads per block of tokens
constexpr int kTok = 1024;         // tokens per partial sum
constexpr int kStat = 8;           // floats per partial sum
constexpr float kFar = 20.0f;      // log ratios are clamped to [-kFar, kFar]

__device__ __forceinline__ float warp_sum_x(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) { return (b > a || b != b) ? b : a; }
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float clamp_far(float x) { return x < -kFar ? -kFar : x > kFar ? kFar : x; }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (not .aligned: the threads of a warp may arrive apart)
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// 16-byte store to the same shared-memory address of CTA `rank` of the cluster
__device__ __forceinline__ void st_cluster_v4(uint32_t saddr, uint32_t rank, float a, float b, float c,
                                              float d) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %0, %1;\n\t"
      "st.shared::cluster.v4.f32 [ra], {%2, %3, %4, %5};\n\t}" ::"r"(saddr), "r"(rank), "f"(a), "f"(b),
      "f"(c), "f"(d)
      : "memory");
}

// ------------------------------------------------------------- workspace --
struct Totals {
  int rows, seqs;      // counted rows; sequences that have some
  unsigned ticket;     // blocks of the token kernel that are done
  int pad;
};
struct PolicyWs {
  Totals* totals;
  int* counts;         // [nseq]
  float2* row;         // [T] weight (0: the row does not count) and advantage
  float* part;         // [blocks, kStat]
};
int64_t token_blocks(int T) { return (int64_t(T) + kTok - 1) / kTok; }
size_t round16(size_t n) { return (n + 15) & ~size_t(15); }
size_t policy_ws_bytes(int T, int nseq) {
  return sizeof(Totals) + round16(size_t(nseq) * 4) + round16(size_t(T) * 8) +
         size_t(token_blocks(T)) * kStat * 4;
}
PolicyWs policy_ws(void* p, int T, int nseq) {
  uint8_t* b = static_cast<uint8_t*>(p);
  PolicyWs w;
  w.totals = reinterpret_cast<Totals*>(b);
  b += sizeof(Totals);
  w.counts = reinterpret_cast<int*>(b);
  b += round16(size_t(nseq) * 4);
  w.row = reinterpret_cast<float2*>(b);
  b += round16(size_t(T) * 8);
  w.part = reinterpret_cast<float*>(b);
  return w;
}

struct PolicyArgs {
  int T, nseq;
  const int32_t* seq_start;
  const uint8_t* mask;
  const float* old_lp;
  const float* ref_lp;
  const float* adv;
  int adv_per_row;
  float lo, hi, dual, beta, gamma;   // lo = 1 - clip_lo, hi = 1 + clip_hi
  int reduce;
  float norm;
  float* stats;
  PolicyWs ws;
  int* err;
};

// ------------------------------------------------------------------ prep --
// the sequence that row t may belong to: the last s < nseq with seq_start[s] <=
// t (-1: none); it does when also t < seq_start[s + 1]
__device__ __forceinline__ int find_seq(const int32_t* start, int nseq, int t) {
  int lo = -1, hi = nseq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// 16 mask bytes from row t on as bits (rows past T: 0)
__device__ __forceinline__ uint32_t mask16(const PolicyArgs& a, int t) {
  const int left = a.T - t;
  if (left <= 0) return 0;
  const uint32_t in = left >= 16 ? 0xFFFFu : (1u << left) - 1u;
  if (!a.mask) return in;
  uint32_t bits = 0;
  if (left >= 16 && (reinterpret_cast<uintptr_t>(a.mask + t) & 15) == 0) {
    const uint4 v = *reinterpret_cast<const uint4*>(a.mask + t);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((w[i >> 2] >> (8 * (i & 3))) & 0xFFu) bits |= 1u << i;
  } else {
    for (int i = 0; i < 16 && i < left; ++i)
      if (a.mask[t + i]) bits |= 1u << i;
  }
  return bits & in;
}

// One cluster: counts per sequence (integer adds: any order gives the same),
// totals, then every row's weight and advantage.
__global__ void __launch_bounds__(kPrepThreads) policy_prep_kernel(const __grid_constant__ PolicyArgs a) {
  __shared__ int s_red[2][kPrepThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int gt = blockIdx.x * kPrepThreads + threadIdx.x, nt = gridDim.x * kPrepThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int s = gt; s < a.nseq; s += nt) {
    a.ws.counts[s] = 0;
    const int b = a.seq_start[s], e = a.seq_start[s + 1];
    if (b < 0 || e < b || e > a.T) raise_error(a.err, kErrBadIndex);
  }
  cluster_sync();
  // 16 rows per lane; the loop's condition is the same for a whole warp
  for (int64_t t0 = int64_t(gt) * 16; t0 - int64_t(lane) * 16 < a.T; t0 += int64_t(nt) * 16) {
    const int t = int(t0 < a.T ? t0 : a.T);
    const uint32_t bits = mask16(a, t);
    int s = find_seq(a.seq_start, a.nseq, t);
    int end = s >= 0 ? a.seq_start[s + 1] : (a.nseq > 0 ? a.seq_start[0] : a.T);
    // a warp inside one sequence adds once
    const bool whole = s >= 0 && (t >= a.T || end >= min(t + 16, a.T));
    const int s0 = __shfl_sync(0xffffffffu, s, 0);
    if (__all_sync(0xffffffffu, t >= a.T || (whole && s == s0)) && s0 >= 0) {
      const int c = __reduce_add_sync(0xffffffffu, t < a.T ? __popc(bits) : 0);
      if (lane == 0 && c) atomicAdd(a.ws.counts + s0, c);
    } else if (t < a.T) {
      int c = 0;
      for (int i = 0; i < 16 && t + i < a.T; ++i) {
        while (t + i >= end && s < a.nseq) {   // the next sequence that reaches past this row
          if (s >= 0 && c) atomicAdd(a.ws.counts + s, c);
          c = 0;
          ++s;
          end = s < a.nseq ? a.seq_start[s + 1] : a.T;
        }
        if (s >= 0 && s < a.nseq && ((bits >> i) & 1u)) ++c;
      }
      if (s >= 0 && s < a.nseq && c) atomicAdd(a.ws.counts + s, c);
    }
    __syncwarp();
  }
  cluster_sync();
  int n = 0, k = 0;
  for (int s = threadIdx.x; s < a.nseq; s += kPrepThreads) {
    const int c = __ldcg(a.ws.counts + s);
    n += c;
    k += c > 0;
  }
  __syncwarp();
  n = __reduce_add_sync(0xffffffffu, n);
  k = __reduce_add_sync(0xffffffffu, k);
  if (lane == 0) {
    s_red[0][warp] = n;
    s_red[1][warp] = k;
  }
  __syncthreads();
  n = __reduce_add_sync(0xffffffffu, s_red[0][lane]);
  k = __reduce_add_sync(0xffffffffu, s_red[1][lane]);
  if (gt == 0) {
    a.ws.totals->rows = n;
    a.ws.totals->seqs = k;
    a.ws.totals->ticket = 0;
  }
  const float wt = a.reduce == BIV_LOSS_SUM ? 1.0f / a.norm : 1.0f / float(max(n, 1));
  for (int64_t t0 = int64_t(gt) * 4; t0 < a.T; t0 += int64_t(nt) * 4) {
    int s = find_seq(a.seq_start, a.nseq, int(t0));
    for (int i = 0; i < 4 && t0 + i < a.T; ++i) {
      const int t = int(t0) + i;
      while (s + 1 < a.nseq && a.seq_start[s + 1] <= t) ++s;
      float2 o = make_float2(0.f, 0.f);
      if (s >= 0 && t < a.seq_start[s + 1] && (!a.mask || a.mask[t])) {
        o.x = a.reduce == BIV_LOSS_SEQ_MEAN
                  ? 1.0f / (float(k) * float(max(__ldcg(a.ws.counts + s), 1)))
                  : wt;
        o.y = a.adv[a.adv_per_row ? t : s];
      }
      a.ws.row[t] = o;
    }
  }
}

// ------------------------------------------------------------- one token --
struct Token {
  float pg, kl, k3, gap;   // k3: exp(d) - 1 - d of the behaviour policy
  float dlp;               // without the weight
  bool cut;
};
// old, ref: the row's entries (not used where the caller gave none)
__device__ __forceinline__ Token policy_token(const PolicyArgs& a, float lp, float A, float old,
                                              float ref) {
  Token o;
  o.gap = a.old_lp ? lp - old : (lp == lp ? 0.f : lp);
  const float d = clamp_far(o.gap);
  const float r = expf(d);
  const float u = -A * r;
  const float rc = r < a.lo ? a.lo : r > a.hi ? a.hi : r;
  const float c = -A * rc;
  bool taken = u >= c;
  o.pg = taken ? u : c;
  if (a.dual > 0.f && A < 0.f && o.pg > -A * a.dual) {
    o.pg = -A * a.dual;
    taken = false;
  }
  o.cut = !taken;
  o.dlp = taken && fabsf(o.gap) < kFar ? u : 0.f;
  o.k3 = expm1f(d) - d;
  o.kl = 0.f;
  if (a.ref_lp) {
    const float far = ref - lp, q = clamp_far(far), em = expm1f(q);
    o.kl = em - q;
    if (!(fabsf(far) >= kFar)) o.dlp -= a.beta * em;
  }
  return o;
}

// Tokens [1024 blk, 1024 blk + 1024): dlp (when asked for) and the block's
// partial sums; thread i takes tokens 4i..4i+3 in order, then a warp xor tree
// and the warps in order.
__device__ __forceinline__ void policy_block(const PolicyArgs& a, const float* lp, const float* ent,
                                             float* dlp, int64_t blk, int tid, float (*red)[kStat]) {
  float v[kStat] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = blk * kTok + tid * 4 + i;
    if (t < a.T) {
      const float2 wa = a.ws.row[t];
      float g = 0.f;
      if (wa.x > 0.f) {
        const Token o = policy_token(a, lp[t], wa.y, a.old_lp ? a.old_lp[t] : 0.f,
                                     a.ref_lp ? a.ref_lp[t] : 0.f);
        const float h = ent ? ent[t] : 0.f;
        g = wa.x * o.dlp;
        v[0] += wa.x * (o.pg + a.beta * o.kl - a.gamma * h);
        v[1] += wa.x * o.pg;
        v[2] += wa.x * o.kl;
        v[3] += wa.x * h;
        v[4] += o.cut ? 1.f : 0.f;
        v[5] += o.k3;
        v[6] = max_nan(v[6], fabsf(o.gap));
      }
      if (dlp) dlp[t] = g;
    }
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 6; ++k) v[k] = warp_sum_x(v[k]);
  v[6] = warp_max_nan(v[6]);
  __syncthreads();
  if ((tid & 31) == 0) {
#pragma unroll
    for (int k = 0; k < 7; ++k) red[tid >> 5][k] = v[k];
  }
  __syncthreads();
  if (tid < 7) {
    float s = red[0][tid];
    for (int i = 1; i < kTB / 32; ++i) s = tid == 6 ? max_nan(s, red[i][tid]) : s + red[i][tid];
    a.ws.part[blk * kStat + tid] = s;
  }
}

// all blocks, by one warp: lane l takes blocks l, l + 32, ... in order
__device__ __forceinline__ void policy_final(const PolicyArgs& a, int64_t blocks, int lane) {
  float v[kStat] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t b = lane; b < blocks; b += 32) {
    const float4* p = reinterpret_cast<const float4*>(a.ws.part + b * kStat);
    const float4 x = __ldcg(p), y = __ldcg(p + 1);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] = max_nan(v[6], y.z);
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 6; ++k) v[k] = warp_sum_x(v[k]);
  v[6] = warp_max_nan(v[6]);
  if (lane == 0) {
    const int n = a.ws.totals->rows;
    const float inv = 1.0f / float(max(n, 1));
    a.stats[0] = v[0]; a.stats[1] = v[1]; a.stats[2] = v[2]; a.stats[3] = v[3];
    a.stats[4] = v[4] * inv;
    a.stats[5] = v[5] * inv;
    a.stats[6] = v[6];
    a.stats[7] = float(n);
  }
}

__global__ void __launch_bounds__(kTB) policy_token_kernel(const __grid_constant__ PolicyArgs a,
                                                           const float* lp, const float* ent,
                                                           float* dlp, int64_t blocks) {
  __shared__ float red[kTB / 32][kStat];
  __shared__ bool s_last;
  pdl_wait();
  pdl_trigger();
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x)
    policy_block(a, lp, ent, dlp, b, threadIdx.x, red);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(&a.ws.totals->ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (s_last && threadIdx.x < 32) {
    __threadfence();
    policy_final(a, blocks, threadIdx.x);
  }
}

// ---------------------------------------------------------------- logits --
// A cluster of CTAs holds one row of logits in shared memory, 1024 logits
// (one group) per buffer; each warp owns its groups' buffers and their
// mbarriers.  Per row: a warp reduces each group to (max, sum, entropy sum)
// as it arrives and writes the triple to every CTA of the cluster; after one
// cluster barrier each warp merges all groups, forms the token's gradient and
// writes its groups' dz straight from shared memory, refilling each buffer
// with the next row's logits as soon as it is done with it.  So logits are
// read once, dz is written once, and the next row streams in while this one is
// written.  A group's arithmetic and the merge order do not depend on the
// cluster size.
constexpr int kGroup = 1024;
constexpr int kMaxWarps = 20;
constexpr int kMaxV = 262144;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct LogitsArgs {
  PolicyArgs p;
  const void* z;
  int64_t ld;
  const int32_t* target;
  int V, G, gpc;            // groups of a row, groups per CTA
  float it, c;              // 1 / temperature, and that times log2(e)
  float* lp;
  float* ent;
  void* dz;
  int64_t ldz;
  int dz_vec;               // dz rows keep 4 elements' alignment
};

// one group of a row from shared memory (SHIFT: its elements are aligned to
// their own size only)
template <bool ZB, bool SHIFT>
__device__ __forceinline__ void read_group(const uint8_t* buf, int lane, float (&x)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = j * 128 + lane * 4;
    if constexpr (ZB) {
      uint32_t w0, w1;
      if constexpr (SHIFT) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(buf) + e;
        w0 = p[0] | (uint32_t(p[1]) << 16);
        w1 = p[2] | (uint32_t(p[3]) << 16);
      } else {
        const uint2 r = *reinterpret_cast<const uint2*>(buf + e * 2);
        w0 = r.x; w1 = r.y;
      }
      x[4 * j] = __uint_as_float(w0 << 16);
      x[4 * j + 1] = __uint_as_float(w0 & 0xFFFF0000u);
      x[4 * j + 2] = __uint_as_float(w1 << 16);
      x[4 * j + 3] = __uint_as_float(w1 & 0xFFFF0000u);
    } else if constexpr (SHIFT) {
      const float* p = reinterpret_cast<const float*>(buf) + e;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * j + i] = p[i];
    } else {
      const float4 r = *reinterpret_cast<const float4*>(buf + e * 4);
      x[4 * j] = r.x; x[4 * j + 1] = r.y; x[4 * j + 2] = r.z; x[4 * j + 3] = r.w;
    }
  }
}

template <bool ZB, bool DB, bool SHIFT>
__global__ void __launch_bounds__(kMaxWarps * 32) policy_logits_kernel(
    const __grid_constant__ LogitsArgs a) {
  constexpr int ES = ZB ? 2 : 4;
  constexpr int GB = kGroup * ES;
  constexpr int BUF = GB + (SHIFT ? 16 : 0);
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* bufs = smem;
  float4* stats = reinterpret_cast<float4*>(smem + size_t(a.gpc) * BUF);   // [2][G]
  uint64_t* bars = reinterpret_cast<uint64_t*>(stats + 2 * a.G);           // [gpc]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  uint32_t ncta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  const int rank = int(cluster_rank());
  const int clusters = int(gridDim.x / ncta), me = int(blockIdx.x / ncta);
  const int g0 = rank * a.gpc, mine = max(0, min(a.gpc, a.G - g0));

  if (tid == 0) {
    for (int i = 0; i < a.gpc; ++i) mbar_init(smem_u32(bars + i), 1);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_trigger();
  cluster_sync();

  auto counted = [&](int r) { return a.p.ws.row[r].x > 0.f; };
  auto next_row = [&](int r) {
    while (r < a.p.T && !counted(r)) r += clusters;
    return r;
  };
  auto row_ptr = [&](int r) { return static_cast<const uint8_t*>(a.z) + int64_t(r) * a.ld * ES; };
  // start the copy of this CTA's group i of row r: the 16-byte units that lie
  // in the row; what is left of the row's first and last unit is read later
  auto load_group = [&](int r, int i) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(row_ptr(r)), e = b + size_t(a.V) * ES;
    const uintptr_t gb = b + size_t(g0 + i) * GB;
    const uintptr_t ge = min(gb + GB, e);
    uintptr_t lo = gb & ~uintptr_t(15), hi = (ge + 15) & ~uintptr_t(15);
    if (lo < b) lo += 16;
    if (hi > e) hi -= 16;
    uint8_t* dst = bufs + size_t(i) * BUF + (lo - (gb & ~uintptr_t(15)));
    const uint32_t bar = smem_u32(bars + i);
    const uint32_t bytes = hi > lo ? uint32_t(hi - lo) : 0u;
    mbar_expect_tx(bar, bytes);
    if (bytes) bulk_load(smem_u32(dst), reinterpret_cast<const void*>(lo), bytes, bar);
  };

  int row = me;
  int ahead = next_row(me);      // the counted row whose loads are in flight
  if (ahead < a.p.T && lane == 0)
    for (int i = warp; i < mine; i += nw) load_group(ahead, i);
  __syncwarp();
  uint32_t phase = 0;
  for (; row < a.p.T; row += clusters) {
    if (row != ahead) {          // a row that does not count: zeros
      if (a.dz) {
        for (int i = warp; i < mine; i += nw)
          for (int j = lane; j < kGroup && (g0 + i) * kGroup + j < a.V; j += 32) {
            const int64_t at = int64_t(row) * a.ldz + (g0 + i) * kGroup + j;
            if (DB) static_cast<uint16_t*>(a.dz)[at] = 0;
            else static_cast<float*>(a.dz)[at] = 0.f;
          }
      }
      if (rank == 0 && tid == 0) {
        a.lp[row] = 0.f;
        a.ent[row] = 0.f;
      }
      continue;
    }
    const int nxt = next_row(row + clusters);
    const float2 wa = a.p.ws.row[row];
    const int tg = a.target[row];
    const float old = a.p.old_lp ? a.p.old_lp[row] : 0.f, ref = a.p.ref_lp ? a.p.ref_lp[row] : 0.f;
    const bool tg_ok = tg >= 0 && tg < a.V;
    float zt = 0.f;
    if (tg_ok) {
      if (ZB) zt = bf2f(reinterpret_cast<const uint16_t*>(row_ptr(row))[tg]);
      else zt = reinterpret_cast<const float*>(row_ptr(row))[tg];
    }
    const int off = SHIFT ? int(reinterpret_cast<uintptr_t>(row_ptr(row)) & 15) : 0;
    float4* st = stats + (phase & 1) * a.G;

    // ---- each group: (max, sum, entropy sum) relative to its own max
    for (int i = warp; i < mine; i += nw) {
      const int g = g0 + i;
      uint8_t* buf = bufs + size_t(i) * BUF + off;
      mbar_wait(smem_u32(bars + i), phase & 1, a.p.err);
      const int left = min(kGroup, a.V - g * kGroup);
      if (g * kGroup + left + 16 / ES > a.V || (SHIFT && g == 0)) {
        // elements of the row's first and last 16-byte unit, where it holds
        // bytes outside the row: not part of any copy
        const uint8_t* src = row_ptr(row);
        const uintptr_t b = reinterpret_cast<uintptr_t>(src), e = b + size_t(a.V) * ES;
        auto fetch = [&](int idx) {
          uint8_t* d = buf + (idx - g * kGroup) * ES;
          if (ZB) *reinterpret_cast<uint16_t*>(d) = reinterpret_cast<const uint16_t*>(src)[idx];
          else *reinterpret_cast<float*>(d) = reinterpret_cast<const float*>(src)[idx];
        };
        if (lane < 16 / ES) {
          const int tail = a.V - 1 - lane;
          if (tail >= g * kGroup && tail < g * kGroup + left && b + size_t(tail) * ES >= (e & ~uintptr_t(15)))
            fetch(tail);
          if (SHIFT && g == 0 && lane < left && (b & 15) && (b & 15) + lane * ES < 16) fetch(lane);
        }
        __syncwarp();
      }
      float x[32];
      read_group<ZB, SHIFT>(buf, lane, x);
      if (left < kGroup) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if ((j >> 2) * 128 + lane * 4 + (j & 3) >= left) x[j] = -INFINITY;
      }
      float m = x[0];
#pragma unroll
      for (int j = 1; j < 32; ++j) m = fmaxf(m, x[j]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float mc = m * a.c;
      float s = 0.f, t = 0.f;
      if (m > -INFINITY) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float y = fmaf(x[j], a.c, -mc);
          const float e = ex2f(y);
          s += e;
          t = fmaf(e, y < -1000.f ? 0.f : y, t);
        }
        s = warp_sum_x(s);
        t = warp_sum_x(t);
      } else {
        bool bad = false;          // only -inf, or NaN among it
#pragma unroll
        for (int j = 0; j < 32; ++j) bad |= x[j] != x[j];
        if (__any_sync(0xffffffffu, bad)) s = t = NAN;
      }
      if (lane < ncta) st_cluster_v4(smem_u32(st + g), lane, mc, s, t, 0.f);
    }
    cluster_sync();

    // ---- merge: lane l takes groups l, l + 32, ... in order
    float M = -INFINITY;
    for (int g = lane; g < a.G; g += 32) M = fmaxf(M, st[g].x);
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float S = 0.f, U = 0.f;
    for (int g = lane; g < a.G; g += 32) {
      const float4 q = st[g];
      if (q.x == -INFINITY) {
        S += q.y;                  // 0, or the NaN of a group without a number
      } else {
        const float d = q.x - M, f = ex2f(d);
        S = fmaf(q.y, f, S);
        U = fmaf(f, fmaf(q.y, fmaxf(d, -1000.f), q.z), U);
      }
    }
    __syncwarp();
    S = warp_sum_x(S);
    U = warp_sum_x(U);
    if (M == -INFINITY) S = NAN;   // no finite logit
    constexpr float kLn2 = 0.6931471805599453f;
    const float lnS = logf(S);
    const float H = lnS - kLn2 * (U / S);
    const float lp = tg_ok ? fmaf(zt, a.c, -M) * kLn2 - lnS : NAN;
    if (rank == 0 && tid == 0) {
      a.lp[row] = lp;
      a.ent[row] = H;
      if (!tg_ok) raise_error(a.p.err, kErrBadIndex);
    }

    // ---- dz = p (a0 + a1 y) (+ it dlp at the target), y = log2 of p S
    float a0 = 0.f, a1 = 0.f, at_target = 0.f;
    if (a.dz) {
      const Token o = policy_token(a.p, lp, wa.y, old, ref);
      const float dlp = wa.x * o.dlp, wg = wa.x * a.p.gamma, is = a.it / S;
      a0 = is * (wg * (H - lnS) - dlp);
      a1 = is * wg * kLn2;
      at_target = a.it * dlp;
    }
    for (int i = warp; i < mine; i += nw) {
      const int g = g0 + i;
      if (a.dz) {
        uint8_t* buf = bufs + size_t(i) * BUF + off;
        const int left = min(kGroup, a.V - g * kGroup);
        float x[32];
        read_group<ZB, SHIFT>(buf, lane, x);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float y = fmaf(x[j], a.c, -M);
          const float e = ex2f(y);
          x[j] = e * fmaf(a1, y < -1000.f ? 0.f : y, a0);
        }
        const int tl = tg - g * kGroup;     // the target inside this group
        if (tl >= 0 && tl < kGroup && ((tl >> 2) & 31) == lane) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if ((j >> 2) * 128 + lane * 4 + (j & 3) == tl) x[j] += at_target;
        }
        const int64_t base = int64_t(row) * a.ldz + g * kGroup;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = j * 128 + lane * 4;
          if (DB) {
            uint16_t* d = static_cast<uint16_t*>(a.dz) + base + e;
            if (a.dz_vec && e + 4 <= left) {
              *reinterpret_cast<uint2*>(d) =
                  make_uint2(pack_bf2(x[4 * j], x[4 * j + 1]), pack_bf2(x[4 * j + 2], x[4 * j + 3]));
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (e + k < left) d[k] = f2bf(x[4 * j + k]);
            }
          } else {
            float* d = static_cast<float*>(a.dz) + base + e;
            if (a.dz_vec && e + 4 <= left) {
              *reinterpret_cast<float4*>(d) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (e + k < left) d[k] = x[4 * j + k];
            }
          }
        }
      }
      if (nxt < a.p.T) {
        fence_proxy_async();       // this warp's accesses to the buffer come first
        __syncwarp();
        if (lane == 0) load_group(nxt, i);
        __syncwarp();
      }
    }
    ahead = nxt;
    ++phase;
  }
  cluster_sync();   // no CTA leaves while another may still write its statistics
}

// -------------------------------------------------------------- host side --
biv_status check_policy(const biv_policy_desc* d, const char* who) {
  BIV_REQUIRE(d, "%s: null descriptor", who);
  BIV_REQUIRE(d->T >= 0 && d->nseq >= 0 && d->T <= (1 << 30), "%s: bad sizes", who);
  if (d->T == 0) return BIV_OK;
  BIV_REQUIRE(d->seq_start && d->adv && d->stats, "%s: null pointer", who);
  BIV_REQUIRE(d->clip_lo >= 0.f && d->clip_lo <= 1.f && d->clip_hi >= 0.f,
              "%s: clip_lo must lie in [0, 1] and clip_hi must not be negative", who);
  BIV_REQUIRE(d->dual_clip == 0.f || d->dual_clip > 1.f, "%s: dual_clip must be 0 or above 1", who);
  BIV_REQUIRE(d->kl_coef == d->kl_coef && d->ent_coef == d->ent_coef, "%s: a coefficient is NaN", who);
  BIV_REQUIRE(d->kl_coef == 0.f || d->ref_lp, "%s: a KL term needs ref_lp", who);
  BIV_REQUIRE(d->reduce >= BIV_LOSS_TOKEN_MEAN && d->reduce <= BIV_LOSS_SUM, "%s: unknown reduce", who);
  BIV_REQUIRE(d->reduce != BIV_LOSS_SUM || (d->norm > 0.f && d->norm < 3e38f),
              "%s: reduce SUM needs a positive finite norm", who);
  const size_t need = policy_ws_bytes(d->T, d->nseq);
  if (!d->workspace || d->workspace_bytes < need)
    return set_error(BIV_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", who, need);
  BIV_REQUIRE(aligned16(d->workspace), "%s: workspace must be 16-byte aligned", who);
  return BIV_OK;
}

PolicyArgs policy_args(const biv_policy_desc& d) {
  PolicyArgs a;
  a.T = d.T; a.nseq = d.nseq; a.seq_start = d.seq_start; a.mask = d.mask;
  a.old_lp = d.old_lp; a.ref_lp = d.ref_lp; a.adv = d.adv; a.adv_per_row = d.adv_per_row;
  a.lo = 1.0f - d.clip_lo; a.hi = 1.0f + d.clip_hi; a.dual = d.dual_clip;
  a.beta = d.kl_coef; a.gamma = d.ent_coef; a.reduce = d.reduce; a.norm = d.norm;
  a.stats = d.stats;
  a.ws = policy_ws(d.workspace, d.T, d.nseq);
  a.err = device_error_word();
  return a;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem,
                           unsigned cluster, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

biv_status launch_prep(const PolicyArgs& a, cudaStream_t s) {
  // a CTA per 4096 rows or 1024 sequences, at most one cluster
  const int64_t want = (std::max<int64_t>(a.T, int64_t(a.nseq) * 4) + 4095) / 4096;
  unsigned ctas = 1;
  while (ctas < unsigned(kPrepCtas) && int64_t(ctas) < want) ctas *= 2;
  launch_cluster(policy_prep_kernel, ctas, kPrepThreads, 0, ctas, s, a);
  return check_launch("policy_prep");
}

biv_status launch_tokens(const PolicyArgs& a, const float* lp, const float* ent, float* dlp,
                         cudaStream_t s) {
  const int64_t blocks = token_blocks(a.T);
  const int sms = sm_count() > 0 ? sm_count() : 148;
  const unsigned grid = unsigned(std::min<int64_t>(blocks, int64_t(sms) * 8));
  launch_pdl(policy_token_kernel, grid, kTB, 0, s, a, lp, ent, dlp, blocks);
  return check_launch("policy_tokens");
}

// clusters of this shape that fit the device at once (asked once per shape)
struct Shape {
  const void* kern;
  int dev;
  unsigned cluster, threads;
  size_t smem;
  int fit;
};
template <typename K>
biv_status max_clusters(K kern, unsigned cluster, unsigned threads, size_t smem, int* fit) {
  static std::mutex mu;
  static Shape cache[64];
  static int used = 0;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return set_error(BIV_ERR_CUDA, "policy_logits: no device");
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < used; ++i) {
    const Shape& c = cache[i];
    if (c.kern == reinterpret_cast<const void*>(kern) && c.dev == dev && c.cluster == cluster &&
        c.threads == threads && c.smem == smem) {
      *fit = c.fit;
      return BIV_OK;
    }
  }
  int most = 0;
  if (cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
    return set_error(BIV_ERR_CUDA, "policy_logits: cannot set the shared memory size: %s",
                     cudaGetErrorString(cudaGetLastError()));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1)
    return set_error(BIV_ERR_CUDA, "policy_logits: no cluster of %u CTAs fits: %s", cluster,
                     cudaGetErrorString(cudaGetLastError()));
  if (used < 64) cache[used++] = Shape{reinterpret_cast<const void*>(kern), dev, cluster, threads, smem, n};
  *fit = n;
  return BIV_OK;
}

constexpr size_t kRowBytesPerCta = 160 << 10;

template <bool ZB, bool DB, bool SHIFT>
biv_status launch_logits(LogitsArgs& a, cudaStream_t s) {
  constexpr int GB = kGroup * (ZB ? 2 : 4);
  const int sms = sm_count() > 0 ? sm_count() : 148;
  unsigned cl = 1;
  while (cl < 8 && size_t((a.G + cl - 1) / cl) * GB > kRowBytesPerCta) cl *= 2;
  // few rows: spread each over more SMs (no bit depends on it)
  while (cl < 8 && int(cl) * 2 <= a.G && int64_t(a.p.T) * cl * 2 <= sms) cl *= 2;
  a.gpc = int((a.G + cl - 1) / cl);
  const int per = (a.gpc + kMaxWarps - 1) / kMaxWarps;
  const unsigned threads = unsigned((a.gpc + per - 1) / per) * 32;
  const size_t smem = size_t(a.gpc) * (GB + (SHIFT ? 16 : 0)) + size_t(a.G) * 32 + size_t(a.gpc) * 8;
  int fit = 0;
  biv_status st = max_clusters(policy_logits_kernel<ZB, DB, SHIFT>, cl, threads, smem, &fit);
  if (st != BIV_OK) return st;
  const unsigned clusters = unsigned(std::min(a.p.T, fit));
  launch_cluster(policy_logits_kernel<ZB, DB, SHIFT>, clusters * cl, threads, smem, cl, s, a);
  return check_launch("policy_logits");
}

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" {

biv_status biv_policy_loss_workspace(int T, int nseq, size_t* bytes) {
  BIV_REQUIRE(T >= 0 && nseq >= 0 && bytes, "policy_loss_workspace: bad arguments");
  *bytes = policy_ws_bytes(T, nseq);
  return BIV_OK;
}

biv_status biv_policy_loss(const biv_policy_desc* d, const float* lp, float* dlp,
                           biv_stream_t stream) {
  biv_status st = check_policy(d, "policy_loss");
  if (st != BIV_OK || d->T == 0) return st;
  BIV_REQUIRE(lp, "policy_loss: null pointer");
  BIV_REQUIRE(d->ent_coef == 0.f, "policy_loss: an entropy term needs the logits");
  const PolicyArgs a = policy_args(*d);
  cudaStream_t s = as_cuda(stream);
  st = launch_prep(a, s);
  if (st != BIV_OK) return st;
  return launch_tokens(a, lp, nullptr, dlp, s);
}

biv_status biv_policy_loss_logits(const biv_policy_desc* d, const void* z, int64_t ld, int z_dtype,
                                  const int32_t* target, int V, float inv_temp, float* lp,
                                  float* entropy, void* dz, int64_t ldz, int dz_dtype,
                                  biv_stream_t stream) {
  biv_status st = check_policy(d, "policy_loss_logits");
  if (st != BIV_OK || d->T == 0) return st;
  BIV_REQUIRE(z && target && lp && entropy, "policy_loss_logits: null pointer");
  BIV_REQUIRE(V >= 1 && V <= kMaxV, "policy_loss_logits: V must lie in [1, %d]", kMaxV);
  BIV_REQUIRE((z_dtype == BIV_F32 || z_dtype == BIV_BF16) &&
                  (!dz || dz_dtype == BIV_F32 || dz_dtype == BIV_BF16),
              "policy_loss_logits: logits and gradient are f32 or bf16");
  BIV_REQUIRE(ld >= V && (!dz || ldz >= V), "policy_loss_logits: a row stride is below V");
  BIV_REQUIRE(inv_temp > 0.f && inv_temp < 3e38f, "policy_loss_logits: inv_temp must be positive and finite");
  const size_t es = z_dtype == BIV_F32 ? 4 : 2, ds = dz_dtype == BIV_F32 ? 4 : 2;
  const uintptr_t zb = reinterpret_cast<uintptr_t>(z), db = reinterpret_cast<uintptr_t>(dz);
  BIV_REQUIRE(zb % es == 0 && db % ds == 0, "policy_loss_logits: a pointer is not aligned to its elements");
  if (dz) {
    const uintptr_t ze = zb + (size_t(d->T - 1) * size_t(ld) + V) * es;
    const uintptr_t de = db + (size_t(d->T - 1) * size_t(ldz) + V) * ds;
    BIV_REQUIRE((zb == db && ld == ldz && z_dtype == dz_dtype) || ze <= db || de <= zb,
                "policy_loss_logits: dz must be the logits themselves or not overlap them");
  }
  LogitsArgs a;
  a.p = policy_args(*d);
  a.z = z; a.ld = ld; a.target = target; a.V = V;
  a.G = (V + kGroup - 1) / kGroup;
  a.gpc = 0;
  a.it = inv_temp;
  a.c = float(double(inv_temp) * 1.4426950408889634);
  a.lp = lp; a.ent = entropy; a.dz = dz; a.ldz = ldz;
  a.dz_vec = db % (4 * ds) == 0 && ldz % 4 == 0;
  const bool shift = zb % 16 != 0 || (size_t(ld) * es) % 16 != 0;
  cudaStream_t s = as_cuda(stream);
  st = launch_prep(a.p, s);
  if (st != BIV_OK) return st;
  const bool zbf = z_dtype == BIV_BF16, dbf = dz && dz_dtype == BIV_BF16;
  if (zbf) {
    st = dbf ? (shift ? launch_logits<true, true, true>(a, s) : launch_logits<true, true, false>(a, s))
             : (shift ? launch_logits<true, false, true>(a, s) : launch_logits<true, false, false>(a, s));
  } else {
    st = dbf ? (shift ? launch_logits<false, true, true>(a, s) : launch_logits<false, true, false>(a, s))
             : (shift ? launch_logits<false, false, true>(a, s) : launch_logits<false, false, false>(a, s));
  }
  if (st != BIV_OK) return st;
  return launch_tokens(a.p, lp, entropy, nullptr, s);
}

}  // extern "C"
