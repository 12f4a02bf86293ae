// Clipped policy loss with a KL term, forward and backward in one call, from
// per-token logprobs or from the logits.
//
// Per token (w its weight, A its advantage):
//   r = exp(lp - old), pg = max(-A r, -A clip(r)), kl = exp(ref - lp) - (ref - lp) - 1
//   loss = sum w (pg + beta kl - gamma H), dlp = w (taken ? -A r : 0 + beta (1 - exp(ref - lp)))
// From logits (x = z / temperature, p = softmax x):
//   dz_v = (dlp ([v = target] - p_v) + w gamma p_v (log p_v + H)) / temperature
//
// Launches.  Weights need the counted rows of each sequence first.  Up to 4096
// rows, one CTA does all of it (policy_small_kernel: from logprobs one launch;
// from logits one before the logits kernel, which writes lp, H and dz row by row
// and whose last CTA mostly sums the loss).  Above that the counts are launches
// before, and policy_token_kernel sums the loss, its last block adding the blocks up.
#include <algorithm>
#include <mutex>

#include "common.cuh"

namespace biv {
namespace {

constexpr int kSmallRows = 4096, kSmallSeqs = 1024;   // what one CTA takes
constexpr int kMidSeqs = 1024;                        // counts by a block per sequence
constexpr int64_t kMidMean = 1 << 17;                 // ... of this length on average at most
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

__device__ __forceinline__ bool aligned16_dev(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

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
  int mid;                           // a block per sequence counts; totals are not stored
  float* stats;
  PolicyWs ws;
  int* err;
};

// ------------------------------------------------------------------ rows --
// The sequence that row t may belong to: the last s < nseq with seq_start[s] <=
// t (-1: none); it does when also t < seq_start[s + 1].
// Looked for in [lo, hi]:
__device__ __forceinline__ int find_seq_between(const int32_t* start, int lo, int hi, int t) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// for rows ta <= tb, by a warp that looks at 32 starts at once
__device__ __forceinline__ void find_seqs_warp(const int32_t* start, int nseq, int ta, int tb, int& sa,
                                               int& sb) {
  const int lane = threadIdx.x & 31;
  int la = -1, ha = nseq, lb = -1, hb = nseq;     // start[la] <= ta < start[ha]
  while (ha - la > 1 || hb - lb > 1) {
    const int pa = (ha - la + 31) >> 5, pb = (hb - lb + 31) >> 5;
    const int ia = la + (lane + 1) * pa, ib = lb + (lane + 1) * pb;
    const int na = __popc(__ballot_sync(0xffffffffu, ia < ha && start[ia] <= ta));
    const int nb = __popc(__ballot_sync(0xffffffffu, ib < hb && start[ib] <= tb));
    la += na * pa;
    ha = min(ha, la + pa);
    lb += nb * pb;
    hb = min(hb, lb + pb);
  }
  sa = la;
  sb = lb;
}

// a thread's four consecutive rows t0..t0+3: the sequence of each that counts
// (-1: it does not).  Called by whole warps.
__device__ __forceinline__ void four_seqs(const PolicyArgs& a, const int32_t* start, int64_t t0,
                                          int (&seq)[4]) {
  const int64_t first = t0 - (threadIdx.x & 31) * 4;   // the warp's rows
  int sa, sb;
  find_seqs_warp(start, a.nseq, int(min(first, int64_t(a.T))), int(min(first + 127, int64_t(a.T))), sa, sb);
#pragma unroll
  for (int i = 0; i < 4; ++i) seq[i] = -1;
  if (t0 >= a.T) return;
  bool on[4];
  if (a.mask && t0 + 4 <= a.T && (reinterpret_cast<uintptr_t>(a.mask + t0) & 3) == 0) {
    const uint32_t m = *reinterpret_cast<const uint32_t*>(a.mask + t0);
#pragma unroll
    for (int i = 0; i < 4; ++i) on[i] = (m >> (8 * i)) & 0xFFu;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) on[i] = t0 + i < a.T && (!a.mask || a.mask[t0 + i]);
  }
  int s = find_seq_between(start, sa, max(sa, sb), int(t0));
  int end = s >= 0 ? start[s + 1] : 0;
  int next = s + 1 < a.nseq ? start[s + 1] : a.T;      // where the next sequence begins
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = int(t0) + i;
    while (t >= next && s + 1 < a.nseq) {
      ++s;
      end = start[s + 1];
      next = s + 1 < a.nseq ? end : a.T;
    }
    if (on[i] && s >= 0 && t < end) seq[i] = s;
  }
}

__device__ __forceinline__ float row_weight(const PolicyArgs& a, int rows, int seqs, int count) {
  if (a.reduce == BIV_LOSS_SUM) return 1.0f / a.norm;
  return 1.0f / (a.reduce == BIV_LOSS_SEQ_MEAN ? float(seqs) * float(max(count, 1)) : float(max(rows, 1)));
}

__device__ __forceinline__ void check_start(const PolicyArgs& a, int s) {
  const int b = a.seq_start[s], e = a.seq_start[s + 1];
  if (b < 0 || e < b || e > a.T) raise_error(a.err, kErrBadIndex);
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

// four consecutive values from t0 on (n: their number, 0 past it)
__device__ __forceinline__ void load4(const float* p, int64_t t0, int64_t n, float (&f)[4]) {
  if (t0 + 4 <= n && aligned16_dev(p)) {
    const float4 v = *reinterpret_cast<const float4*>(p + t0);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = t0 + i < n ? p[t0 + i] : 0.f;
}

// What a thread has of its four rows: weights (0: not counted), advantages and
// the inputs.
struct Four {
  float w[4], A[4], lp[4], old[4], ref[4], ent[4];
};
__device__ __forceinline__ void load_inputs(const PolicyArgs& a, const float* lp, const float* ent,
                                            int64_t t0, Four& f) {
  load4(lp, t0, a.T, f.lp);
#pragma unroll
  for (int i = 0; i < 4; ++i) f.old[i] = f.ref[i] = f.ent[i] = 0.f;
  if (a.old_lp) load4(a.old_lp, t0, a.T, f.old);
  if (a.ref_lp) load4(a.ref_lp, t0, a.T, f.ref);
  if (ent) load4(ent, t0, a.T, f.ent);
}

// A thread's four rows: dlp, and the sums over its warp's 128 rows (the thread's
// in order, then a xor tree).
__device__ __forceinline__ void policy_four(const PolicyArgs& a, const Four& f, float (&g)[4],
                                            float (&v)[kStat]) {
#pragma unroll
  for (int k = 0; k < kStat; ++k) v[k] = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[i] = 0.f;
    if (f.w[i] > 0.f) {
      const Token o = policy_token(a, f.lp[i], f.A[i], f.old[i], f.ref[i]);
      g[i] = f.lp[i] == -INFINITY ? 0.f : f.w[i] * o.dlp;   // (also where no old_lp is far from it)
      v[0] += f.w[i] * (o.pg + a.beta * o.kl - a.gamma * f.ent[i]);
      v[1] += f.w[i] * o.pg;
      v[2] += f.w[i] * o.kl;
      v[3] += f.w[i] * f.ent[i];
      v[4] += o.cut ? 1.f : 0.f;
      v[5] += o.k3;
      v[6] = max_nan(v[6], fabsf(o.gap));
    }
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 6; ++k) v[k] = warp_sum_x(v[k]);
  v[6] = warp_max_nan(v[6]);
}
// what the sums of the eight warps of 1024 rows add up to, in order: entry k
__device__ __forceinline__ float block_entry(const float (*red)[kStat], int k) {
  float s = red[0][k];
  for (int i = 1; i < kTB / 32; ++i) s = k == 6 ? max_nan(s, red[i][k]) : s + red[i][k];
  return s;
}
// dlp of the four rows (when asked for) and the sums over a block of 1024 rows.
// tid: the thread within its block of 256; `sync` joins those threads.
template <typename Sync>
__device__ __forceinline__ void policy_block(const PolicyArgs& a, const Four& f, float* dlp, int64_t t0,
                                             int tid, float (*red)[kStat], float* part, Sync sync) {
  float v[kStat], g[4];
  policy_four(a, f, g, v);
  if (dlp) {
    if (t0 + 4 <= a.T && aligned16_dev(dlp)) {
      *reinterpret_cast<float4*>(dlp + t0) = make_float4(g[0], g[1], g[2], g[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < a.T) dlp[t0 + i] = g[i];
    }
  }
  sync();
  if ((tid & 31) == 0) {
#pragma unroll
    for (int k = 0; k < 7; ++k) red[tid >> 5][k] = v[k];
  }
  sync();
  if (tid < 7) part[tid] = block_entry(red, tid);
}

// all blocks' sums (in shared or global memory), by one warp: lane l takes blocks
// l, l + 32, ... in order
template <bool SHARED>
__device__ __forceinline__ void policy_final(const PolicyArgs& a, const float* part, int64_t blocks,
                                             int rows, int lane) {
  float v[kStat] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int64_t b = lane; b < blocks; b += 32) {
    const float4* p = reinterpret_cast<const float4*>(part + b * kStat);
    const float4 x = SHARED ? p[0] : __ldcg(p), y = SHARED ? p[1] : __ldcg(p + 1);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] = max_nan(v[6], y.z);
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 6; ++k) v[k] = warp_sum_x(v[k]);
  v[6] = warp_max_nan(v[6]);
  if (lane == 0) {
    const float inv = 1.0f / float(max(rows, 1));
    a.stats[0] = v[0]; a.stats[1] = v[1]; a.stats[2] = v[2]; a.stats[3] = v[3];
    a.stats[4] = v[4] * inv;
    a.stats[5] = v[5] * inv;
    a.stats[6] = v[6];
    a.stats[7] = float(rows);
  }
}

// ----------------------------------------------------------- small calls --
// One CTA, four rows per thread (8 sequences of 150 rows: 4.0 us, a launch and two
// trips to memory); counts and starts in shared memory, the rows'
// inputs on their way meanwhile.  From logprobs: all of it; ROWS: weights and
// advantages for the logits kernel.
template <bool ROWS>
__global__ void __launch_bounds__(kSmallRows / 4) policy_small_kernel(
    const __grid_constant__ PolicyArgs a, const float* lp, float* dlp) {
  __shared__ int32_t s_start[kSmallSeqs + 1];
  __shared__ int s_count[kSmallSeqs], s_red[2][32];
  __shared__ float red[4][kTB / 32][kStat];
  __shared__ __align__(16) float part[4 * kStat];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int64_t t0 = int64_t(tid) * 4;
  Four f;
  if (!ROWS) load_inputs(a, lp, nullptr, t0, f);
  for (int s = tid; s <= a.nseq; s += nt) {
    s_start[s] = a.seq_start[s];
    if (s < a.nseq) {
      s_count[s] = 0;
      check_start(a, s);
    }
  }
  __syncthreads();
  int seq[4];
  four_seqs(a, s_start, t0, seq);
  const bool one = seq[0] >= 0 && seq[0] == seq[1] && seq[0] == seq[2] && seq[0] == seq[3];
  const int first = __shfl_sync(0xffffffffu, seq[0], 0);
  if (__all_sync(0xffffffffu, one && seq[0] == first)) {
    if (lane == 0) atomicAdd(s_count + first, 128);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (seq[i] >= 0) atomicAdd(s_count + seq[i], 1);
  }
  float adv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) adv[i] = seq[i] >= 0 ? a.adv[a.adv_per_row ? t0 + i : seq[i]] : 0.f;
  __syncthreads();
  int n = 0, k = 0;
  for (int s = tid; s < a.nseq; s += nt) {
    n += s_count[s];
    k += s_count[s] > 0;
  }
  __syncwarp();
  n = __reduce_add_sync(0xffffffffu, n);
  k = __reduce_add_sync(0xffffffffu, k);
  if (lane == 0) {
    s_red[0][warp] = n;
    s_red[1][warp] = k;
  }
  __syncthreads();
  const int rows = __reduce_add_sync(0xffffffffu, lane < nt / 32 ? s_red[0][lane] : 0);
  k = __reduce_add_sync(0xffffffffu, lane < nt / 32 ? s_red[1][lane] : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.w[i] = seq[i] >= 0 ? row_weight(a, rows, k, s_count[seq[i]]) : 0.f;
    f.A[i] = adv[i];
  }
  if (ROWS) {
    if (tid == 0) *a.ws.totals = Totals{rows, k, 0u, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + i < a.T) a.ws.row[t0 + i] = make_float2(f.w[i], f.A[i]);
    return;
  }
  const int grp = tid / kTB;           // blocks of 1024 rows: groups of 256 threads
  policy_block(a, f, dlp, t0, tid % kTB, red[grp], part + grp * kStat, [] { __syncthreads(); });
  __syncthreads();
  if (warp == 0) policy_final<true>(a, part, nt / kTB, rows, lane);
}

// ----------------------------------------------------------- large calls --
// Up to 1024 sequences of 131072 rows on average two launches: counts by a block
// per sequence, then the sums, each block adding the counts up for itself.  300 K
// rows in 512 ragged sequences take 10.6 us against 15.1 by the general way (a launch
// that zeroes the counts, rows that add to them, and the sums).  With a mask and an
// old logprob, this way against the general one (us):
//   131072 rows in 16 sequences 7.9 / 9.6;   524288 in 64 11.7 / 16.4
//   2^20 in 16 18.9 / 25.8, in 1024 19.0 / 21.8;   2^22 in 64 55 / 79, in 1024 57 / 67
//   2^24 in 256 239 / 317, in 1024 246 / 293;   2^26 in 1024 959 / 1239
// so the number of rows sets no limit.  Few long sequences leave most SMs idle: one
// of 524288 rows 20.4 / 17.0, one of 2^20 36 / 25, four of 2^22 372 / 319 (and so
// does one that holds nearly all rows, which the host cannot see).  Many have
// each block of the sums add many counts up: 4096 of 32 rows 12.5 / 11.5, 4096 of 256
// 23.9 / 23.4 (from 2^21 rows on they would gain too: 61 / 66 for 2^22).  A rollout's
// bytes are a few us at HBM's rate at most: the launches and the dependent loads of
// each (starts, counts, rows) take the time.
__global__ void policy_zero_kernel(const __grid_constant__ PolicyArgs a) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s == 0) *a.ws.totals = Totals{0, 0, 0u, 0};
  if (s < a.nseq) {
    a.ws.counts[s] = 0;
    check_start(a, s);
  }
}

// Counts per sequence and their totals (integer adds: any order gives the same)
__global__ void __launch_bounds__(kTB) policy_count_kernel(const __grid_constant__ PolicyArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t(blockIdx.x) * kTB + threadIdx.x) * 4;
  int seq[4];
  four_seqs(a, a.seq_start, t0, seq);
  auto add = [&](int s, int c) {
    if (atomicAdd(a.ws.counts + s, c) == 0) atomicAdd(&a.ws.totals->seqs, 1);
  };
  __syncwarp();
  int any = max(max(seq[0], seq[1]), max(seq[2], seq[3]));
  any = __reduce_max_sync(0xffffffffu, any);      // a sequence that counts here
  bool other = false;
  int c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    other |= seq[i] >= 0 && seq[i] != any;
    c += seq[i] >= 0;
  }
  const int n = __reduce_add_sync(0xffffffffu, c);
  __shared__ int s_rows;
  if (threadIdx.x == 0) s_rows = 0;
  __syncthreads();
  if (lane == 0 && n) atomicAdd(&s_rows, n);
  __syncthreads();
  if (threadIdx.x == 0 && s_rows) atomicAdd(&a.ws.totals->rows, s_rows);
  if (any < 0) return;
  if (!__any_sync(0xffffffffu, other)) {          // the warp's only one: add once
    if (lane == 0) add(any, n);
    return;
  }
  for (int i = 0; i < 4; ++i) {                   // runs of one sequence
    if (seq[i] < 0) continue;
    int m = 1;
    while (i + 1 < 4 && seq[i + 1] == seq[i]) {
      ++m;
      ++i;
    }
    add(seq[i], m);
  }
}

// The same by a block per sequence, which no other one adds to: no zeroing before,
// no atomics.
__global__ void __launch_bounds__(kTB) policy_seq_count_kernel(const __grid_constant__ PolicyArgs a) {
  __shared__ int red[kTB / 32];
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, tid = threadIdx.x;
  if (s == 0 && tid == 0) *a.ws.totals = Totals{0, 0, 0u, 0};
  if (s >= a.nseq) return;
  const int b = min(max(a.seq_start[s], 0), a.T), e = min(max(a.seq_start[s + 1], b), a.T), len = e - b;
  if (tid == 0) check_start(a, s);
  int n = 0;
  if (!a.mask) {
    n = tid == 0 ? len : 0;
  } else {
    const uint8_t* p = a.mask + b;
    const int head = min(len, int(-reinterpret_cast<uintptr_t>(p) & 15)), units = (len - head) >> 4;
    const uint4* u = reinterpret_cast<const uint4*>(p + head);
    auto nonzero = [](uint32_t x) {    // bytes of x that are not 0
      return __popc((((x & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | x) & 0x80808080u);
    };
    if (tid < head) n += p[tid] != 0;
    if (head + units * 16 + tid < len) n += tid < 16 && p[head + units * 16 + tid] != 0;
#pragma unroll 4
    for (int i = tid; i < units; i += kTB) {
      const uint4 v = u[i];
      n += nonzero(v.x) + nonzero(v.y) + nonzero(v.z) + nonzero(v.w);
    }
  }
  __syncwarp();
  n = __reduce_add_sync(0xffffffffu, n);
  if ((tid & 31) == 0) red[tid >> 5] = n;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kTB / 32; ++i) n += red[i];
    a.ws.counts[s] = n;
  }
}

// counted rows, and sequences that have some: for whole blocks
__device__ __forceinline__ void block_totals(const PolicyArgs& a, int& rows, int& seqs) {
  if (!a.mid) {
    rows = a.ws.totals->rows;
    seqs = a.ws.totals->seqs;
    return;
  }
  __shared__ int red[2][kTB / 32];
  int n = 0, k = 0;
#pragma unroll 4
  for (int s = threadIdx.x; s < a.nseq; s += kTB) {
    const int c = a.ws.counts[s];
    n += c;
    k += c > 0;
  }
  __syncwarp();
  n = __reduce_add_sync(0xffffffffu, n);
  k = __reduce_add_sync(0xffffffffu, k);
  if ((threadIdx.x & 31) == 0) {
    red[0][threadIdx.x >> 5] = n;
    red[1][threadIdx.x >> 5] = k;
  }
  __syncthreads();
  rows = seqs = 0;
  for (int i = 0; i < kTB / 32; ++i) {
    rows += red[0][i];
    seqs += red[1][i];
  }
}

__device__ __forceinline__ void four_rows(const PolicyArgs& a, int64_t t0, int rows, int seqs, Four& f) {
  int seq[4];
  four_seqs(a, a.seq_start, t0, seq);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.w[i] = f.A[i] = 0.f;
    if (seq[i] >= 0) {
      f.w[i] = row_weight(a, rows, seqs, a.ws.counts[seq[i]]);
      f.A[i] = a.adv[a.adv_per_row ? t0 + i : seq[i]];
    }
  }
}

// weights and advantages as the rows kernels stored them
__device__ __forceinline__ void stored_rows(const PolicyArgs& a, int64_t t0, Four& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 wa = t0 + i < a.T ? a.ws.row[t0 + i] : make_float2(0.f, 0.f);
    f.w[i] = wa.x;
    f.A[i] = wa.y;
  }
}

__global__ void __launch_bounds__(kTB) policy_rows_kernel(const __grid_constant__ PolicyArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = (int64_t(blockIdx.x) * kTB + threadIdx.x) * 4;
  Four f;
  int rows, seqs;
  block_totals(a, rows, seqs);
  if (a.mid && blockIdx.x == 0 && threadIdx.x == 0) a.ws.totals->rows = rows;
  four_rows(a, t0, rows, seqs, f);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t0 + i < a.T) a.ws.row[t0 + i] = make_float2(f.w[i], f.A[i]);
}

__global__ void __launch_bounds__(kTB) policy_token_kernel(const __grid_constant__ PolicyArgs a,
                                                           const float* lp, const float* ent,
                                                           float* dlp, int64_t blocks) {
  __shared__ float red[kTB / 32][kStat];
  __shared__ bool s_last;
  pdl_wait();
  pdl_trigger();
  int rows, seqs;
  if (ent) rows = a.ws.totals->rows, seqs = 0;      // (after the logits kernel: weights are stored)
  else block_totals(a, rows, seqs);
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t t0 = b * kTok + threadIdx.x * 4;
    Four f;
    load_inputs(a, lp, ent, t0, f);
    if (ent) stored_rows(a, t0, f);
    else four_rows(a, t0, rows, seqs, f);
    policy_block(a, f, dlp, t0, threadIdx.x, red, a.ws.part + b * kStat, [] { __syncthreads(); });
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(&a.ws.totals->ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (s_last && threadIdx.x < 32) {
    __threadfence();
    policy_final<false>(a, a.ws.part, blocks, rows, threadIdx.x);
  }
}

// ---------------------------------------------------------------- logits --
// A cluster of CTAs holds one row of logits in shared memory, 4 KB (one group:
// 1024 FP32 or 2048 bf16 logits) per buffer; each warp owns a ring of buffers
// for its groups of all rows.  Per row: a warp reduces each group, as it
// arrives, to (max, sum, entropy sum) and writes the triple to every CTA of the
// cluster; after one cluster barrier each warp merges all groups, forms the
// token's gradient and writes its groups' dz from shared memory, handing each
// buffer to the next group to be loaded.  Logits are read once, dz is written
// once, and the next rows stream in while this one is reduced and written.  A
// group's arithmetic and the merge order do not depend on the cluster size.
//
// Bound by HBM for long rows: 4096 x 151936 FP32 take 790 us, 93% of the copy rate
// (734 us with a sixth of the rows masked, which are not read: 92%).  With bf16 on
// either side by HBM and issue, two exponentials and eight FP32 operations a logit: the
// same rows FP32 to bf16 767 us, bf16 to FP32 780, bf16 480 (71 to 77%).  Short and
// unaligned rows by the cluster barrier and the merge of each row and by moving
// logits to 16 bytes' alignment in shared memory: 1000 x 32003 FP32 66 us (38 us of
// HBM time), bf16 to FP32 140 us, whose stores on such rows are single words.  Few rows
// by latency: 64 x 151936 FP32 to bf16 20 us (8.5 us), 13 x 4096 10.5 us, of which the
// rows kernel before it is 3 us; the loss is summed by the last CTA.
constexpr int kGroupBytes = 4096;
constexpr int kMaxWarps = 16;
constexpr int kMaxV = 262144;
constexpr int kMaxMerge = kMaxV * 4 / kGroupBytes / 32;   // groups per lane of the merge
// Logits of kMasked or less are masked: what a mask of -inf or of the type's
// lowest value leaves has p = 0.
constexpr float kMasked = -1e30f;
// After a wait that ran out (reported; results are wrong) the others wait no longer
// than this: every row still goes through the cluster's barriers.
constexpr uint64_t kLateNs = 10000000;

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
  int V, G, gpc, slots;     // groups of a row, groups per CTA, buffers per warp
  float it, c, eta;         // 1 / temperature; that times log2(e); ln 2 times what c's rounding took, by c
  float* lp;
  float* ent;
  void* dz;
  int64_t ldz;
  int tail;                 // the last CTA to be done sums the loss
};

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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// two FP32 values rounded to bf16 by one conversion (two single ones go through
// the unit that also serves the exponentials)
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// max that gives NaN where either is one
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float warp_max_keep_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// A lane's logits of a group are 8 runs of 16 bytes: run j starts at element
// (32 j + lane) RUN.  One run as pairs of FP32.
template <bool ZB>
struct Run {
  static constexpr int RUN = ZB ? 8 : 4;
  uint4 v;
  __device__ __forceinline__ Run(const uint8_t* buf, int j, int lane)
      : v(reinterpret_cast<const uint4*>(buf)[j * 32 + lane]) {}
  __device__ __forceinline__ uint64_t pair(int i) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (ZB) return pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
};

// largest of a lane's logits, run by run
template <bool ZB>
struct LaneMax {
  uint32_t a = ZB ? 0xFF80FF80u : 0xFF800000u, b = a;   // -inf
  __device__ __forceinline__ void add(const uint4& v) {
    if constexpr (ZB) {
      a = max_bf16x2_nan(a, max_bf16x2_nan(v.x, v.y));
      b = max_bf16x2_nan(b, max_bf16x2_nan(v.z, v.w));
    } else {
      a = __float_as_uint(fmax3_nan(__uint_as_float(a), __uint_as_float(v.x), __uint_as_float(v.y)));
      b = __float_as_uint(fmax3_nan(__uint_as_float(b), __uint_as_float(v.z), __uint_as_float(v.w)));
    }
  }
  __device__ __forceinline__ float value() const {
    if constexpr (ZB) {
      const uint32_t m = max_bf16x2_nan(a, b);
      return fmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    return fmax_nan(__uint_as_float(a), __uint_as_float(b));
  }
};
// of the group, over the warp
template <bool ZB>
__device__ __forceinline__ float group_max(const uint8_t* buf, int lane) {
  LaneMax<ZB> m;
#pragma unroll
  for (int j = 0; j < 8; ++j) m.add(reinterpret_cast<const uint4*>(buf)[j * 32 + lane]);
  return warp_max_keep_nan(m.value());
}

// sums over the group's 2^y and 2^y y, y = x c - mc, over the warp
template <bool ZB>
__device__ __forceinline__ void group_sums(const uint8_t* buf, int lane, float c, float mc, float& s,
                                           float& t) {
  const uint64_t c2 = pack2(c, c), n2 = pack2(-mc, -mc);
  uint64_t sa = 0, sb = 0, ta = 0, tb = 0;
#pragma unroll 4
  for (int j = 0; j < 8; ++j) {
    const Run<ZB> r(buf, j, lane);
#pragma unroll
    for (int i = 0; i < Run<ZB>::RUN / 2; ++i) {
      const uint64_t y2 = fma2(r.pair(i), c2, n2);
      float y0, y1;
      unpack2(y2, y0, y1);
      const uint64_t e2 = pack2(ex2f(y0), ex2f(y1));
      if (i & 1) {
        sb = add2(sb, e2);
        tb = fma2(e2, y2, tb);
      } else {
        sa = add2(sa, e2);
        ta = fma2(e2, y2, ta);
      }
    }
  }
  float s0, s1, t0, t1;
  unpack2(add2(sa, sb), s0, s1);
  unpack2(add2(ta, tb), t0, t1);
  s = warp_sum_x(s0 + s1);
  t = warp_sum_x(t0 + t1);
}

// every logit of the group at least kMasked (a NaN stays)
template <bool ZB>
__device__ __forceinline__ void clamp_group(uint8_t* buf, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint4* p = reinterpret_cast<uint4*>(buf) + j * 32 + lane;
    uint4 v = *p;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i)   // (for bf16 the next value below kMasked, twice)
      w[i] = ZB ? max_bf16x2_nan(w[i], 0xF14AF14Au)
                : __float_as_uint(fmax_nan(__uint_as_float(w[i]), kMasked));
    *p = v;
  }
}

// Bring a group that starts `off` bytes into its buffer (a row that is not
// 16-byte aligned) to the buffer's start.  Lanes take consecutive words, so that
// neither side has bank conflicts at any offset (16 bytes a lane, put together
// from two units, took 69 us where this takes 53: 1000 rows of 32003 FP32 logits
// without padding).  Returns the largest of the lane's logits.
template <bool ZB, bool HALF>
__device__ __forceinline__ float settle(uint8_t* buf, int lane, int off) {
  const uint32_t* src = reinterpret_cast<const uint32_t*>(buf + (off & ~3)) + lane;
  uint32_t r[32];
#pragma unroll
  for (int k = 0; k < 32; ++k)
    r[k] = HALF ? __funnelshift_r(src[k * 32], src[k * 32 + 1], 16) : src[k * 32];
  __syncwarp();
  LaneMax<ZB> m;
#pragma unroll
  for (int k = 0; k < 32; ++k) reinterpret_cast<uint32_t*>(buf)[k * 32 + lane] = r[k];
#pragma unroll
  for (int k = 0; k < 32; k += 4) m.add(make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]));
  return m.value();
}
// ... and mask what lies behind `left` logits.  Returns the largest logit, over
// the warp.
template <bool ZB, bool SHIFT>
__device__ __forceinline__ float settle_group(uint8_t* buf, int lane, int off, int left) {
  constexpr int kGroup = kGroupBytes / (ZB ? 2 : 4);
  __syncwarp();
  if (SHIFT && off) {
    const float m = ZB && (off & 2) ? settle<ZB, ZB>(buf, lane, off) : settle<ZB, false>(buf, lane, off);
    __syncwarp();
    if (left == kGroup) return warp_max_keep_nan(m);
  }
  for (int e = left + lane; e < kGroup; e += 32) {
    if (ZB) reinterpret_cast<uint16_t*>(buf)[e] = 0xF14A;
    else reinterpret_cast<float*>(buf)[e] = kMasked;
  }
  __syncwarp();
  return group_max<ZB>(buf, lane);
}

// Copy a group's N results (`left` of them, DS bytes each, from the start of its
// buffer) to a row of any alignment, in words of the destination.
template <int DS, int N>
__device__ __forceinline__ void store_unaligned(uint8_t* dst, const uint8_t* buf, int lane, int left) {
  const uint32_t* src = reinterpret_cast<const uint32_t*>(buf) + lane;
  const bool half = DS == 2 && (reinterpret_cast<uintptr_t>(dst) & 2);
  const int head = half ? 1 : 0, words = (left - head) * DS / 4;
  uint32_t* d = reinterpret_cast<uint32_t*>(dst + head * DS) + lane;
  if (half) {
#pragma unroll 8
    for (int k = 0; k < N * DS / 128; ++k)
      if (k * 32 + lane < words) d[k * 32] = __funnelshift_r(src[k * 32], src[k * 32 + 1], 16);
  } else {
#pragma unroll 16
    for (int k = 0; k < N * DS / 128; ++k)
      if (k * 32 + lane < words) d[k * 32] = src[k * 32];
  }
  if (DS == 2) {   // the first and last elements, where they share their word with a neighbour
    uint16_t* h = reinterpret_cast<uint16_t*>(dst);
    const uint16_t* b = reinterpret_cast<const uint16_t*>(buf);
    if (lane == 0 && head) h[0] = b[0];
    if (lane == 1 && head + words * 2 < left) h[left - 1] = b[left - 1];
  }
}

// `bytes` zeros (elements of `ds` bytes) from d on, by a warp
__device__ __forceinline__ void zero_fill(uint8_t* d, int bytes, int ds, int lane) {
  const int head = min(bytes, int(-reinterpret_cast<uintptr_t>(d) & 15));
  const int units = (bytes - head) >> 4;
  uint4* u = reinterpret_cast<uint4*>(d + head);
#pragma unroll 4
  for (int i = lane; i < units; i += 32) u[i] = make_uint4(0, 0, 0, 0);
  // the first and last elements, which share their 16 bytes with others
  for (int i = lane * ds; i < head; i += 32 * ds) {
    if (ds == 2) *reinterpret_cast<uint16_t*>(d + i) = 0;
    else *reinterpret_cast<float*>(d + i) = 0.f;
  }
  for (int i = head + units * 16 + lane * ds; i < bytes; i += 32 * ds) {
    if (ds == 2) *reinterpret_cast<uint16_t*>(d + i) = 0;
    else *reinterpret_cast<float*>(d + i) = 0.f;
  }
}

// The loss over all rows, by the CTA that was the last to have its rows' lp and
// entropy written: its warps take 128 rows each in turn, so that the sums are
// those of any number of warps.  (A launch less than a kernel of its own.)
__device__ __forceinline__ void policy_tail(const PolicyArgs& a, const float* lp, const float* ent,
                                            uint8_t* smem) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float(*red)[kStat] = reinterpret_cast<float(*)[kStat]>(smem);   // [32]
  float* part = reinterpret_cast<float*>(smem) + 32 * kStat;      // [4][kStat]
  const int rows = a.ws.totals->rows;
  const int blocks = (a.T + kTok - 1) / kTok;
  const int warps = (a.T + 127) / 128;          // of 128 rows
  for (int i = threadIdx.x; i < 32 * kStat; i += blockDim.x)
    if (i >= warps * kStat) (&red[0][0])[i] = 0.f;
  for (int i = warp; i < warps; i += nw) {
    const int64_t t0 = int64_t(i) * 128 + lane * 4;
    Four f;
    load_inputs(a, lp, ent, t0, f);
    stored_rows(a, t0, f);
    float v[kStat], g[4];
    policy_four(a, f, g, v);
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < 7; ++k) red[i][k] = v[k];
    }
  }
  __syncthreads();
  if (warp != 0) return;
  if (lane < 28 && lane / 7 < blocks) part[lane / 7 * kStat + lane % 7] = block_entry(red + lane / 7 * 8, lane % 7);
  __syncwarp();
  policy_final<true>(a, part, blocks, rows, lane);
}

template <bool ZB, bool DB, bool SHIFT>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) policy_logits_kernel(
    const __grid_constant__ LogitsArgs a) {
  constexpr int ES = ZB ? 2 : 4, DS = DB ? 2 : 4, RUN = Run<ZB>::RUN;
  constexpr int kGroup = kGroupBytes / ES;
  constexpr int BUF = kGroupBytes + (SHIFT ? 16 : 0);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  uint8_t* bufs = smem + size_t(warp) * a.slots * BUF;                          // this warp's ring
  float4* stats = reinterpret_cast<float4*>(smem + size_t(nw) * a.slots * BUF); // [2][G]
  uint64_t* bars = reinterpret_cast<uint64_t*>(stats + 2 * a.G) + warp * a.slots;
  uint32_t ncta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncta));
  const int rank = int(cluster_rank());
  const int clusters = int(gridDim.x / ncta), me = int(blockIdx.x / ncta);
  const int g0 = rank * a.gpc, mine = max(0, min(a.gpc, a.G - g0));   // this CTA's groups
  const int per = warp < mine ? (mine - warp - 1) / nw + 1 : 0;       // of these, this warp's

  if (lane == 0) {
    for (int i = 0; i < a.slots; ++i) mbar_init(smem_u32(bars + i), 1);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_trigger();
  cluster_sync();

  // The cluster's rows are me + q clusters, q < rows.  Lane l holds what the
  // token's gradient needs of row 32 win + l (and its target's logit); a bit
  // per row says whether it counts.
  const int rows = me < a.p.T ? (a.p.T - 1 - me) / clusters + 1 : 0;
  auto row_of = [&](int q) { return me + q * clusters; };
  auto row_ptr = [&](int q) {
    return static_cast<const uint8_t*>(a.z) + int64_t(row_of(q)) * a.ld * ES;
  };
  auto counted = [&](int w) {
    const int q = w * 32 + lane;
    return __ballot_sync(0xffffffffu, q < rows && a.p.ws.row[row_of(q)].x > 0.f);
  };
  int win = 0;
  uint32_t on0 = counted(0), on1 = counted(1);      // windows win and win + 1
  float2 m_wa;
  int m_tg;
  float m_old, m_ref, m_zt;
  auto load_window = [&]() {
    const int q = win * 32 + lane;
    m_wa = make_float2(0.f, 0.f);
    m_tg = -1;
    m_old = m_ref = m_zt = 0.f;
    if ((on0 >> lane) & 1u) {
      const int r = row_of(q);
      m_wa = a.p.ws.row[r];
      const int tg = a.target[r];
      if (a.p.old_lp) m_old = a.p.old_lp[r];
      if (a.p.ref_lp) m_ref = a.p.ref_lp[r];
      // a target outside [0, V) stays -1: the row's last group may reach past V, and
      // no element there is the target's
      if (tg >= 0 && tg < a.V) {
        m_tg = tg;
        if (ZB) m_zt = bf2f(reinterpret_cast<const uint16_t*>(row_ptr(q))[tg]);
        else m_zt = reinterpret_cast<const float*>(row_ptr(q))[tg];
      }
    }
  };
  load_window();
  // the first row from q on that counts (rows: none)
  auto next_counted = [&](int q) {
    while (q < rows) {
      const int w = q >> 5;
      const uint32_t bits = (w == win ? on0 : w == win + 1 ? on1 : counted(w)) >> (q & 31);
      if (bits) return q + __ffs(int(bits)) - 1;
      q = (w + 1) << 5;
    }
    return rows;
  };

  // A warp's groups of all its rows form one sequence, n = 0, 1, ...; group n
  // sits in slot n % slots, and is loaded when group n - slots is done with
  // (at most two rows ahead).
  const uint32_t slots = uint32_t(min(a.slots, 2 * per));
  // q0: the row whose dz is written; q1: the one that is reduced
  int q0 = -1, q1 = next_counted(0), q2 = next_counted(q1 + 1), q3 = next_counted(q2 + 1);
  int ahead = 1, ai = 0;           // next group to load: the ai-th of row q<ahead>
  // starts the copy of that group: the 16-byte units that lie in the row; what
  // is left of the row's first and last unit is read later
  auto load_next = [&](uint32_t slot) {
    const int q = ahead == 1 ? q1 : ahead == 2 ? q2 : q3;
    if (q < rows && lane == 0) {
      const uint32_t bar = smem_u32(bars + slot), dst = smem_u32(bufs + slot * BUF);
      const int g = g0 + warp + ai * nw;
      const uint8_t* gp = row_ptr(q) + size_t(g) * kGroupBytes;
      if (!SHIFT) {
        const uint32_t bytes = uint32_t(min(kGroup, a.V - g * kGroup) * ES) & ~15u;
        mbar_expect_tx(bar, bytes);
        if (bytes) bulk_load(dst, gp, bytes, bar);
      } else {
        const uintptr_t gb = reinterpret_cast<uintptr_t>(gp), b = gb - size_t(g) * kGroupBytes;
        const uintptr_t e = b + size_t(a.V) * ES, ge = min(gb + kGroupBytes, e);
        uintptr_t lo = gb & ~uintptr_t(15), hi = (ge + 15) & ~uintptr_t(15);
        if (lo < b) lo += 16;
        if (hi > e) hi -= 16;
        const uint32_t bytes = hi > lo ? uint32_t(hi - lo) : 0u;
        mbar_expect_tx(bar, bytes);
        if (bytes)
          bulk_load(dst + uint32_t(lo - (gb & ~uintptr_t(15))), reinterpret_cast<const void*>(lo), bytes, bar);
      }
    }
    if (++ai == per) {
      ai = 0;
      ++ahead;
    }
  };
  for (uint32_t i = 0; i < slots; ++i) load_next(i);
  __syncwarp();
  uint32_t slot0 = 0;              // of row q0's next group
  uint32_t slot1 = 0, phase1 = 0;  // of row q1's next group
  uint32_t dirty = 0;              // slots (mod 32) this warp has written to
  uint32_t flip = 0;
  bool late = false;               // a wait has run out
  // of row q0, where there is one
  constexpr float kLn2 = 0.6931471805599453f;
  float M = 0.f, a0 = 0.f, a1 = 0.f, at_target = 0.f, zt = 0.f;
  int tg0 = -1;
  // The thread that writes a row's lp and entropy (of the warp with the fewest
  // groups).  Behind the last counted row it adds 1 to the ticket, before that
  // row's dz is written: the fence and the atomic take their time meanwhile.
  const bool teller = rank == 0 && tid == (nw - 1) * 32;
  unsigned told = 0;
  auto tell = [&]() {
    __threadfence();
    told = atomicAdd(&a.p.ws.totals->ticket, 1u);
  };
  if (teller && a.tail && q1 >= rows) tell();
  while (true) {
    // ---- row q0: dz = p (a0 + a1 y) (+ at_target), y = log2 of p S
    if (q0 >= 0) {
      uint8_t* row = static_cast<uint8_t*>(a.dz) + int64_t(row_of(q0)) * a.ldz * DS;
      for (int i = 0; i < per; ++i) {
        const int g = g0 + warp + i * nw;
        if (a.dz) {
          const int left = min(kGroup, a.V - g * kGroup);
          uint8_t* buf = bufs + slot0 * BUF;
          uint8_t* dst = row + int64_t(g) * kGroup * DS;
          const uint64_t c2 = pack2(a.c, a.c), n2 = pack2(-M, -M);
          const uint64_t p0 = pack2(a0, a0), p1 = pack2(a1, a1);
          const bool ent = a1 != 0.f;
          float at = 0.f;              // dz at the target
          const int tl = tg0 - g * kGroup;
          if (tl >= 0 && tl < kGroup) {
            const float y = fmaf(zt, a.c, -M), e = ex2f(y);
            at = fmaf(e, a0, ent ? e * fmaxf(y, kMasked) * a1 : 0.f) + at_target;
          }
#pragma unroll 4
          for (int j = 0; j < 8; ++j) {
            const Run<ZB> r(buf, j, lane);
            float x[RUN];
#pragma unroll
            for (int k = 0; k < RUN / 2; ++k) {
              const uint64_t y2 = fma2(r.pair(k), c2, n2);
              float y0, y1;
              unpack2(y2, y0, y1);
              const uint64_t e2 = pack2(ex2f(y0), ex2f(y1));
              // (e y first: with e = 0 and y far below, y a1 may overflow)
              const uint64_t ea = mul2(e2, p0);
              unpack2(ent ? fma2(mul2(e2, y2), p1, ea) : ea, x[2 * k], x[2 * k + 1]);
            }
            const int el = (j * 32 + lane) * RUN;
            if (SHIFT && DS <= ES) {
              // results take their logits' place in the buffer
              if (DS < ES) __syncwarp();
              if constexpr (DB) {
                uint32_t h[RUN / 2];
#pragma unroll
                for (int k = 0; k < RUN / 2; ++k) h[k] = cvt_bf16x2(x[2 * k], x[2 * k + 1]);
                if constexpr (RUN == 8) *reinterpret_cast<uint4*>(buf + el * 2) = make_uint4(h[0], h[1], h[2], h[3]);
                else *reinterpret_cast<uint2*>(buf + el * 2) = make_uint2(h[0], h[1]);
              } else {
                *reinterpret_cast<float4*>(buf + el * 4) = make_float4(x[0], x[1], x[2], x[3]);
              }
            } else if (!SHIFT && el + RUN <= left) {
              if constexpr (DB) {
                uint32_t h[RUN / 2];
#pragma unroll
                for (int k = 0; k < RUN / 2; ++k) h[k] = cvt_bf16x2(x[2 * k], x[2 * k + 1]);
                if constexpr (RUN == 8) *reinterpret_cast<uint4*>(dst + el * 2) = make_uint4(h[0], h[1], h[2], h[3]);
                else *reinterpret_cast<uint2*>(dst + el * 2) = make_uint2(h[0], h[1]);
              } else {
#pragma unroll
                for (int k = 0; k < RUN; k += 4)
                  *reinterpret_cast<float4*>(dst + (el + k) * 4) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < RUN; ++k)
                if (el + k < left) {
                  if (DB) reinterpret_cast<uint16_t*>(dst)[el + k] = f2bf(x[k]);
                  else reinterpret_cast<float*>(dst)[el + k] = x[k];
                }
            }
          }
          // the target's element again, by the lane that wrote it
          if (tl >= 0 && tl < kGroup && ((tl / RUN) & 31) == lane) {
            uint8_t* d = (SHIFT && DS <= ES ? buf : dst) + tl * DS;
            if (DB) *reinterpret_cast<uint16_t*>(d) = f2bf(at);
            else *reinterpret_cast<float*>(d) = at;
          }
          if (SHIFT && DS <= ES) {
            __syncwarp();
            store_unaligned<DS, kGroup>(dst, buf, lane, left);
            dirty |= 1u << (slot0 & 31);
          }
        }
        // the warp's reads of the buffer are done (their values were used);
        // what it wrote there is ordered before the copy that comes next
        if ((dirty >> (slot0 & 31)) & 1u) fence_proxy_async();
        dirty &= ~(1u << (slot0 & 31));
        __syncwarp();
        load_next(slot0);
        if (++slot0 == slots) slot0 = 0;
      }
    }
    // rows that do not count, up to q1 (all that are left: q1 = rows): zeros
    for (int q = q0 + 1; q < q1; ++q) {
      if (a.dz) {
        uint8_t* row = static_cast<uint8_t*>(a.dz) + int64_t(row_of(q)) * a.ldz * DS;
        for (int i = 0; i < per; ++i) {
          const int g = g0 + warp + i * nw;
          zero_fill(row + int64_t(g) * kGroup * DS, min(kGroup, a.V - g * kGroup) * DS, DS, lane);
        }
      }
      if (teller) {
        a.lp[row_of(q)] = 0.f;
        a.ent[row_of(q)] = 0.f;
      }
    }
    if (q1 >= rows) break;
    __syncwarp();
    while ((q1 >> 5) != win) {     // the next window of rows
      ++win;
      on0 = on1;
      on1 = counted(win + 1);
      if ((q1 >> 5) == win) load_window();
    }
    // ---- row q1: each group's (max, sum, entropy sum), relative to its own max
    const uint8_t* src = row_ptr(q1);
    const int off = SHIFT ? int(reinterpret_cast<uintptr_t>(src) & 15) : 0;
    float4* st = stats + flip * a.G;
    for (int i = 0; i < per; ++i) {
      const int g = g0 + warp + i * nw;
      const int left = min(kGroup, a.V - g * kGroup);
      uint8_t* buf = bufs + slot1 * BUF;
      if (!mbar_wait(smem_u32(bars + slot1), phase1, a.p.err, late ? kLateNs : kWaitLimitNs)) late = true;
      float m;
      if ((SHIFT && off) || left < kGroup) {
        // elements of the row's first and last 16-byte unit, where it holds
        // bytes outside the row: not part of any copy
        if (g * kGroup + left + 16 / ES > a.V || (SHIFT && g == 0)) {
          const uintptr_t b = reinterpret_cast<uintptr_t>(src), e = b + size_t(a.V) * ES;
          auto fetch = [&](int idx) {
            uint8_t* d = buf + off + (idx - g * kGroup) * ES;
            if (ZB) *reinterpret_cast<uint16_t*>(d) = reinterpret_cast<const uint16_t*>(src)[idx];
            else *reinterpret_cast<float*>(d) = reinterpret_cast<const float*>(src)[idx];
          };
          if (lane < 16 / ES) {
            const int tail = a.V - 1 - lane;
            if (tail >= g * kGroup && tail < g * kGroup + left &&
                b + size_t(tail) * ES >= (e & ~uintptr_t(15)))
              fetch(tail);
            if (SHIFT && g == 0 && lane < left && (b & 15) && (b & 15) + lane * ES < 16) fetch(lane);
          }
        }
        m = settle_group<ZB, SHIFT>(buf, lane, off, left);
        dirty |= 1u << (slot1 & 31);
      } else {
        m = group_max<ZB>(buf, lane);
      }
      float mc = -INFINITY, s = 0.f, t = 0.f;
      if (!(m <= kMasked)) {         // (a NaN comes through)
        mc = __fmul_rn(m, a.c);
        group_sums<ZB>(buf, lane, a.c, mc, s, t);
      }
      // masked logits among the others (0 times an exponent of -inf), or alone:
      // clamped once, for these sums and for dz
      if (t != t || m <= kMasked) {
        __syncwarp();
        clamp_group<ZB>(buf, lane);
        __syncwarp();
        dirty |= 1u << (slot1 & 31);
        if (t != t) group_sums<ZB>(buf, lane, a.c, mc, s, t);
        if (m <= kMasked) m = -INFINITY;
      }
      if (lane < ncta) st_cluster_v4(smem_u32(st + g), lane, m, s, t, mc);
      if (++slot1 == slots) {
        slot1 = 0;
        phase1 ^= 1;
      }
    }
    cluster_sync();

    // ---- merge row q1's groups: lane l takes groups l, l + 32, ... in order
    float4 q[kMaxMerge];
    float top = -INFINITY;             // the row's largest logit
#pragma unroll
    for (int k = 0; k < kMaxMerge; ++k) {
      const int g = k * 32 + lane;
      q[k] = g < a.G ? st[g] : make_float4(-INFINITY, 0.f, 0.f, -INFINITY);
      top = fmax_nan(top, q[k].x);
    }
    top = warp_max_keep_nan(top);
    M = __fmul_rn(top, a.c);
    const float xm = __fmul_rn(top, a.it);
    const float r_M = -kLn2 * fmaf(top, a.c, -M), r_x = fmaf(top, a.it, -xm);   // what these roundings took
    float S = 0.f, U = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxMerge; ++k) {
      // a group of masked logits alone (M may be -inf too) adds nothing
      const bool has = q[k].x != -INFINITY;
      const float d = q[k].w - M, f = ex2f(d);
      S = has ? fmaf(q[k].y, f, S) : S;
      U = has ? fmaf(f, fmaf(q[k].y, d, q[k].z), U) : U;
    }
    S = warp_sum_x(S);
    U = warp_sum_x(U);
    if (top == -INFINITY) S = NAN;   // nothing but masked logits
    const float rS = __frcp_rn(S);
    // lp = (x_t - max x) - log of the sum of exp(x - max x), x = z / temperature, as
    // these FP32 operations.  That sum is S + t to first order: M's rounding is in all
    // of S, that of max x in all but the largest term, c's in U.  (From the base-2
    // exponent, fma(z_t, c, -M) ln 2 - lnS, lp was off by twice as much.)
    const float t = fmaf(r_x, S - 1.0f, fmaf(r_M, S, a.eta * U)), ratio = t * rS;
    const bool near = fabsf(t) < 0x1p-12f * S;        // (not so for logits of some thousands)
    const float l0 = logf(near ? S + t : S);
    const float ls = near ? l0 : l0 + ratio;
    const float lnS = near ? l0 - ratio : l0;
    const float H = lnS - kLn2 * (U * rS);
    const int from = q1 & 31;
    tg0 = __shfl_sync(0xffffffffu, m_tg, from);
    zt = __shfl_sync(0xffffffffu, m_zt, from);
    const bool tg_ok = tg0 >= 0;
    const float lp = tg_ok ? __fsub_rn(__fsub_rn(__fmul_rn(zt, a.it), xm), ls) : NAN;
    if (teller) {
      a.lp[row_of(q1)] = lp;
      a.ent[row_of(q1)] = H;
      if (!tg_ok) raise_error(a.p.err, kErrBadIndex);
      if (a.tail && q2 >= rows) tell();
    }
    if (a.dz) {
      const float wt = __shfl_sync(0xffffffffu, m_wa.x, from), A = __shfl_sync(0xffffffffu, m_wa.y, from);
      const float old = __shfl_sync(0xffffffffu, m_old, from), ref = __shfl_sync(0xffffffffu, m_ref, from);
      const Token o = policy_token(a.p, lp, A, old, ref);
      // (a masked target: no gradient by way of lp)
      const float dlp = zt <= kMasked ? 0.f : wt * o.dlp, wg = wt * a.p.gamma, is = a.it * rS;
      a0 = is * (wg * (H - lnS) - dlp);
      a1 = is * wg * kLn2;
      at_target = a.it * dlp;
    }
    flip ^= 1;
    --ahead;
    q0 = q1;
    q1 = q2;
    q2 = q3;
    q3 = next_counted(q3 + 1);
  }
  cluster_sync();   // no CTA leaves while another may still write its statistics
  if (a.tail && rank == 0) {
    int* last = reinterpret_cast<int*>(smem);
    if (teller) *last = told == unsigned(clusters) - 1u;
    __syncthreads();
    const bool sum = *last;
    __syncthreads();
    if (!sum) return;
    __threadfence();
    policy_tail(a.p, a.lp, a.ent, smem);
  }
}

// -------------------------------------------------------------- host side --
biv_status check_policy(const biv_policy_desc* d, const char* who) {
  BIV_REQUIRE(d, "%s: null descriptor", who);
  BIV_REQUIRE(d->T >= 0 && d->nseq >= 0 && d->T <= (1 << 30), "%s: bad sizes", who);
  BIV_REQUIRE(d->stats, "%s: null pointer", who);
  if (d->T == 0) return BIV_OK;
  BIV_REQUIRE(d->seq_start && (d->adv || (d->nseq == 0 && !d->adv_per_row)), "%s: null pointer", who);
  BIV_REQUIRE(d->clip_lo >= 0.f && d->clip_lo <= 1.f && d->clip_hi >= 0.f,
              "%s: clip_lo must lie in [0, 1] and clip_hi must not be negative", who);
  BIV_REQUIRE(d->dual_clip == 0.f || d->dual_clip > 1.f, "%s: dual_clip must be 0 or above 1", who);
  BIV_REQUIRE(d->kl_coef >= -1e3f && d->kl_coef <= 1e3f && d->ent_coef >= -1e3f && d->ent_coef <= 1e3f,
              "%s: kl_coef and ent_coef must lie in [-1000, 1000]", who);
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

// no row at all: statistics are zeros
biv_status no_rows(const biv_policy_desc& d, biv_stream_t stream) {
  if (cudaMemsetAsync(d.stats, 0, kStat * sizeof(float), as_cuda(stream)) != cudaSuccess)
    return set_error(BIV_ERR_CUDA, "policy_loss: %s", cudaGetErrorString(cudaGetLastError()));
  return BIV_OK;
}

PolicyArgs policy_args(const biv_policy_desc& d) {
  PolicyArgs a;
  a.T = d.T; a.nseq = d.nseq; a.seq_start = d.seq_start; a.mask = d.mask;
  a.old_lp = d.old_lp; a.ref_lp = d.ref_lp; a.adv = d.adv; a.adv_per_row = d.adv_per_row;
  a.lo = 1.0f - d.clip_lo; a.hi = 1.0f + d.clip_hi; a.dual = d.dual_clip;
  a.beta = d.kl_coef; a.gamma = d.ent_coef; a.reduce = d.reduce; a.norm = d.norm;
  a.mid = d.nseq <= kMidSeqs && d.T <= kMidMean * d.nseq;
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

bool small_call(const PolicyArgs& a) { return a.T <= kSmallRows && a.nseq <= kSmallSeqs; }
unsigned small_threads(const PolicyArgs& a) { return unsigned(token_blocks(a.T)) * kTB; }

// counts per sequence (large calls)
biv_status launch_counts(const PolicyArgs& a, cudaStream_t s) {
  if (a.mid) {
    launch_pdl(policy_seq_count_kernel, unsigned(std::max(1, a.nseq)), kTB, 0, s, a);
    return check_launch("policy_seq_count");
  }
  launch_pdl(policy_zero_kernel, unsigned(std::max(1, (a.nseq + kTB - 1) / kTB)), kTB, 0, s, a);
  biv_status st = check_launch("policy_zero");
  if (st != BIV_OK) return st;
  launch_pdl(policy_count_kernel, unsigned(token_blocks(a.T)), kTB, 0, s, a);
  return check_launch("policy_count");
}

// weight and advantage of every row, for the logits kernel
biv_status launch_rows(const PolicyArgs& a, cudaStream_t s) {
  if (small_call(a)) {
    launch_pdl(policy_small_kernel<true>, 1, small_threads(a), 0, s, a, static_cast<const float*>(nullptr),
               static_cast<float*>(nullptr));
    return check_launch("policy_rows");
  }
  biv_status st = launch_counts(a, s);
  if (st != BIV_OK) return st;
  launch_pdl(policy_rows_kernel, unsigned(token_blocks(a.T)), kTB, 0, s, a);
  return check_launch("policy_rows");
}

// the sums over all rows (and dlp): after launch_counts or the small rows kernel
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

// Shape of the logits kernel (GB300, GPU time of the whole call, as measured when
// each choice was made).  A row is spread over as few CTAs as hold it in 160 KB
// each, one CTA per SM: 4096 rows x 151936 FP32 take 726 us on clusters of 4, 1069
// us on clusters of 8 with two CTAs per SM; 2037 x 131072 bf16 188 us on clusters
// of 2, 201 us on 4.  Up to 16 warps (128 registers each): 24 take 786 us on the
// first case, 189 us on the second.  What is left of 216 KB prefetches the next
// row: without it the first case takes 786 us.  Shorter rows run two CTAs per SM,
// so that one's barrier and merge overlap the other's traffic: 1000 x 16384 FP32
// 28.8 us against 31.6 us; 2000 x 50257 bf16 (100 KB), which would lose its
// prefetch, 122 us against 104.
constexpr size_t kRowBytesPerCta = 160 << 10, kPairBytes = 80 << 10, kRingBytes = 216 << 10;

template <bool ZB, bool DB, bool SHIFT>
biv_status launch_logits(LogitsArgs& a, cudaStream_t s) {
  constexpr int BUF = kGroupBytes + (SHIFT ? 16 : 0);
  const int sms = sm_count() > 0 ? sm_count() : 148;
  a.G = (a.V + kGroupBytes / (ZB ? 2 : 4) - 1) / (kGroupBytes / (ZB ? 2 : 4));
  unsigned cl = 1;
  while (cl < 8 && size_t((a.G + cl - 1) / cl) * kGroupBytes > kRowBytesPerCta) cl *= 2;
  // few rows: spread each over more SMs (no bit depends on it)
  while (cl < 8 && int(cl) * 2 <= a.G && int64_t(a.p.T) * cl * 2 <= sms) cl *= 2;
  a.gpc = int((a.G + cl - 1) / cl);
  const bool pair = size_t(a.gpc) * kGroupBytes <= kPairBytes;
  const int most = pair ? kMaxWarps / 2 : kMaxWarps, per = (a.gpc + most - 1) / most;
  const size_t ring = pair ? kRingBytes / 2 - 1024 : kRingBytes;
  const unsigned warps = unsigned((a.gpc + per - 1) / per), threads = warps * 32;
  // The loss by the last CTA, where its warps take at most twice 128 rows each: 13 x
  // 4096 FP32 14.5 us a call, bound by the host's launches, against 20.7 us with a
  // kernel for it (10.8 us of GPU time against 9.9; with eight turns of one warp 13.9)
  a.tail = a.p.T <= kSmallRows && a.p.T <= int(warps) * 256;
  // a warp's ring: its groups of a row, and of the next one what the room allows
  a.slots = per;
  while (a.slots < 2 * per && size_t(a.slots + 1) * warps * BUF <= ring) ++a.slots;
  const size_t smem = size_t(a.slots) * warps * (BUF + 8) + size_t(a.G) * 32;
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
  if (st != BIV_OK) return st;
  if (d->T == 0) return no_rows(*d, stream);
  BIV_REQUIRE(lp, "policy_loss: null pointer");
  BIV_REQUIRE(d->ent_coef == 0.f, "policy_loss: an entropy term needs the logits");
  const PolicyArgs a = policy_args(*d);
  cudaStream_t s = as_cuda(stream);
  if (small_call(a)) {
    launch_pdl(policy_small_kernel<false>, 1, small_threads(a), 0, s, a, lp, dlp);
    return check_launch("policy_loss");
  }
  st = launch_counts(a, s);
  if (st != BIV_OK) return st;
  return launch_tokens(a, lp, nullptr, dlp, s);
}

biv_status biv_policy_loss_logits(const biv_policy_desc* d, const void* z, int64_t ld, int z_dtype,
                                  const int32_t* target, int V, float inv_temp, float* lp,
                                  float* entropy, void* dz, int64_t ldz, int dz_dtype,
                                  biv_stream_t stream) {
  biv_status st = check_policy(d, "policy_loss_logits");
  if (st != BIV_OK) return st;
  if (d->T == 0) return no_rows(*d, stream);
  BIV_REQUIRE(z && target && lp && entropy, "policy_loss_logits: null pointer");
  BIV_REQUIRE(V >= 1 && V <= kMaxV, "policy_loss_logits: V must lie in [1, %d]", kMaxV);
  BIV_REQUIRE((z_dtype == BIV_F32 || z_dtype == BIV_BF16) &&
                  (!dz || dz_dtype == BIV_F32 || dz_dtype == BIV_BF16),
              "policy_loss_logits: logits and gradient are f32 or bf16");
  BIV_REQUIRE(ld >= V && (!dz || ldz >= V), "policy_loss_logits: a row stride is below V");
  BIV_REQUIRE(inv_temp >= 0.01f && inv_temp <= 100.f,
              "policy_loss_logits: inv_temp must lie in [0.01, 100]");
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
  a.G = a.gpc = a.slots = 0;
  a.it = inv_temp;
  const double c = double(inv_temp) * 1.4426950408889634;
  a.c = float(c);
  a.eta = float((c / a.c - 1.0) * 0.6931471805599453);
  a.lp = lp; a.ent = entropy; a.dz = dz; a.ldz = ldz;
  // rows of logits and gradient that all keep 16 bytes' alignment
  const bool shift = zb % 16 != 0 || (size_t(ld) * es) % 16 != 0 ||
                     (dz && (db % 16 != 0 || (size_t(ldz) * ds) % 16 != 0));
  cudaStream_t s = as_cuda(stream);
  st = launch_rows(a.p, s);
  if (st != BIV_OK) return st;
  const bool zbf = z_dtype == BIV_BF16, dbf = dz && dz_dtype == BIV_BF16;
  if (zbf) {
    st = dbf ? (shift ? launch_logits<true, true, true>(a, s) : launch_logits<true, true, false>(a, s))
             : (shift ? launch_logits<true, false, true>(a, s) : launch_logits<true, false, false>(a, s));
  } else {
    st = dbf ? (shift ? launch_logits<false, true, true>(a, s) : launch_logits<false, true, false>(a, s))
             : (shift ? launch_logits<false, false, true>(a, s) : launch_logits<false, false, false>(a, s));
  }
  if (st != BIV_OK || a.tail) return st;
  return launch_tokens(a.p, lp, entropy, nullptr, s);
}

}  // extern "C"
