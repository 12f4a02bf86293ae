// Cross entropy of the LM head and its gradient without stored logits.
//
// Forward (biv_lm_head_loss): the GEMM of biv_lm_head_logprob leaves a
// (max, sum exp) pair per row and 128 columns; lse_rows_kernel merges them as
// biv_lm_head_logprob does (the same bits) and loss_rows_kernel forms the
// weighted mean and each row's coefficients for the backward.
//
// Backward (biv_lm_head_backward): with z = h.W^T and p = exp(z - lse),
//   dz = dlp (onehot(target) - p) + dlse p,   dh = dz.W,   dW = dz^T.h.
// The logits are formed again in chunks of the vocabulary: per chunk a product
// whose epilogue turns its FP32 accumulators into bf16 dz, then both products
// of that dz, all on tcgen05 with FP32 accumulators in TMEM, in one persistent
// kernel.
//  - Rows whose coefficients are 0 (prompts, padding, clipped tokens) have no
//    gradient: the rows that count are gathered first, so that what the others
//    hold is never multiplied, and no time is spent on them.
//  - The term of a row's own target is usually the largest by far.  It stays
//    out of the matrix products: its coefficient is formed while the rows are
//    gathered, and it is added in FP32, to dh by the fold and to dW by the
//    epilogue of the tile that holds the target.  The p terms enter
//    the products as bf16, the type of the other operands: an error of at most
//    2^-8 of each of them; for FP32 gradients as two bf16 parts, hi + lo (2^-16).
//  - dh is summed over the vocabulary in chunks (at most kMaxChunk columns, a
//    length that follows V and K), each accumulated from zero in TMEM in
//    ascending columns, and the chunks added in ascending order in FP32: a row's
//    dh depends on that row, V, K and the gradients' types only.  dW is one
//    accumulation over the counted rows in ascending order.
#include <algorithm>
#include <climits>
#include <cstring>

#include "common.cuh"

namespace biv {
// gemm.cu: the fused head's GEMM.  lse[row * ng + g] = (max, sum exp(z - max)) of
// columns [128 g, 128 g + 128), zt[row] = the logit at target[row] (unset where
// the target is outside [0, V)).  m_tiles (or null: all rows): on the device, the
// number of 128-row tiles to compute and their indexes.
biv_status lm_head_groups(const char* what, const uint16_t* h, int64_t ldh, const uint16_t* W,
                          int64_t ldw, int M, int V, int K, const int32_t* target, int mode,
                          const int* m_tiles, void* ws, size_t ws_bytes, const float2** lse, const float** zt, int* ng,
                          biv_stream_t stream);

namespace {

// Vocabulary columns per FP32 partial of dh: a length that follows V and K.  As
// many chunks as make two dh tiles of 256 rows for each of 76 pairs of CTAs, but
// chunks of 4096 to 8192 columns (a dh tile of K = 256 and 8192 columns is as long
// as all the rest of 9 rows: 250 us, now 190; shorter ones cost partials); a
// vocabulary of less than 32768 in eighths, rounded up to 256 columns.
constexpr int kMinChunk = 4096, kMaxChunk = 8192;
constexpr int kTM = 256;          // tile rows: 128 TMEM lanes in each CTA of a pair
constexpr int kTN = 256;          // tile columns: each CTA brings half of B
constexpr int kTK = 64;           // K elements per stage
constexpr int kOperand = 128 * kTK * 2;   // bytes of a CTA's part of A or B in a stage
constexpr int kStages = 6;
constexpr int kEpi = 8;
constexpr int kThreads = 96 + 32 * kEpi;
constexpr int kLong = 16;         // stages of a long item
constexpr int kTickets = 2;       // work items announced ahead
constexpr int kTile = 32 * 128;   // bytes of an epilogue warp's staging: 32 rows of 128 bytes
constexpr int kKeys = 256;        // targets kept in shared memory, when no more rows count
constexpr int kSmem = 1024 + kStages * 2 * kOperand + kEpi * kTile + 512 + kKeys * 4;
// Stages of a FP32 gradient's products that are added up in TMEM (see lm_grad_kernel).
constexpr int kPiece = 12;

// Device-side state of one call, in its workspace.
struct Rows {
  int* n;                   // [1] rows that count
  int* idx;                 // [cap] their row numbers, ascending
  int* target;              // [cap]
  int* skey;                // [cap] targets in ascending order (rows ascending among equals)
  int* srow;                // [cap] the counted row that each belongs to
  float* lse;               // [cap]
  float* cp;                // [cap] dlse - dlp: the factor of p
  float* dzt;               // [cap] dz at the target
  uint16_t* h;              // [cap][kp] gathered rows, zeros behind them and behind K
  float* acc;               // [slots][cap][ka] chunk partials of dh
  uint16_t* dz;             // [parts][cap][ring * chunk]
  int* ticket;              // next work item
  int* sdone;               // [chunks] warps that have written their part of a chunk's dz
  int* hdone;               // [chunks] warps that have added their part of its dh
  int* gdone;               // [chunks] products that have read it
  // more than kRun rows: runs of kRun of them, sorted
  int* run;                 // [runs][kRun] targets in ascending order, INT_MAX behind them
  int* run_n;               // [runs] rows that count
  // sums of dzt * h over 8 and 64 places of that order that have one target
  float* sum8;              // [cap / 8][kp]
  float* sum64;             // [cap / 64][kp]
  int2* run_at;             // [T] a row's place among those of its run that count, in row and in target order
};

struct Layout {
  int cap, kp, ka;          // rows, gathered row pitch, partial row pitch
  int chunk, chunks;        // columns per chunk, their number
  int slots;                // chunks: partials side by side; 1: added up as they come
  int ahead;                // chunks whose scores are formed ahead of their products
  int ring;                 // chunks of dz held
  int parts;                // bf16 parts of dz
  size_t off[20], bytes;
};

constexpr int kRun = 1024;
constexpr int kSums = 64;         // rows above which sums over equal targets are formed

// dh's partials lie side by side up to this size (few rows: its chunks are then
// independent of one another, and one kernel adds them up); above, each chunk
// is added to one array as it comes (4096 x 2048 rows: 34 MB, which L2 holds).
constexpr size_t kSlotBytes = size_t(192) << 20;
// dz held of each of its parts, where three chunks are less
constexpr int64_t kRingBytes = int64_t(192) << 20;

Layout layout(int T, int V, int K, bool f32) {
  Layout l;
  l.cap = (T + kTM - 1) / kTM * kTM;
  l.kp = (K + kTK - 1) / kTK * kTK;
  l.ka = (K + kTN - 1) / kTN * kTN;
  const int want = std::max(1, 152 / (l.ka / kTN));
  l.chunk = std::min(std::max(kMinChunk, (V + want - 1) / want), std::min(kMaxChunk, (V + 7) / 8));
  l.chunk = (l.chunk + kTN - 1) / kTN * kTN;
  l.chunks = (V + l.chunk - 1) / l.chunk;
  l.parts = f32 ? 2 : 1;
  const size_t part = size_t(l.cap) * l.ka * 4;
  l.slots = part * l.chunks <= kSlotBytes ? l.chunks : 1;
  // The scores of a chunk have to be done when its products start: enough
  // chunks ahead for about 256 stages of work in each of 76 pairs of CTAs, the
  // time of two dh items (200 x 151936: 48 stages 508 us, 144 430, 256 427; 284 x
  // 151936 x 256 with a FP32 gradient: 144 246 us, 256 233).
  const int64_t tm = l.cap / kTM, tk = l.ka / kTN, tn = l.chunk / kTN;
  const int64_t stages = tm * tn * (l.kp / kTK) + l.parts * (tm * tk * (l.chunk / kTK) + tn * tk * (l.cap / kTK));
  l.ahead = int(std::max<int64_t>(1, std::min<int64_t>(l.chunks - 1, (256 * 76 + stages - 1) / stages)));
  l.ring = std::min(l.chunks, 2 * l.ahead + 1);
  // No more of dz than kRingBytes of each part, or three chunks (T x V x K, bf16, with
  // what those stages ask for and with this: 8192 x 131072 x 256 589 MiB of workspace,
  // 2020 us, and 205, 1954; 1500 x 131072 x 256 433, 377, and 241, 357; 65536 x 4096 x
  // 256 619, 2126, and 299, 2181.  FP32: 2000 x 151936 x 256 621, 965, and 461, 977;
  // 8192 x 32000 x 256 709, 832, and 453, 862).  120 MiB, what L2 holds, made 16384 x
  // 4096 x 256 378 us instead of 283, and in FP32 2000 x 151936 x 256 1472.
  const int64_t most = std::max<int64_t>(3, kRingBytes / (int64_t(l.cap) * l.chunk * 2));
  if (l.ring > most) {
    l.ring = int(most);
    l.ahead = (l.ring - 1) / 2;
  }
  const size_t runs = T > kRun ? (T + kRun - 1) / kRun : 0;
  const size_t sums = T > kSums ? size_t(l.cap) * l.kp * 4 : 0;
  const size_t sizes[20] = {16, size_t(l.cap) * 4, size_t(l.cap) * 4, size_t(l.cap) * 4,
                            size_t(l.cap) * 4, size_t(l.cap) * 4, size_t(l.cap) * 4,
                            size_t(l.cap) * 4, size_t(l.cap) * l.kp * 2, part * l.slots,
                            size_t(l.parts) * l.cap * l.ring * l.chunk * 2, 16,
                            size_t(l.chunks) * 4, size_t(l.chunks) * 4, size_t(l.chunks) * 4,
                            runs * kRun * 4, runs * 4, runs * kRun * 8, sums / 8, sums / 64};
  l.bytes = 0;
  for (int i = 0; i < 20; ++i) {
    l.off[i] = l.bytes;
    l.bytes += (sizes[i] + 255) / 256 * 256;
  }
  return l;
}

Rows rows_of(const Layout& l, void* ws) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  Rows r;
  r.n = reinterpret_cast<int*>(b + l.off[0]);
  r.idx = reinterpret_cast<int*>(b + l.off[1]);
  r.target = reinterpret_cast<int*>(b + l.off[2]);
  r.skey = reinterpret_cast<int*>(b + l.off[3]);
  r.srow = reinterpret_cast<int*>(b + l.off[4]);
  r.lse = reinterpret_cast<float*>(b + l.off[5]);
  r.cp = reinterpret_cast<float*>(b + l.off[6]);
  r.dzt = reinterpret_cast<float*>(b + l.off[7]);
  r.h = reinterpret_cast<uint16_t*>(b + l.off[8]);
  r.acc = reinterpret_cast<float*>(b + l.off[9]);
  r.dz = reinterpret_cast<uint16_t*>(b + l.off[10]);
  r.ticket = reinterpret_cast<int*>(b + l.off[11]);
  r.sdone = reinterpret_cast<int*>(b + l.off[12]);
  r.hdone = reinterpret_cast<int*>(b + l.off[13]);
  r.gdone = reinterpret_cast<int*>(b + l.off[14]);
  r.run = reinterpret_cast<int*>(b + l.off[15]);
  r.run_n = reinterpret_cast<int*>(b + l.off[16]);
  r.run_at = reinterpret_cast<int2*>(b + l.off[17]);
  r.sum8 = reinterpret_cast<float*>(b + l.off[18]);
  r.sum64 = reinterpret_cast<float*>(b + l.off[19]);
  return r;
}

// ------------------------------------------------------------- gathering --
__device__ __forceinline__ int warp_add(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// whether row t has a gradient (a NaN is not 0: its row counts)
__device__ __forceinline__ bool row_counts(const float* __restrict__ dlp, const float* __restrict__ dlse, int t) {
  return !(dlp[t] == 0.f) || (dlse && !(dlse[t] == 0.f));
}

// The targets of a run of kRun rows in ascending order (bitonic, by target and
// row), and each row's places.
__global__ void __launch_bounds__(kRun) sort_rows_kernel(const int32_t* __restrict__ target,
                                                         const float* __restrict__ dlp,
                                                         const float* __restrict__ dlse, int T, int V, Rows r) {
  pdl_wait();
  pdl_trigger();
  __shared__ unsigned long long key[kRun];
  __shared__ int counts[32];
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31, t = blockIdx.x * kRun + i;
  int k = INT_MAX;
  if (t < T && row_counts(dlp, dlse, t)) {
    k = target[t];
    if (k < 0 || k >= V) k = INT_MAX;
  }
  const unsigned on = __ballot_sync(0xffffffffu, k != INT_MAX);
  if (lane == 0) counts[warp] = __popc(on);
  key[i] = (static_cast<unsigned long long>(k) << 32) | unsigned(i);
  __syncthreads();
  int before = __popc(on & ((1u << lane) - 1)), all = 0;
  for (int w = 0; w < 32; ++w) {
    before += w < warp ? counts[w] : 0;
    all += counts[w];
  }
  if (i == 0) r.run_n[blockIdx.x] = all;
  for (int size = 2; size <= kRun; size *= 2)
    for (int step = size / 2; step > 0; step /= 2) {
      const int a = 2 * i - (i & (step - 1)), b = a + step;
      if (i < kRun / 2 && (key[a] > key[b]) == ((a & size) == 0)) {
        const unsigned long long x = key[a];
        key[a] = key[b];
        key[b] = x;
      }
      __syncthreads();
    }
  r.run[blockIdx.x * kRun + i] = int(key[i] >> 32);
  // places in row order by their own thread, in target order by the thread they came to
  int2* at = r.run_at + blockIdx.x * kRun;
  at[i].x = before;
  at[unsigned(key[i])].y = i;
}

// A warp per row t of [0, cap).  It finds the number of rows that count (n) and
// of those before t (t's place i among them), and of those that come before it
// in the order of (target, row); writes row i's scalars, gathers its h, or clears
// dh of a row that does not count; and writes zeros to gathered row t where t lies
// between n and the next multiple of 256.  Up to kRun rows it counts over all of
// them; above, from the sorted runs, a lane searching every 32nd (65536 x 4096 x
// 256: the call took 4535 us with the former).
template <bool RUNS>
__global__ void __launch_bounds__(256) gather_kernel(
    const uint16_t* __restrict__ h, int64_t ldh, const uint16_t* __restrict__ W, int64_t ldw,
    const int32_t* __restrict__ target,
    const float* __restrict__ lse, const float* __restrict__ dlp, const float* __restrict__ dlse,
    int T, int V, int K, int kp, int cap, int chunks, void* dh, int64_t lddh, int dh_f32, Rows r,
    int* err) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) int key[kRun];      // the target of a row that counts, or -1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x * 8 + warp;
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < chunks; i += 256) r.sdone[i] = r.hdone[i] = r.gdone[i] = 0;
    if (threadIdx.x == 0) *r.ticket = 0;
  }
  int tg = -1;
  if (t < T) {
    const int x = target[t];
    if (row_counts(dlp, dlse, t)) {
      if (x >= 0 && x < V)
        tg = x;
      else if (lane == 0)
        raise_error(err, kErrBadIndex);
    }
  }
  int before = 0, all = 0, lower = 0;
  if (RUNS) {
    const int mine = t / kRun;
    for (int b = lane; b * kRun < T; b += 32) {
      const int n = r.run_n[b];
      all += n;
      before += b < mine ? n : 0;
      if (tg < 0 || b == mine) continue;
      // targets of the run below tg, or (rows before t) not above it
      const int limit = tg + (b < mine);
      int lo = 0, hi = n;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (r.run[b * kRun + mid] < limit) lo = mid + 1; else hi = mid;
      }
      lower += lo;
    }
    if (t < T && lane == 0) {
      const int2 at = r.run_at[t];
      before += at.x;
      lower += at.y;
    }
  } else {
    for (int j = threadIdx.x; j < kRun; j += 256) {
      int k = -1;
      if (j < T && row_counts(dlp, dlse, j)) {
        k = target[j];
        if (k < 0 || k >= V) k = -1;
      }
      key[j] = k;
    }
    __syncthreads();
    const int m = (T + 127) / 128 * 128;
    for (int j = lane * 4; j < m; j += 128) {
      const int4 k4 = *reinterpret_cast<const int4*>(key + j);
      const int k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool on = k[x] >= 0, first = j + x < t;
        all += on;
        before += on && first;
        lower += on && (k[x] < tg || (k[x] == tg && first));
      }
    }
  }
  all = warp_add(all);
  before = warp_add(before);
  lower = warp_add(lower);
  if (t == 0 && lane == 0) *r.n = all;
  if (t >= cap) return;
  if (t >= all && t < (all + kTM - 1) / kTM * kTM) {
    uint4* z = reinterpret_cast<uint4*>(r.h + int64_t(t) * kp);
    for (int c = lane; c < kp / 8; c += 32) z[c] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (t >= T) return;
  if (tg < 0) {
    if (dh) {
      if (dh_f32) {
        float* d = static_cast<float*>(dh) + t * lddh;
        for (int c = lane; c < K; c += 32) d[c] = 0.f;
      } else {
        uint16_t* d = static_cast<uint16_t*>(dh) + t * lddh;
        for (int c = lane; c < K; c += 32) d[c] = 0;
      }
    }
    return;
  }
  const int i = before;
  const uint4* src = reinterpret_cast<const uint4*>(h + t * ldh);
  const uint4* wt = reinterpret_cast<const uint4*>(W + tg * ldw);
  uint4* dst = reinterpret_cast<uint4*>(r.h + int64_t(i) * kp);
  float z = 0.f;
  constexpr int kAhead = 8;      // pieces in flight (2048 columns)
  for (int c0 = lane; c0 < kp / 8; c0 += 32 * kAhead) {
    uint4 v[kAhead], w[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      v[q] = w[q] = make_uint4(0u, 0u, 0u, 0u);
      if (c0 + 32 * q < K / 8) {
        v[q] = __ldg(src + c0 + 32 * q);
        w[q] = __ldg(wt + c0 + 32 * q);
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (c0 + 32 * q < kp / 8) dst[c0 + 32 * q] = v[q];
      const uint32_t a[4] = {v[q].x, v[q].y, v[q].z, v[q].w}, b[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        z = fmaf(__uint_as_float(a[x] << 16), __uint_as_float(b[x] << 16), z);
        z = fmaf(__uint_as_float(a[x] & 0xFFFF0000u), __uint_as_float(b[x] & 0xFFFF0000u), z);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (lane == 0) {
    r.idx[i] = t;
    r.target[i] = tg;
    r.skey[lower] = tg;
    r.srow[lower] = i;
    const float c = dlp[t], l = lse[t], cp = (dlse ? dlse[t] : 0.f) - c;
    r.lse[i] = l;
    r.cp[i] = cp;
    r.dzt[i] = fmaf(cp, expf(z - l), c);
  }
}

// v += f * 8 bf16
__device__ __forceinline__ void add_row8(float (&v)[8], float f, const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    v[2 * y] = fmaf(f, __uint_as_float(w[y] << 16), v[2 * y]);
    v[2 * y + 1] = fmaf(f, __uint_as_float(w[y] & 0xFFFF0000u), v[2 * y + 1]);
  }
}

// Of every 8 places of the order by target that have one target, the sum of
// dzt * h, and of every 64 the sum of these.  A token that many rows have as
// their target would otherwise have as many rows added to its row of dW one
// after another, by one lane (2458 rows of two targets: 1700 us).  A CTA per 64 places
// and 2048 columns.
__global__ void __launch_bounds__(256) target_sums_kernel(Rows r, int kp) {
  pdl_wait();
  pdl_trigger();
  const int n = *r.n, p0 = blockIdx.x * 64, c = blockIdx.y * 2048 + threadIdx.x * 8;
  if (p0 + 8 > n || c >= kp) return;
  float all[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) all[x] = 0.f;
  for (int p = p0; p < p0 + 64 && p + 8 <= n; p += 8) {
    if (r.skey[p] != r.skey[p + 7]) continue;
    uint4 u[8];
    float f[8], s[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int row = r.srow[p + x];
      f[x] = r.dzt[row];
      u[x] = *reinterpret_cast<const uint4*>(r.h + int64_t(row) * kp + c);
      s[x] = 0.f;
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) add_row8(s, f[x], u[x]);
    float4* d = reinterpret_cast<float4*>(r.sum8 + int64_t(p / 8) * kp + c);
    d[0] = make_float4(s[0], s[1], s[2], s[3]);
    d[1] = make_float4(s[4], s[5], s[6], s[7]);
#pragma unroll
    for (int x = 0; x < 8; ++x) all[x] += s[x];
  }
  if (p0 + 64 <= n && r.skey[p0] == r.skey[p0 + 63]) {
    float4* d = reinterpret_cast<float4*>(r.sum64 + int64_t(p0 / 64) * kp + c);
    d[0] = make_float4(all[0], all[1], all[2], all[3]);
    d[1] = make_float4(all[4], all[5], all[6], all[7]);
  }
}

// ----------------------------------------------------------------- GEMMs --
struct Maps {
  // K-major operands: boxes of 64 K elements of 128 rows; MN-major ones: boxes of
  // 64 K indices (rows) by two panels of 64 columns (W when K % 64: one panel)
  CUtensorMap hk, hn;   // gathered h: A of the scores, B of dW
  CUtensorMap wk, wn;   // W: B of the scores, B of dh
  CUtensorMap dk, dn;   // dz: A of dh, A of dW
  // stores of 32 rows by 128 bytes (dz in two parts: by 64 bytes)
  CUtensorMap ds, ws;   // dz, dW
};

struct Args {
  Rows r;
  int V, K, kp, ka, cap;
  int sums;                // sums over equal targets are there
  int w2;                  // W's map brings two panels at once (K % 64 == 0)
  int chunk, chunks, ahead, ring, slots;
  int parts, parts_h, parts_w;
  const uint16_t* W; int64_t ldw;
  void* dh; int64_t lddh; int dh_f32, dh_vec;
  void* dW; int64_t lddw; int dw_f32, dw_tma, accumulate;
  int* err;
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

enum { kScores = 0, kDh = 1, kDw = 2 };
// a work item as it is announced: type, origin of the tile, chunk
struct __align__(16) Item {
  int type, m0, n0, p;
};

// The work items of a call, in the order in which they are handed out: scores
// S(p) and products G(p) = dh and dW of chunk p as
//   S(0) .. S(ahead), G(0), S(ahead + 1), G(1), S(ahead + 2), ..., G(chunks - 1)
// so that a group's inputs are (all but) done when its turn comes.  Where dh's
// partials lie side by side, the groups behind the last scores are handed out
// together, the longer kind of item (dh where few rows count) first: one of these
// that starts last is the call's tail (2 x 131072 x 256 FP32: 176 us, now 141; 200 x 151936 433, now 423).
struct Plan {
  int n, tm, tk;
  int chunks, ahead;
  int last;                // columns of the last chunk
  int s, s_last;           // items of S
  int dh;                  // dh items of G
  bool h_first;            // dh's items are longer than dW's
  int g, g_last;           // items of G
  int head, body, total;   // S(0..ahead); those and the pairs G(p), S(p + ahead + 1)
};

__device__ __forceinline__ Plan plan_of(const Args& a) {
  Plan p;
  p.n = *a.r.n;
  p.tm = cdiv(p.n, kTM);
  p.tk = cdiv(a.K, kTN);
  p.chunks = a.chunks;
  p.ahead = a.ahead;
  p.last = a.V - (a.chunks - 1) * a.chunk;
  p.s = p.tm * (a.chunk / kTN);
  p.s_last = p.tm * cdiv(p.last, kTN);
  p.dh = a.dh ? p.tm * p.tk : 0;
  p.h_first = a.chunk / kTK * a.parts_h >= cdiv(p.n, kTK) * a.parts_w;
  p.g = p.dh + (a.dW ? p.tk * (a.chunk / kTM) : 0);
  p.g_last = p.dh + (a.dW ? p.tk * cdiv(p.last, kTM) : 0);
  const int first = min(p.ahead + 1, p.chunks);      // groups of scores at the head
  p.head = first == p.chunks ? (first - 1) * p.s + p.s_last : first * p.s;
  const int both = p.chunks - first;                 // pairs of groups
  p.body = p.head + (both ? both * (p.g + p.s) - p.s + p.s_last : 0);
  p.total = p.body + (p.chunks - both - 1) * p.g + p.g_last;
  return p;
}

__device__ __forceinline__ Item item_at(const Args& a, const Plan& p, int i) {
  Item it;
  bool scores = false;
  int j;                   // the item of its group
  const int both = p.chunks - min(p.ahead + 1, p.chunks);
  if (i < p.head) {
    scores = true;
    it.p = min(i / p.s, p.chunks - 1);
    j = i - it.p * p.s;
  } else if (i < p.body) {
    const int q = min((i - p.head) / (p.g + p.s), both - 1);
    j = i - p.head - q * (p.g + p.s);
    scores = j >= p.g;
    if (scores) j -= p.g;
    it.p = scores ? q + p.ahead + 1 : q;
  } else if (a.slots == 1) {
    const int q = min((i - p.body) / p.g, p.chunks - both - 1);
    j = i - p.body - q * p.g;
    it.p = both + q;
  } else {
    // dh's and dW's items that are left
    const int left = p.chunks - both, per = p.g - p.dh;
    const int all_h = p.dh * left, all_w = (left - 1) * per + p.g_last - p.dh;
    j = i - p.body;
    const bool h = p.h_first ? j < all_h : j >= all_w;
    if (h != p.h_first) j -= h ? all_w : all_h;
    const int q = h ? j / p.dh : min(j / per, left - 1);
    it.p = both + q;
    j = h ? j - q * p.dh : p.dh + j - q * per;
  }
  if (scores) {
    it.type = kScores;
    it.m0 = j % p.tm * kTM;
    it.n0 = j / p.tm * kTN;
  } else {
    it.type = j < p.dh ? kDh : kDw;       // dh's items come first: they are the long ones
    if (j >= p.dh) j -= p.dh;
    it.m0 = j / p.tk * kTM;
    it.n0 = j % p.tk * kTN;
  }
  return it;
}

// stages of one part of an item, and its parts
__device__ __forceinline__ int item_stages(const Args& a, const Plan& p, const Item& it, int& parts) {
  parts = it.type == kScores ? 1 : it.type == kDh ? a.parts_h : a.parts_w;
  if (it.type == kScores) return a.kp / kTK;
  return cdiv(it.type == kDw ? p.n : it.p == p.chunks - 1 ? p.last : a.chunk, kTK);
}

__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}
// a counter of finished warps reaches `want` (bounded wait)
__device__ bool wait_count(const int* p, int want, int* err) {
  if (load_acquire(p) >= want) return true;
  const uint64_t t0 = globaltimer_ns();
  while (load_acquire(p) < want) {
    __nanosleep(64);
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      raise_error(err, kErrTimeout);
      return false;
    }
  }
  return true;
}

// Everything that an item reads has been written, and nothing still reads what
// it overwrites.  sdone and hdone count kEpi warps of two CTAs per item, gdone items.
// A chunk that a pair has found ready is not asked for again.
struct Ready {
  int free = -1, scores = -1, sums = -1;
};
__device__ bool item_ready(const Args& a, const Plan& p, const Item& it, Ready& known) {
  constexpr int kPer = 2 * kEpi;
  const bool end = it.p == p.chunks - 1;
  if (it.type == kScores) {      // the ring's chunk of dz is free
    if (it.p < a.ring || known.free == it.p) return true;
    known.free = it.p;
    return wait_count(a.r.gdone + it.p - a.ring, p.g, a.err);
  }
  if (known.scores != it.p) {
    known.scores = it.p;
    if (!wait_count(a.r.sdone + it.p, kPer * (end ? p.s_last : p.s), a.err)) return false;
  }
  // partials that are added up as they come: the chunk before is in
  if (it.type != kDh || a.slots > 1 || it.p == 0 || known.sums == it.p) return true;
  known.sums = it.p;
  return wait_count(a.r.hdone + it.p - 1, kPer * p.dh, a.err);
}

// The first of n ascending keys that is v or more, by a warp: 32 probes a round
// (two rounds for 1024 keys, where a lane alone takes ten loads in a chain).
__device__ __forceinline__ int warp_lower_bound(const int* key, int n, int v, int lane) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int span = hi - lo, step = (span + 31) / 32;
    const int below = __popc(__ballot_sync(0xffffffffu, key[lo + min((lane + 1) * step, span) - 1] < v));
    hi = below == 32 ? hi : lo + min((below + 1) * step, span) - 1;
    lo += min(below * step, span);
  }
  return lo;
}

// The keys in [first, end) that are v0 + lane, of n ascending ones.
__device__ __forceinline__ void warp_keys(const int* key, int n, int v0, int lane, int& first, int& end) {
  const int base = warp_lower_bound(key, n, v0, lane);
  const int k = base + lane < n ? key[base + lane] - v0 : 32;
  const int some = __popc(__ballot_sync(0xffffffffu, k < 32));
  first = end = base;
  if (some < 32) {
    for (int i = 0; i < some; ++i) {
      const int o = __shfl_sync(0xffffffffu, k, i);
      first += o < lane;
      end += o <= lane;
    }
  } else {
    for (int up = 0; up < 2; ++up) {
      int lo = base, hi = n;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (key[mid] < v0 + lane + up) lo = mid + 1; else hi = mid;
      }
      (up ? end : first) = lo;
    }
  }
}

// 32 columns of a row from registers, bf16 or FP32
__device__ __forceinline__ void store32(void* base, int64_t off, int f32, bool vec, int left,
                                        const float (&v)[32]) {
  if (f32) {
    float* d = static_cast<float*>(base) + off;
    if (vec) {
#pragma unroll
      for (int x = 0; x < 32; x += 8) {
        uint32_t w[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) w[y] = __float_as_uint(v[x + y]);
        st_global_v8(d + x, w);
      }
    } else {
#pragma unroll
      for (int x = 0; x < 32; ++x)
        if (x < left) d[x] = v[x];
    }
  } else {
    uint16_t* d = static_cast<uint16_t*>(base) + off;
    if (vec) {
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) w[x] = bf2(v[2 * x], v[2 * x + 1]);
      st_global_v8(d, w);
      st_global_v8(d + 16, w + 8);
    } else {
#pragma unroll
      for (int x = 0; x < 32; ++x)
        if (x < left) d[x] = f2bf(v[x]);
    }
  }
}

// 32 columns of a lane's row into its warp's staging, as TMA reads them: 16-byte
// pieces, those of 128-byte rows exchanged by (row % 8), those of 64-byte rows by
// (row / 2 % 4), so that neither side meets bank conflicts.
__device__ __forceinline__ void stage_f32(uint32_t base, int lane, const float (&v)[32]) {
#pragma unroll
  for (int x = 0; x < 8; ++x)
    store_shared4(base + lane * 128 + ((x ^ (lane & 7)) << 4), __float_as_uint(v[4 * x]), __float_as_uint(v[4 * x + 1]),
                  __float_as_uint(v[4 * x + 2]), __float_as_uint(v[4 * x + 3]));
}
// the first (half 0) or second half of a 128-byte row
__device__ __forceinline__ void stage_bf16(uint32_t base, int lane, int half, const float (&v)[32]) {
#pragma unroll
  for (int x = 0; x < 4; ++x)
    store_shared4(base + lane * 128 + (((half * 4 + x) ^ (lane & 7)) << 4), bf2(v[8 * x], v[8 * x + 1]),
                  bf2(v[8 * x + 2], v[8 * x + 3]), bf2(v[8 * x + 4], v[8 * x + 5]), bf2(v[8 * x + 6], v[8 * x + 7]));
}
// a 64-byte row
__device__ __forceinline__ void stage_part(uint32_t base, int lane, const float (&v)[32]) {
#pragma unroll
  for (int x = 0; x < 4; ++x)
    store_shared4(base + lane * 64 + ((x ^ ((lane >> 1) & 3)) << 4), bf2(v[8 * x], v[8 * x + 1]),
                  bf2(v[8 * x + 2], v[8 * x + 3]), bf2(v[8 * x + 4], v[8 * x + 5]), bf2(v[8 * x + 6], v[8 * x + 7]));
}

// v += 32 columns of a row, bf16 or FP32
__device__ __forceinline__ void add32(const void* base, int64_t off, int f32, bool vec, int left, float (&v)[32]) {
  if (vec && f32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float4 o = s[x];
      v[4 * x] += o.x; v[4 * x + 1] += o.y; v[4 * x + 2] += o.z; v[4 * x + 3] += o.w;
    }
  } else if (vec) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint4 u = s[x];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        v[8 * x + 2 * y] += __uint_as_float(w[y] << 16);
        v[8 * x + 2 * y + 1] += __uint_as_float(w[y] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (x < left) v[x] += f32 ? static_cast<const float*>(base)[off + x] : bf2f(static_cast<const uint16_t*>(base)[off + x]);
  }
}

// v += f * 32 bf16 of a row (16-byte aligned), the first `left` of them
__device__ __forceinline__ void add_row32(float (&v)[32], float f, const uint16_t* row, int left) {
  const uint4* r = reinterpret_cast<const uint4*>(row);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if (8 * x >= left) break;
    const uint4 u = __ldg(r + x);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      v[8 * x + 2 * y] = fmaf(f, __uint_as_float(w[y] << 16), v[8 * x + 2 * y]);
      v[8 * x + 2 * y + 1] = fmaf(f, __uint_as_float(w[y] & 0xFFFF0000u), v[8 * x + 2 * y + 1]);
    }
  }
}

// All three products of a call in one launch: persistent pairs of CTAs
// (clusters of two), 352 threads each.  Warp 0 = TMA producer; warp 1 = TMEM
// owner and, in the pair's first CTA, MMA issuer, in the second the one that
// counts finished products; warps 2..9 = epilogue (lane quarter = warp % 4,
// column half = (warp - 2) / 4); warp 10 of the first CTA takes work items.
// A tile is 256 x 256: each CTA loads its 128 rows of A and of B, the first CTA
// issues cta_group::2 MMAs over both, and each CTA's TMEM gets its 128 rows.
// full barriers live in the first CTA and count both CTAs' bytes; empty and
// tfull are signalled in both by multicast commits; both epilogues arrive on
// the first CTA's tempty.
//
// Items are taken from a counter in their order and announced to both CTAs
// through a ring in shared memory.  An item depends on items before it only,
// and those are taken by pairs that run: whatever else the GPU runs, the waits
// end.  Taking an item, finding its inputs ready and announcing it is a chain of
// round trips to L2, thousands of cycles long, which is why a warp of its own
// does it (by the producer, 13 rows x 4096: 25.4 us, now 22.1; 4096 x 151936:
// 3815 -> 3700 us), but only two ahead: items held by a pair that is busy are
// late for those that wait for them (200 x 151936, four ahead 524 us, two 430).
// Barrier arrivals that hand nothing over are relaxed, since a release waits
// for the warp's stores; an epilogue warp stores through shared memory and TMA,
// 32 rows of 128 bytes at a time (stores by lanes, a row each: 541 us, now 504).
//
// F32: the MMAs' FP32 accumulators truncate, so that a sum's error grows with
// its number of steps.  For FP32 gradients an accumulator takes kPiece stages
// (768 K elements); the epilogue adds the pieces up in registers, rounding to
// nearest.  1000 x 32003 x 2048, 2-norm against 64 bits: without pieces 3.3e-6 (dh)
// and 2.2e-6 (dW), with pieces of 16 stages 1.2e-6 and 1.1e-6, of 12 7.0e-7 and
// 6.4e-7 (391 us), of 8 5.8e-7 and 5.5e-7 (409 us).
//
// What bounds it: at 4096 x 151936 a stage of 64 K elements (512 cycles at the
// MMA's rate) takes 670 under the card's power limit, as cuBLAS's products do;
// small calls the chain of scores, products and fold.
template <bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    lm_grad_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  extern __shared__ uint8_t smem_raw[];
  // (the offset is the same in both CTAs of a pair)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kOperand;
  uint8_t* staging = sB + kStages * kOperand;
  int* keys = reinterpret_cast<int*>(staging + kEpi * kTile);
  uint64_t* bars = reinterpret_cast<uint64_t*>(keys + kKeys);
  Item* ring = reinterpret_cast<Item*>(bars);                        // [kTickets]
  bars += 2 * kTickets;
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kStages);
  const uint32_t tfull0 = smem_u32(bars + 2 * kStages), tempty0 = smem_u32(bars + 2 * kStages + 2);
  const uint32_t kfull0 = smem_u32(bars + 2 * kStages + 4);
  const uint32_t kempty0 = smem_u32(bars + 2 * kStages + 4 + kTickets);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4 + 2 * kTickets);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_rank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(tfull0 + 8 * j, 1);
      mbar_init(tempty0 + 8 * j, 2 * kEpi + 1);     // (and the counter of finished products)
    }
    for (int j = 0; j < kTickets; ++j) {
      mbar_init(kfull0 + 8 * j, 1);
      mbar_init(kempty0 + 8 * j, 2 * kEpi + 4);     // readers: the warps of both CTAs but the taker
    }
    fence_barrier_init();
    tma_prefetch_desc(&maps.hk);
    tma_prefetch_desc(&maps.wk);
    tma_prefetch_desc(&maps.dk);
    tma_prefetch_desc(&maps.hn);
    tma_prefetch_desc(&maps.wn);
    tma_prefetch_desc(&maps.dn);
    tma_prefetch_desc(&maps.ds);
    if (a.dw_tma) tma_prefetch_desc(&maps.ws);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc2(smem_u32(tmem_slot), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const Plan plan = plan_of(a);

  // the next announced item (type < 0: no more); false: the wait ran out
  int seq = 0;
  auto next_item = [&](Item& it) {
    const int k = seq % kTickets;
    if (!mbar_wait_cluster(kfull0 + 8 * k, (seq / kTickets) & 1, a.err)) return false;
    const int4 v = load_shared4(smem_u32(ring + k));
    it.type = v.x; it.m0 = v.y; it.n0 = v.z; it.p = v.w;
    ++seq;
    return true;
  };
  // (behind a branch on what was read: the slot may be written from then on)
  auto release_item = [&]() {
    mbar_arrive_relaxed(cluster_addr(kempty0 + 8 * ((seq - 1) % kTickets), 0));
  };

  // accumulators that an item's products go through
  auto pieces = [&](const Item& it) {
    int parts;
    const int nk = item_stages(a, plan, it, parts) * parts;
    return F32 ? cdiv(nk, kPiece) : int(nk > 0);
  };

  int issued = 0;
  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int s = 0, turn = 0;      // stage, its use
      Item it, before;
      before.type = before.p = -1;
      while (ok && next_item(it)) {
        if (it.type < 0) break;
        release_item();
        if (it.type != before.type || it.p != before.p)
          fence_proxy_async_all();    // what others wrote is read by TMA
        before = it;
        int parts;
        const int nk = item_stages(a, plan, it, parts);
        const int dz0 = it.p % a.ring * a.chunk, v0 = it.p * a.chunk;
        const int m = it.m0 + rank * 128, nn = it.n0 + rank * 128;
        for (int part = 0; part < parts && ok; ++part) {
          const int dzr = part * a.cap;
          for (int k = 0; k < nk; ++k) {
            if (turn > 0 && !mbar_wait(empty0 + 8 * s, (turn - 1) & 1, a.err)) {
              ok = false;
              break;
            }
            const uint32_t bar = cluster_addr(full0 + 8 * s, 0);
            const uint32_t da = smem_u32(sA + s * kOperand), db = smem_u32(sB + s * kOperand);
            if (rank == 0) mbar_expect_tx(full0 + 8 * s, 4 * kOperand);
            if (it.type == kScores) {
              tma2_load_2d(da, &maps.hk, bar, k * kTK, m);
              tma2_load_2d(db, &maps.wk, bar, k * kTK, v0 + nn);
            } else if (it.type == kDh) {
              tma2_load_2d(da, &maps.dk, bar, dz0 + k * kTK, dzr + m);
              if (a.w2) {
                tma2_load_3d(db, &maps.wn, bar, 0, v0 + k * kTK, nn / 64);
              } else {
                tma2_load_2d(db, &maps.wn, bar, nn, v0 + k * kTK);
                tma2_load_2d(db + kOperand / 2, &maps.wn, bar, nn + 64, v0 + k * kTK);
              }
            } else {
              tma2_load_3d(da, &maps.dn, bar, 0, dzr + k * kTK, (dz0 + m) / 64);
              tma2_load_3d(db, &maps.hn, bar, 0, k * kTK, nn / 64);
            }
            ++issued;
            if (++s == kStages) {
              s = 0;
              ++turn;
            }
          }
        }
      }
    }
  } else if (warp == 2 + kEpi) {
    // takes work items, waits for what they read and announces them
    if (lane == 0 && rank == 0) {
      Ready known;
      bool ok = true;
      while (ok) {
        Item it;
        it.type = -1;
        const int taken = atomicAdd(a.r.ticket, 1);
        if (taken < plan.total) {
          it = item_at(a, plan, taken);
          if (!item_ready(a, plan, it, known)) it.type = -1;
        }
        const int k = seq % kTickets;
        if (seq >= kTickets && !mbar_wait_cluster(kempty0 + 8 * k, ((seq / kTickets) - 1) & 1, a.err)) break;
        for (int c = 0; c < 2; ++c) {
          store_cluster(cluster_addr(smem_u32(ring + k), c), make_int4(it.type, it.m0, it.n0, it.p));
          mbar_arrive_cluster(cluster_addr(kfull0 + 8 * k, c));
        }
        ++seq;
        ok = it.type >= 0;
        // (F32, whose long items are twice as long: the next one once all have read
        // this one; 1000 x 32003 437 us, now 418, but 200 x 151936 in bf16 444, then 462)
        int parts;
        if (F32 && ok && item_stages(a, plan, it, parts) * parts >= kLong)
          ok = mbar_wait_cluster(kempty0 + 8 * k, ((seq - 1) / kTickets) & 1, a.err);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int s = 0, turn = 0, j = 0;
      bool ok = true;
      Item it;
      while (ok && next_item(it)) {
        if (it.type < 0) break;
        release_item();
        int parts;
        const int nk = item_stages(a, plan, it, parts) * parts;
        uint32_t dt = 0;
        // K-major: 64 K elements of a row in 128 bytes; MN-major: 64 rows or
        // columns of the output of one K index
        const bool a_mn = it.type == kDw, b_mn = it.type != kScores;
        const uint32_t idesc =
            idesc_mma(1u, kTM, kTN) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
        const uint32_t astep = a_mn ? 2048 : 32, bstep = b_mn ? 2048 : 32;
        for (int kb = 0; kb < nk; ++kb) {
          const bool begin = F32 ? kb % kPiece == 0 : kb == 0;
          if (begin) {
            if (j >= 2 && !mbar_wait_cluster(tempty0 + 8 * (j & 1), ((j >> 1) - 1) & 1, a.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            dt = tmem + (j & 1) * kTN;
          }
          if (!mbar_wait(full0 + 8 * s, turn & 1, a.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * kOperand), b0 = smem_u32(sB + s * kOperand);
          const uint64_t ad = a_mn ? sdesc_mn_sw128(a0, kOperand / 2, 1024) : sdesc_k_sw128(a0);
          const uint64_t bd = b_mn ? sdesc_mn_sw128(b0, kOperand / 2, 1024) : sdesc_k_sw128(b0);
#pragma unroll
          for (int kk = 0; kk < kTK / 16; ++kk)     // (addresses count 16 bytes)
            umma2_f16(dt, ad + kk * (astep >> 4), bd + kk * (bstep >> 4), idesc, begin && kk == 0 ? 0u : 1u);
          umma2_commit(empty0 + 8 * s);
          if (kb == nk - 1 || (F32 && kb % kPiece == kPiece - 1)) {
            umma2_commit(tfull0 + 8 * (j & 1));
            ++j;
          }
          if (++s == kStages) {
            s = 0;
            ++turn;
          }
        }
      }
    } else if (lane == 0) {
      // A product is finished: its reads of dz are done.  (The epilogue's own
      // threads would wait for their stores first.)
      int j = 0;
      Item it;
      while (next_item(it)) {
        if (it.type < 0) break;
        release_item();
        bool ok = true;
        for (int left = pieces(it); ok && left > 0; --left, ++j) {
          ok = mbar_wait(tfull0 + 8 * (j & 1), (j >> 1) & 1, a.err);
          if (ok) mbar_arrive_relaxed(cluster_addr(tempty0 + 8 * (j & 1), 0));
        }
        if (!ok) break;
        if (it.type != kScores) add_release(a.r.gdone + it.p, 1);
      }
    }
  } else {
    const int q = warp & 3, col0 = ((warp - 2) >> 2) * (kTN / 2);
    const uint32_t tile = smem_u32(staging) + (warp - 2) * kTile;
    const int* skey = a.r.skey;
    if (plan.n <= kKeys) {
      for (int i = threadIdx.x - 64; i < plan.n; i += 32 * kEpi) keys[i] = a.r.skey[i];
      asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpi) : "memory");
      skey = keys;
    }
    // the staging may be written again; it has been written and is stored
    auto stage_begin = [&]() {
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    };
    auto stage_end = [&](const CUtensorMap* map, int x, int y, int y2) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(map, tile, x, y);
        if (y2 >= 0) tma_store_2d(map, tile + kTile / 2, x, y2);
        bulk_commit();
      }
    };
    int j = 0;
    Item it;
    while (__all_sync(0xffffffffu, next_item(it))) {
      if (it.type < 0) break;
      if (lane == 0) release_item();
      const int np = pieces(it);
      const uint32_t ta = tmem + col0 + (uint32_t(q * 32) << 16);
      const int row = it.m0 + rank * 128 + q * 32 + lane;
      const int v0 = it.p * a.chunk, cols = min(a.chunk, a.V - v0);
      // What the row needs is loaded before its products are waited for (after
      // them, these chains of loads were most of the epilogue of a call of few
      // rows, whose dW tiles are four stages long).
      const bool live = it.type == kDw ? row < cols : row < plan.n;
      const bool end = it.type == kDh && a.slots == 1 && it.p == a.chunks - 1;
      float lse = 0.f, cp = 0.f, dzt = 0.f;
      int tgt = -1, first = 0, last = 0, r0 = 0;
      int64_t out = 0;
      if (it.type == kDw) {
        // the counted rows whose target this row of dW is
        warp_keys(skey, plan.n, v0 + row - lane, lane, first, last);
        if (first < last) {
          r0 = a.r.srow[first];
          dzt = a.r.dzt[r0];
        }
      } else if (live && it.type == kScores) {
        lse = a.r.lse[row];
        cp = a.r.cp[row];
        tgt = a.r.target[row];
      } else if (live && end) {
        dzt = a.r.dzt[row];
        out = a.r.idx[row] * a.lddh;
        tgt = a.r.target[row];
      }
      bool ok = true;
      // (bf16: unrolled by two; the three kinds of items unrolled whole miss the
      // instruction cache, 200 x 151936 439 us against 433)
      constexpr int kUnroll = F32 ? kTN / 64 : 2;
      float acc[F32 ? kTN / 64 : 1][32];
      if (F32) {
#pragma unroll
        for (int g = 0; g < kTN / 64; ++g)
#pragma unroll
          for (int x = 0; x < 32; ++x) acc[F32 ? g : 0][x] = 0.f;
        for (int i = 0; i < np; ++i, ++j) {
          ok = __all_sync(0xffffffffu, mbar_wait(tfull0 + 8 * (j & 1), (j >> 1) & 1, a.err));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < kTN / 64; ++g) {
            uint32_t v[32];
            tmem_ld32(ta + (j & 1) * kTN + g * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) acc[F32 ? g : 0][x] += __uint_as_float(v[x]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(cluster_addr(tempty0 + 8 * (j & 1), 0));
        }
      } else if (np > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(tfull0 + 8 * (j & 1), (j >> 1) & 1, a.err));
        tc_fence_after();
      }
      if (!ok) break;
      // the products of 32 columns
      auto product = [&](int g, float (&f)[32]) {
        if (F32) {
#pragma unroll
          for (int x = 0; x < 32; ++x) f[x] = acc[F32 ? g : 0][x];
        } else if (np > 0) {
          uint32_t v[32];
          tmem_ld32(ta + (j & 1) * kTN + g * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x) f[x] = __uint_as_float(v[x]);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) f[x] = 0.f;
        }
      };
      if (it.type == kScores) {
        const int tc = live ? tgt - v0 : -1;                 // the target's column of the chunk
        const int x0 = it.p % a.ring * a.chunk + it.n0 + col0, y0 = row - lane;
#pragma unroll(kUnroll)
        for (int g = 0; g < kTN / 64; ++g) {
          float d[32];
          product(g, d);
          const int c = it.n0 + col0 + g * 32;               // column of the chunk
          // (without a condition: one per column compiled to branches, and the tile's
          // exponentials took 13000 cycles, now 5000)
#pragma unroll
          for (int x = 0; x < 32; ++x) d[x] = cp * expf(d[x] - lse);
          if (y0 + 32 > plan.n) {                            // (0 times an infinite weight)
#pragma unroll
            for (int x = 0; x < 32; ++x) d[x] = live ? d[x] : 0.f;
          }
          if (c + 32 > cols) {
#pragma unroll
            for (int x = 0; x < 32; ++x) d[x] = c + x < cols ? d[x] : 0.f;
          }
          if (tc >= c && tc < c + 32) {                      // (the target's term is added apart)
#pragma unroll
            for (int x = 0; x < 32; ++x) d[x] = c + x == tc ? 0.f : d[x];
          }
          if (F32) {
            stage_begin();
            stage_part(tile, lane, d);
#pragma unroll
            for (int x = 0; x < 32; ++x) d[x] -= bf2f(f2bf(d[x]));
            stage_part(tile + kTile / 2, lane, d);
            stage_end(&maps.ds, x0 + g * 32, y0, a.cap + y0);
          } else {
            if (g % 2 == 0) stage_begin();
            stage_bf16(tile, lane, g % 2, d);
            if (g % 2) stage_end(&maps.ds, x0 + (g - 1) * 32, y0, -1);
          }
        }
      } else if (it.type == kDh) {
        const bool add = a.slots == 1 && it.p > 0;
        float* dst = a.r.acc + (int64_t(a.slots > 1 ? it.p : 0) * a.cap + row) * a.ka + it.n0 + col0;
        const uint16_t* wr = a.W + (end && live ? tgt * a.ldw : 0);
#pragma unroll(kUnroll)
        for (int g = 0; g < kTN / 64; ++g) {
          const int c = it.n0 + col0 + g * 32;
          float f[32];
          product(g, f);
          if (!live) continue;
          if (add) {
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 o = __ldcg(reinterpret_cast<const float4*>(dst + g * 32 + x));
              f[x] = o.x + f[x];
              f[x + 1] = o.y + f[x + 1];
              f[x + 2] = o.z + f[x + 2];
              f[x + 3] = o.w + f[x + 3];
            }
          }
          if (!end) {
            store32(dst, g * 32, 1, true, 32, f);
          } else if (c < a.K) {
            add_row32(f, dzt, wr + c, a.K - c);
            store32(a.dh, out + c, a.dh_f32, a.dh_vec && c + 32 <= a.K, a.K - c, f);
          }
        }
      } else {
        const int vr = v0 + row;                             // row of dW
        const bool targets = __any_sync(0xffffffffu, first < last);
#pragma unroll(kUnroll)
        for (int g = 0; g < kTN / 64; ++g) {
          const int c = it.n0 + col0 + g * 32;
          float f[32];
          product(g, f);
          const bool on = live && c < a.K;
          if (targets && on) {
            // (sums over equal targets where they are)
            for (int t = first; t < last;) {
              if (a.sums && (t & 7) == 0 && t + 8 <= last) {
                const bool more = (t & 63) == 0 && t + 64 <= last;
                add32(more ? a.r.sum64 : a.r.sum8, int64_t(t >> (more ? 6 : 3)) * a.kp + c, 1, true, 32, f);
                t += more ? 64 : 8;
              } else {
                const int r = t == first ? r0 : a.r.srow[t];
                add_row32(f, t == first ? dzt : a.r.dzt[r], a.r.h + int64_t(r) * a.kp + c, 32);
                ++t;
              }
            }
          }
          if (a.accumulate && on)
            add32(a.dW, int64_t(vr) * a.lddw + c, a.dw_f32, a.dw_tma && c + 32 <= a.K, a.K - c, f);
          // (a tile's store leaves out what lies behind V and K, but none starts there)
          if (!a.dw_tma) {
            if (on) store32(a.dW, int64_t(vr) * a.lddw + c, a.dw_f32, false, a.K - c, f);
          } else if (a.dw_f32) {
            stage_begin();
            stage_f32(tile, lane, f);
            if (c < a.K && vr - lane < a.V) stage_end(&maps.ws, c, vr - lane, -1);
          } else {
            if (g % 2 == 0) stage_begin();
            stage_bf16(tile, lane, g % 2, f);
            if (g % 2 && c - 32 < a.K && vr - lane < a.V) stage_end(&maps.ws, c - 32, vr - lane, -1);
          }
        }
      }
      if (!F32 && np > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(cluster_addr(tempty0 + 8 * (j & 1), 0));
        ++j;
      }
      if (it.type == kScores || (it.type == kDh && a.slots == 1)) {
        __syncwarp();
        if (lane == 0) {
          if (it.type == kScores) {      // dz was written by TMA and is read by TMA
            bulk_wait();
            fence_proxy_async_all();
          }
          __threadfence();
          add_release((it.type == kScores ? a.r.sdone : a.r.hdone) + it.p, 1);
        }
      }
    }
    if (lane == 0) bulk_wait();
  }
  // the pair's copies have landed, and its last remote arrivals, before it exits
  if (warp == 0 && lane == 0 && rank == 0) {
    for (int i = max(0, issued - kStages); i < issued; ++i)
      mbar_wait(full0 + 8 * (i % kStages), (i / kStages) & 1, a.err, 100000000ull);
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, 512);
}

// dh of the counted rows from partials side by side: the chunks in ascending
// order, then the target's term.  4 columns a thread, a CTA per row and 1024
// columns; 8 chunks are loaded ahead of their additions.
__global__ void __launch_bounds__(256) dh_fold_kernel(Rows r, const uint16_t* __restrict__ W,
                                                      int64_t ldw, int K, int ka, int cap, int slots,
                                                      void* dh, int64_t lddh, int f32) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, c = blockIdx.y * 1024 + threadIdx.x * 4;
  if (i >= *r.n || c >= K) return;
  const int64_t out = r.idx[i] * lddh + c;
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(W + r.target[i] * ldw + c));
  const float dzt = r.dzt[i];
  const float* src = r.acc + int64_t(i) * ka + c;
  const int64_t pitch = int64_t(cap) * ka;
  float4 s = __ldcg(reinterpret_cast<const float4*>(src));
  for (int k0 = 1; k0 < slots; k0 += 8) {
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k0 + k < slots) v[k] = __ldcg(reinterpret_cast<const float4*>(src + (k0 + k) * pitch));
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k0 + k < slots) {
        s.x += v[k].x; s.y += v[k].y; s.z += v[k].z; s.w += v[k].w;
      }
  }
  const float o[4] = {fmaf(dzt, __uint_as_float(w.x << 16), s.x), fmaf(dzt, __uint_as_float(w.x & 0xFFFF0000u), s.y),
                      fmaf(dzt, __uint_as_float(w.y << 16), s.z), fmaf(dzt, __uint_as_float(w.y & 0xFFFF0000u), s.w)};
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if (f32)
      static_cast<float*>(dh)[out + x] = o[x];
    else
      static_cast<uint16_t*>(dh)[out + x] = f2bf(o[x]);
  }
}

// bf16 rows: boxes of 64 columns and box_rows rows, or (panels) of two such
// panels of {64, rows, K / 64}
// (stores) of `cols` columns
bool map_rows(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int64_t ld, int box_rows,
              bool panels, int cols = 64, bool f32 = false) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint32_t es[3] = {1, 1, 1}, box[3] = {cuuint32_t(cols), cuuint32_t(box_rows), 2};
  const cuuint64_t panel_dims[3] = {64, cuuint64_t(rows), cuuint64_t(K / 64)};
  const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
  const int size = f32 ? 4 : 2;
  const cuuint64_t strides[2] = {cuuint64_t(ld * size), 128};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, panels ? 3 : 2, const_cast<void*>(base),
            panels ? panel_dims : dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            cols * size == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F32>
biv_status launch_grad(const Maps& maps, const Args& a, cudaStream_t s) {
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (cudaFuncSetAttribute(lm_grad_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
        cudaSuccess)
      return set_error(BIV_ERR_CUDA, "lm_head_backward: cannot set shared memory size");
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  // no more pairs than a chunk's items can be, and one per two SMs
  const int64_t tm = a.cap / kTM, tn = a.chunk / kTN, tk = a.ka / kTN;
  const int64_t most = std::max(tm * tn, tk * (tm + tn)) * a.chunks;
  const int sms = sm_count() > 0 ? sm_count() : 148;
  const int pairs = int(std::max<int64_t>(1, std::min<int64_t>(most, sms / 2)));
  launch_pdl(lm_grad_kernel<F32>, 2 * pairs, kThreads, kSmem, s, maps, a);
  return check_launch("lm_head_backward");
}

// --------------------------------------------------------------- forward --
constexpr int kLossRows = 8;      // rows per CTA, a warp each
constexpr int kMaxParts = 1024;   // blocks whose sums the last kernel adds up

struct LossSums { double w, nll, sq; };

// whether a row counts
__device__ __forceinline__ bool row_on(int target, float weight, int ignore) {
  return target != ignore && weight != 0.f;
}

// The 128-row tiles with a counted row, in ascending order: their number, then
// their indexes.  One CTA, a warp per tile.
__global__ void __launch_bounds__(1024) row_tiles_kernel(const int32_t* __restrict__ target,
                                                         const float* __restrict__ weight, int T, int ignore,
                                                         int* __restrict__ list) {
  pdl_wait();
  pdl_trigger();
  __shared__ int some[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int t0 = 0; t0 < T; t0 += 32 * 128) {
    bool on = false;
    for (int t = t0 + warp * 128 + lane, i = 0; i < 4 && t < T; ++i, t += 32)
      on |= row_on(target[t], weight ? weight[t] : 1.f, ignore);
    on = __any_sync(0xffffffffu, on);
    if (lane == 0) some[warp] = on;
    __syncthreads();
    const unsigned all = __ballot_sync(0xffffffffu, some[lane]);
    if (on && lane == 0) list[1 + n + __popc(all & ((1u << warp) - 1))] = t0 / 128 + warp;
    n += __popc(all);
    __syncthreads();
  }
  if (threadIdx.x == 0) list[0] = n;
}

// lp and lse of a row as biv_lm_head_logprob merges the groups (lane l takes
// groups l, l + 32, ... in order, then a xor tree), and on lane 0 its terms of the sums.
__device__ __forceinline__ void row_loss(const float2* __restrict__ g, int ng, const float* __restrict__ zt,
                                         int row, int tg, float wt, int V, float* lp, float* lse, int* err,
                                         LossSums& mine, float& l) {
  const int lane = threadIdx.x & 31;
  g += int64_t(row) * ng;
  float mx = -INFINITY;
  for (int i = lane; i < ng; i += 32) mx = fmaxf(mx, g[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float s = 0.f;
  for (int i = lane; i < ng; i += 32) {
    const float2 v = g[i];
    s = fmaf(v.y, expf(v.x - mx), s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) {
    l = mx + logf(s);
    float p = NAN;
    if (tg < 0 || tg >= V)
      raise_error(err, kErrBadIndex);
    else
      p = zt[row] - l;
    lp[row] = p;
    lse[row] = l;
    mine.w += wt;
    mine.nll -= double(wt) * p;
    mine.sq += double(wt) * l * l;
  }
}

__device__ __forceinline__ LossSums warp_sums(LossSums s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
    s.nll += __shfl_xor_sync(0xffffffffu, s.nll, o);
    s.sq += __shfl_xor_sync(0xffffffffu, s.sq, o);
  }
  return s;
}

// what the loss divides by
__device__ __forceinline__ double loss_scale(const LossSums& s, int mean, float norm) {
  const double over = mean ? s.w : double(norm);
  return over != 0. ? 1. / over : 0.;
}
__device__ __forceinline__ void write_stats(const LossSums& s, double inv, float z_coef, float* stats) {
  stats[0] = float((s.nll + double(z_coef) * s.sq) * inv);
  stats[1] = float(s.nll * inv);
  stats[2] = float(s.sq * inv);
  stats[3] = float(s.w);
}
__device__ __forceinline__ void write_coefs(int t, float wt, bool on, float l, double inv, float z_coef, float* dlp,
                                            float* dlse) {
  const float c = on ? float(wt * inv) : 0.f;
  if (dlp) dlp[t] = -c;
  if (dlse) dlse[t] = c == 0.f ? 0.f : float(2. * z_coef * c * l);
}

// Rows, and sums of the counted rows of each CTA.
__global__ void __launch_bounds__(kLossRows * 32) lse_rows_kernel(
    const float2* __restrict__ groups, int ng, const float* __restrict__ zt,
    const int32_t* __restrict__ target, const float* __restrict__ weight, int T, int V, int ignore,
    float* __restrict__ lp, float* __restrict__ lse, LossSums* __restrict__ parts, int* err) {
  pdl_wait();
  pdl_trigger();
  __shared__ LossSums sums[kLossRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  LossSums mine = {0., 0., 0.};
  for (int row = blockIdx.x * kLossRows + warp; row < T; row += gridDim.x * kLossRows) {
    const int tg = target[row];
    const float wt = weight ? weight[row] : 1.f;
    float l;
    if (row_on(tg, wt, ignore))
      row_loss(groups, ng, zt, row, tg, wt, V, lp, lse, err, mine, l);
    else if (lane == 0)
      lp[row] = lse[row] = 0.f;
  }
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    LossSums t = sums[0];
    for (int w = 1; w < kLossRows; ++w) {
      t.w += sums[w].w;
      t.nll += sums[w].nll;
      t.sq += sums[w].sq;
    }
    parts[blockIdx.x] = t;
  }
}

// Every CTA adds the blocks' sums in one order (32 lanes, then a xor tree) and
// writes its rows' coefficients; CTA 0 the statistics.
__global__ void __launch_bounds__(256) loss_rows_kernel(
    const LossSums* __restrict__ parts, int nparts, const int32_t* __restrict__ target,
    const float* __restrict__ weight, const float* __restrict__ lse, int T, int ignore,
    float z_coef, int mean, float norm, float* __restrict__ dlp, float* __restrict__ dlse,
    float* __restrict__ stats) {
  pdl_wait();
  pdl_trigger();
  __shared__ double scale;
  if (threadIdx.x < 32) {
    LossSums s = {0., 0., 0.};
    for (int i = threadIdx.x; i < nparts; i += 32) {
      s.w += parts[i].w;
      s.nll += parts[i].nll;
      s.sq += parts[i].sq;
    }
    s = warp_sums(s);
    if (threadIdx.x == 0) {
      scale = loss_scale(s, mean, norm);
      if (blockIdx.x == 0) write_stats(s, scale, z_coef, stats);
    }
  }
  __syncthreads();
  const double inv = scale;
  for (int t = blockIdx.x * 256 + threadIdx.x; t < T; t += gridDim.x * 256) {
    const float wt = weight ? weight[t] : 1.f;
    write_coefs(t, wt, row_on(target[t], wt, ignore), lse[t], inv, z_coef, dlp, dlse);
  }
}

// Both for at most 32 rows, a warp each, in one CTA (13 rows of 4096: 15.3 us,
// with two kernels 17.1).
__global__ void __launch_bounds__(1024) few_rows_kernel(
    const float2* __restrict__ groups, int ng, const float* __restrict__ zt,
    const int32_t* __restrict__ target, const float* __restrict__ weight, int T, int V, int ignore,
    float z_coef, int mean, float norm, float* __restrict__ lp, float* __restrict__ lse,
    float* __restrict__ dlp, float* __restrict__ dlse, float* __restrict__ stats, int* err) {
  pdl_wait();
  pdl_trigger();
  __shared__ LossSums sums[32];
  __shared__ double scale;
  const int row = threadIdx.x >> 5, lane = threadIdx.x & 31;
  LossSums mine = {0., 0., 0.};
  const float wt = row < T && weight ? weight[row] : 1.f;
  bool on = false;
  float l = 0.f;
  if (row < T) {
    const int tg = target[row];
    on = row_on(tg, wt, ignore);
    if (on)
      row_loss(groups, ng, zt, row, tg, wt, V, lp, lse, err, mine, l);
    else if (lane == 0)
      lp[row] = lse[row] = 0.f;
  }
  if (lane == 0) sums[row] = mine;
  __syncthreads();
  // (one warp: FP64 is slow on this GPU, and all 32 would queue for it)
  if (row == 0) {
    const LossSums tot = warp_sums(sums[lane]);
    if (lane == 0) {
      scale = loss_scale(tot, mean, norm);
      write_stats(tot, scale, z_coef, stats);
    }
  }
  __syncthreads();
  if (row < T && lane == 0) write_coefs(row, wt, on, l, scale, z_coef, dlp, dlse);
}

// Tiles of rows that do not count (prompts, padding) are left out of the
// product where that can save more than finding them costs: 3 us, against 100 us
// or more of a product of this many multiplications.
bool skip_tiles(int T, int V, int K) { return T > 256 && double(T) * V * K >= 8e10; }

size_t loss_bytes(int T, int V) {
  size_t g = 0;
  biv_lm_head_logprob_workspace(T, V, &g);
  return (g + 255) / 256 * 256 + kMaxParts * sizeof(LossSums) + ((T + 127) / 128 + size_t(1)) * 4;
}

}  // namespace
}  // namespace biv

using namespace biv;

extern "C" {

biv_status biv_lm_head_loss_workspace(int T, int V, size_t* bytes) {
  BIV_REQUIRE(bytes && T >= 0 && V > 0 && V < (1 << 24), "lm_head_loss_workspace: bad arguments");
  *bytes = loss_bytes(T, V);
  return BIV_OK;
}

biv_status biv_lm_head_loss(const biv_lm_loss_desc* d, biv_stream_t stream) {
  BIV_REQUIRE(d, "lm_head_loss: null descriptor");
  BIV_REQUIRE(d->T >= 0 && d->V > 0 && d->K > 0, "lm_head_loss: bad sizes T=%d V=%d K=%d", d->T, d->V, d->K);
  BIV_REQUIRE(d->stats && (d->T == 0 || (d->h && d->W && d->target && d->lp && d->lse)),
              "lm_head_loss: null pointer");
  BIV_REQUIRE(d->reduce == BIV_LOSS_TOKEN_MEAN || d->reduce == BIV_LOSS_SUM,
              "lm_head_loss: reduce is TOKEN_MEAN or SUM");
  BIV_REQUIRE(d->reduce != BIV_LOSS_SUM || (d->norm > 0.f && d->norm <= 3e38f), "lm_head_loss: norm must be > 0");
  BIV_REQUIRE(d->z_coef >= 0.f && d->z_coef <= 1000.f, "lm_head_loss: z_coef in [0, 1000]");
  if (!d->workspace || d->workspace_bytes < loss_bytes(d->T, d->V))
    return set_error(BIV_ERR_WORKSPACE, "lm_head_loss: workspace of %zu bytes needed", loss_bytes(d->T, d->V));
  BIV_REQUIRE(aligned16(d->workspace), "lm_head_loss: workspace must be 16-byte aligned");
  cudaStream_t s = as_cuda(stream);
  size_t gb = 0;
  biv_lm_head_logprob_workspace(d->T, d->V, &gb);
  gb = (gb + 255) / 256 * 256;
  LossSums* parts = reinterpret_cast<LossSums*>(static_cast<uint8_t*>(d->workspace) + gb);
  int* tiles = reinterpret_cast<int*>(parts + kMaxParts);
  const int mean = d->reduce == BIV_LOSS_TOKEN_MEAN;
  biv_status st;
  int blocks = 0;
  if (d->T > 0) {
    const float2* groups;
    const float* zt;
    int ng;
    const bool skip = skip_tiles(d->T, d->V, d->K);
    if (skip) {
      launch_pdl(row_tiles_kernel, 1, 1024, 0, s, d->target, d->weight, d->T, d->ignore_index, tiles);
      if ((st = check_launch("lm_head_loss tiles")) != BIV_OK) return st;
    }
    st = lm_head_groups("lm_head_loss", d->h, d->ldh, d->W, d->ldw, d->T, d->V, d->K, d->target,
                        BIV_MODE_INVARIANT, skip ? tiles : nullptr, d->workspace, gb, &groups, &zt, &ng, stream);
    if (st != BIV_OK) return st;
    if (d->T <= 32) {
      launch_pdl(few_rows_kernel, 1, 1024, 0, s, groups, ng, zt, d->target, d->weight, d->T, d->V, d->ignore_index,
                 d->z_coef, mean, d->norm, d->lp, d->lse, d->dlp, d->dlse, d->stats, device_error_word());
      return check_launch("lm_head_loss");
    }
    blocks = int(std::min<int64_t>((d->T + kLossRows - 1) / kLossRows, kMaxParts));
    launch_pdl(lse_rows_kernel, blocks, kLossRows * 32, 0, s, groups, ng, zt, d->target, d->weight, d->T,
               d->V, d->ignore_index, d->lp, d->lse, parts, device_error_word());
    if ((st = check_launch("lm_head_loss rows")) != BIV_OK) return st;
  }
  launch_pdl(loss_rows_kernel, std::max(1, std::min((d->T + 255) / 256, 152)), 256, 0, s,
             static_cast<const LossSums*>(parts), blocks, d->target, d->weight,
             static_cast<const float*>(d->lse), d->T, d->ignore_index, d->z_coef, mean, d->norm, d->dlp, d->dlse,
             d->stats);
  return check_launch("lm_head_loss");
}

static biv_status lm_grad_sizes(const char* what, int T, int V, int K, int dh_dtype, int dw_dtype) {
  BIV_REQUIRE(T >= 0 && V > 0 && K > 0 && K % 8 == 0, "%s: T=%d V=%d K=%d, K a multiple of 8", what, T, V, K);
  BIV_REQUIRE(T <= (1 << 20) && V < (1 << 24) && K <= (1 << 16), "%s: size too large", what);
  BIV_REQUIRE((dh_dtype == BIV_BF16 || dh_dtype == BIV_F32) && (dw_dtype == BIV_BF16 || dw_dtype == BIV_F32),
              "%s: gradients are bf16 or f32", what);
  return BIV_OK;
}

biv_status biv_lm_head_backward_workspace(int T, int V, int K, int dh_dtype, int dw_dtype,
                                          size_t* bytes) {
  biv_status st = lm_grad_sizes("lm_head_backward_workspace", T, V, K, dh_dtype, dw_dtype);
  if (st != BIV_OK) return st;
  BIV_REQUIRE(bytes, "lm_head_backward_workspace: null output");
  *bytes = T == 0 ? 0 : layout(T, V, K, dh_dtype == BIV_F32 || dw_dtype == BIV_F32).bytes;
  return BIV_OK;
}

biv_status biv_lm_head_backward(const biv_lm_grad_desc* d, biv_stream_t stream) {
  BIV_REQUIRE(d, "lm_head_backward: null descriptor");
  const int T = d->T, V = d->V, K = d->K;
  biv_status st = lm_grad_sizes("lm_head_backward", T, V, K, d->dh_dtype, d->dw_dtype);
  if (st != BIV_OK) return st;
  BIV_REQUIRE(d->accumulate == 0 || d->accumulate == 1, "lm_head_backward: accumulate is 0 or 1");
  BIV_REQUIRE(!d->dW || d->lddw >= K, "lm_head_backward: dW's rows overlap");
  const int wb = d->dw_dtype == BIV_F32 ? 4 : 2, hb = d->dh_dtype == BIV_F32 ? 4 : 2;
  BIV_REQUIRE((reinterpret_cast<uintptr_t>(d->dW) & (wb - 1)) == 0 &&
                  (reinterpret_cast<uintptr_t>(d->dh) & (hb - 1)) == 0,
              "lm_head_backward: misaligned gradient");
  cudaStream_t s = as_cuda(stream);
  if (T == 0) {
    if (d->dW && !d->accumulate &&
        cudaMemset2DAsync(d->dW, size_t(d->lddw) * wb, 0, size_t(K) * wb, V, s) != cudaSuccess)
      return set_error(BIV_ERR_CUDA, "lm_head_backward: cannot clear dW");
    return BIV_OK;
  }
  BIV_REQUIRE(d->h && d->W && d->target && d->lse && d->dlp, "lm_head_backward: null pointer");
  BIV_REQUIRE(aligned16(d->h) && aligned16(d->W) && d->ldh >= K && d->ldw >= K && d->ldh % 8 == 0 &&
                  d->ldw % 8 == 0,
              "lm_head_backward: h and W need 16-byte aligned rows");
  BIV_REQUIRE(!d->dh || d->lddh >= K, "lm_head_backward: dh's rows overlap");
  const Layout l = layout(T, V, K, d->dh_dtype == BIV_F32 || d->dw_dtype == BIV_F32);
  if (!d->workspace || d->workspace_bytes < l.bytes)
    return set_error(BIV_ERR_WORKSPACE, "lm_head_backward: workspace of %zu bytes needed", l.bytes);
  BIV_REQUIRE((reinterpret_cast<uintptr_t>(d->workspace) & 255) == 0,
              "lm_head_backward: workspace must be 256-byte aligned");
  if (!d->dh && !d->dW) return BIV_OK;
  Args a;
  memset(&a, 0, sizeof(a));
  a.r = rows_of(l, d->workspace);
  Maps m;
  memset(&m, 0, sizeof(m));
  a.dw_tma = d->dW && aligned16(d->dW) && (d->lddw * wb) % 16 == 0;
  a.w2 = K % 64 == 0;
  a.sums = d->dW && T > kSums;
  const int64_t tm = l.cap / kTM, tk = l.ka / kTN, tn = (int64_t(V) + kTN - 1) / kTN + l.chunks;
  BIV_REQUIRE(tm * tn + tk * (tm * l.chunks + tn) < (int64_t(1) << 30), "lm_head_backward: too many tiles");
  const int64_t dzc = int64_t(l.ring) * l.chunk, dzr = int64_t(l.cap) * l.parts;
  if (!map_rows(&m.hk, a.r.h, l.kp, l.cap, l.kp, 128, false) ||
      !map_rows(&m.hn, a.r.h, l.kp, l.cap, l.kp, 64, true) ||
      !map_rows(&m.wk, d->W, K, V, d->ldw, 128, false) ||
      !map_rows(&m.wn, d->W, K, V, d->ldw, 64, K % 64 == 0) ||
      !map_rows(&m.dk, a.r.dz, dzc, dzr, dzc, 128, false) || !map_rows(&m.dn, a.r.dz, dzc, dzr, dzc, 64, true) ||
      !map_rows(&m.ds, a.r.dz, dzc, dzr, dzc, 32, false, l.parts == 2 ? 32 : 64) ||
      (a.dw_tma && !map_rows(&m.ws, d->dW, K, V, d->lddw, 32, false, d->dw_dtype == BIV_F32 ? 32 : 64,
                             d->dw_dtype == BIV_F32)))
    return set_error(BIV_ERR_CUDA, "lm_head_backward: tensor map encoding failed");
  a.V = V; a.K = K; a.kp = l.kp; a.ka = l.ka; a.cap = l.cap;
  a.chunk = l.chunk; a.chunks = l.chunks; a.ahead = l.ahead; a.ring = l.ring; a.slots = l.slots;
  a.parts = l.parts;
  a.parts_h = d->dh_dtype == BIV_F32 ? 2 : 1;
  a.parts_w = d->dw_dtype == BIV_F32 ? 2 : 1;
  a.W = d->W; a.ldw = d->ldw;
  a.dh = d->dh; a.lddh = d->lddh; a.dh_f32 = d->dh_dtype == BIV_F32;
  a.dh_vec = (reinterpret_cast<uintptr_t>(d->dh) & 31) == 0 && (d->lddh * hb) % 32 == 0;
  a.dW = d->dW; a.lddw = d->lddw; a.dw_f32 = d->dw_dtype == BIV_F32;
  a.accumulate = d->accumulate;
  a.err = device_error_word();
  if (T > kRun) {
    launch_pdl(sort_rows_kernel, (T + kRun - 1) / kRun, kRun, 0, s, d->target, d->dlp, d->dlse, T, V, a.r);
    if ((st = check_launch("lm_head_backward order")) != BIV_OK) return st;
  }
  launch_pdl(T > kRun ? gather_kernel<true> : gather_kernel<false>, (l.cap + 7) / 8, 256, 0, s, d->h, d->ldh, d->W, d->ldw, d->target, d->lse, d->dlp, d->dlse, T, V,
             K, l.kp, l.cap, l.chunks, d->dh, d->lddh, a.dh_f32, a.r, a.err);
  if ((st = check_launch("lm_head_backward rows")) != BIV_OK) return st;
  if (a.sums) {
    launch_pdl(target_sums_kernel, dim3(l.cap / 64, (l.kp + 2047) / 2048), 256, 0, s, a.r, l.kp);
    if ((st = check_launch("lm_head_backward targets")) != BIV_OK) return st;
  }
  if ((st = l.parts == 2 ? launch_grad<true>(m, a, s) : launch_grad<false>(m, a, s)) != BIV_OK) return st;
  if (!d->dh || l.slots == 1) return BIV_OK;
  launch_pdl(dh_fold_kernel, dim3(T, (K + 1023) / 1024), 256, 0, s, a.r, d->W, d->ldw, K, l.ka, l.cap,
             l.slots, d->dh, d->lddh, a.dh_f32);
  return check_launch("lm_head_backward fold");
}

}  // extern "C"
