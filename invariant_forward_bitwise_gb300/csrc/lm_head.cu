// Cross entropy of the LM head and its gradient without stored logits.
//
// Forward (biv_lm_head_loss): the GEMM of biv_lm_head_logprob leaves a
// (max, sum exp) pair per row and 128 columns; lse_rows_kernel merges them as
// biv_lm_head_logprob does (the same bits) and loss_rows_kernel forms the
// weighted mean and each row's coefficients for the backward.
//
// Backward (biv_lm_head_backward): with z = h.W^T and p = exp(z - lse),
//   dz = dlp (onehot(target) - p) + dlse p,   dh = dz.W,   dW = dz^T.h.
// The logits are formed again in pieces of the vocabulary: per piece one GEMM
// whose epilogue turns its FP32 accumulators into bf16 dz (scores kernel),
// then both products of that dz (grads kernel), each on tcgen05 with FP32
// accumulators in TMEM.
//  - Rows whose coefficients are 0 (prompts, padding, clipped tokens) have no
//    gradient: the rows that count are gathered first, so that what the others
//    hold is never multiplied, and no time is spent on them.
//  - The term of a row's own target is usually the largest by far.  It stays
//    out of the matrix products and is added in FP32, to dh by the fold and to
//    dW by the epilogue of the tile that holds the target.  The p terms enter
//    the products as bf16, the type of the other operands: an error of at most
//    2^-8 of each of them; for FP32 gradients as two bf16 parts, hi + lo (2^-16).
//  - dh is summed over the vocabulary in chunks of kChunk columns, each
//    accumulated from zero in TMEM in ascending columns, and the chunks added
//    in ascending order in FP32: a row's dh depends on that row, V and K only.
//    dW is one accumulation over the counted rows in ascending order.
#include <algorithm>
#include <cstring>

#include "common.cuh"

namespace biv {
// gemm.cu: the fused head's GEMM.  lse[row * ng + g] = (max, sum exp(z - max)) of
// columns [128 g, 128 g + 128), zt[row] = the logit at target[row] (unset where
// the target is outside [0, V)).
biv_status lm_head_groups(const char* what, const uint16_t* h, int64_t ldh, const uint16_t* W,
                          int64_t ldw, int M, int V, int K, const int32_t* target, int mode,
                          void* ws, size_t ws_bytes, const float2** lse, const float** zt, int* ng,
                          biv_stream_t stream);

namespace {

constexpr int kChunk = 8192;      // vocabulary columns per FP32 partial of dh
constexpr int kTM = 256;          // tile rows: 128 TMEM lanes in each CTA of a pair
constexpr int kTN = 256;          // tile columns: each CTA brings half of B
constexpr int kTK = 128;          // K elements per stage: two 128-byte panels
constexpr int kPanel = 128 * 128; // bytes of a 128-row panel of 64 bf16
constexpr int kOperand = 2 * kPanel;   // a CTA's part of A or B in a stage
constexpr int kStages = 3;
constexpr int kEpi = 8;
constexpr int kThreads = 64 + 32 * kEpi;
constexpr int kSmem = 1024 + kStages * 2 * kOperand + 256;

// Device-side state of one call, at the head of its workspace.
struct Rows {
  int* n;             // [1] rows that count
  int* idx;           // [cap] their row numbers, ascending
  int* target;        // [cap]
  int* head;          // [V] first counted row with that target, or -1
  int* next;          // [cap] next counted row with the same target, or -1
  float* lse;         // [cap]
  float* dlp;         // [cap]
  float* cp;          // [cap] dlse - dlp: the factor of p
  float* dzt;         // [cap] dz at the target
  uint16_t* h;        // [cap][kp] gathered rows, zeros behind them and behind K
  float* acc;         // [slots][cap][ka] chunk partials of dh
  uint16_t* dz;       // [parts][cap][cols]
};

struct Layout {
  int cap, kp, ka;          // rows, gathered row pitch, partial row pitch
  int chunks, per_pass;     // chunks of V, chunks per pass
  int slots;                // 1: the partials are added up as they come
  int cols;                 // dz row pitch
  int parts;                // bf16 parts of dz
  size_t off[12], bytes;
};

constexpr size_t kSlotBytes = size_t(192) << 20;
constexpr size_t kPieceBytes = size_t(96) << 20;

Layout layout(int T, int V, int K, bool want_dh, bool f32) {
  Layout l;
  l.cap = (T + kTM - 1) / kTM * kTM;
  l.kp = (K + kTK - 1) / kTK * kTK;
  l.ka = (K + kTN - 1) / kTN * kTN;
  l.chunks = (V + kChunk - 1) / kChunk;
  l.parts = f32 ? 2 : 1;
  const size_t part = size_t(l.cap) * l.ka * 4;
  l.slots = want_dh && l.chunks > 1 && part * l.chunks <= kSlotBytes ? l.chunks : 1;
  const size_t piece = size_t(l.cap) * kChunk * 2 * l.parts;
  l.per_pass = l.slots > 1 || !want_dh
                   ? int(std::min<size_t>(l.chunks, std::max<size_t>(1, kPieceBytes / piece)))
                   : 1;
  l.cols = int(std::min<int64_t>(int64_t(l.per_pass) * kChunk, (int64_t(V) + kTN - 1) / kTN * kTN));
  const size_t sizes[12] = {16, size_t(l.cap) * 4, size_t(l.cap) * 4, size_t(V) * 4,
                            size_t(l.cap) * 4, size_t(l.cap) * 4, size_t(l.cap) * 4,
                            size_t(l.cap) * 4, size_t(l.cap) * 4, size_t(l.cap) * l.kp * 2,
                            want_dh ? part * l.slots : 0,
                            size_t(l.parts) * l.cap * l.cols * 2};
  l.bytes = 0;
  for (int i = 0; i < 12; ++i) {
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
  r.head = reinterpret_cast<int*>(b + l.off[3]);
  r.next = reinterpret_cast<int*>(b + l.off[4]);
  r.lse = reinterpret_cast<float*>(b + l.off[5]);
  r.dlp = reinterpret_cast<float*>(b + l.off[6]);
  r.cp = reinterpret_cast<float*>(b + l.off[7]);
  r.dzt = reinterpret_cast<float*>(b + l.off[8]);
  r.h = reinterpret_cast<uint16_t*>(b + l.off[9]);
  r.acc = reinterpret_cast<float*>(b + l.off[10]);
  r.dz = reinterpret_cast<uint16_t*>(b + l.off[11]);
  return r;
}

// ------------------------------------------------------------- gathering --
// CTA 0 lists the rows that count; the others set head to -1.
__global__ void __launch_bounds__(1024) pick_rows_kernel(const int32_t* __restrict__ target,
                                                         const float* __restrict__ dlp,
                                                         const float* __restrict__ dlse, int T,
                                                         int V, Rows r, int* err) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x > 0) {
    for (int v = (blockIdx.x - 1) * 1024 + threadIdx.x; v < V; v += (gridDim.x - 1) * 1024)
      r.head[v] = -1;
    return;
  }
  __shared__ int warp_n[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int base = 0;
  for (int t0 = 0; t0 < T; t0 += 1024) {
    const int t = t0 + threadIdx.x;
    bool on = false;
    int tg = 0;
    if (t < T) {
      tg = target[t];
      // (a NaN is not 0: its row counts)
      on = !(dlp[t] == 0.f) || (dlse && !(dlse[t] == 0.f));
      if (on && (tg < 0 || tg >= V)) {
        raise_error(err, kErrBadIndex);
        on = false;
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, on);
    __syncthreads();
    if (lane == 0) warp_n[warp] = __popc(m);
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warp_n[w];
      all += warp_n[w];
    }
    if (on) {
      const int i = before + __popc(m & ((1u << lane) - 1));
      r.idx[i] = t;
      r.target[i] = tg;
    }
    base += all;
  }
  if (threadIdx.x == 0) *r.n = base;
}

__device__ __forceinline__ void zero_row(void* base, int64_t ld, int f32, int64_t row, int K, int lane) {
  if (f32) {
    float* d = static_cast<float*>(base) + row * ld;
    for (int c = lane; c < K; c += 32) d[c] = 0.f;
  } else {
    uint16_t* d = static_cast<uint16_t*>(base) + row * ld;
    for (int c = lane; c < K; c += 32) d[c] = 0;
  }
}

// A warp per row of [0, cap): counted row i is gathered with its scalars and
// its place in the chain of rows with the same target; up to the next multiple
// of 128 behind the last one zeros are written.  The warp also clears row i of
// dh where that row does not count.
__global__ void __launch_bounds__(256) gather_kernel(
    const uint16_t* __restrict__ h, int64_t ldh, const float* __restrict__ lse,
    const float* __restrict__ dlp, const float* __restrict__ dlse, int T, int K, int kp, int cap,
    void* dh, int64_t lddh, int dh_f32, Rows r) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= cap) return;
  const int n = *r.n;
  if (dh && i < T) {
    const float c = dlp[i], z = dlse ? dlse[i] : 0.f;
    bool on = !(c == 0.f) || !(z == 0.f);
    if (on) {   // a row with a bad target is not in the list
      int lo = 0, hi = n;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (r.idx[mid] < i) lo = mid + 1; else hi = mid;
      }
      on = lo < n && r.idx[lo] == i;
    }
    if (!on) zero_row(dh, lddh, dh_f32, i, K, lane);
  }
  if (i >= (n + kTM - 1) / kTM * kTM) return;
  uint4* dst = reinterpret_cast<uint4*>(r.h + int64_t(i) * kp);
  if (i >= n) {
    for (int c = lane; c < kp / 8; c += 32) dst[c] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int t = r.idx[i], tg = r.target[i];
  const uint4* src = reinterpret_cast<const uint4*>(h + int64_t(t) * ldh);
  for (int c = lane; c < kp / 8; c += 32)
    dst[c] = c < K / 8 ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
  // the chain of rows with this target
  int nx = -1;
  for (int j0 = i + 1; j0 < n && nx < 0; j0 += 32) {
    const int j = j0 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, j < n && r.target[j] == tg);
    if (m) nx = j0 + __ffs(m) - 1;
  }
  bool first = true;
  for (int j0 = 0; j0 < i && first; j0 += 32) {
    const int j = j0 + lane;
    first = __ballot_sync(0xffffffffu, j < i && r.target[j] == tg) == 0;
  }
  if (lane == 0) {
    r.next[i] = nx;
    if (first) r.head[tg] = i;
    const float c = dlp[t];
    r.lse[i] = lse[t];
    r.dlp[i] = c;
    r.cp[i] = (dlse ? dlse[t] : 0.f) - c;
  }
}

// ----------------------------------------------------------------- GEMMs --
struct Maps {
  // boxes of {64 columns, 128 rows, 2 panels} ({64, 128} of W when K % 64)
  CUtensorMap h;     // gathered h: K-major A of the scores, MN-major B of dW
  CUtensorMap w;     // W: K-major B of the scores, MN-major B of dh
  CUtensorMap dz;    // dz: K-major A of dh, MN-major A of dW
};

struct Args {
  Rows r;
  int V, K, kp, ka, cap, cols;
  int w3;                  // W's maps bring several panels at once (K % 64 == 0)
  int v0, vn;              // this pass: columns [v0, v0 + vn) of V
  int c0, nc;              // its chunks
  int slots;
  int parts, parts_h, parts_w;
  void* dW; int64_t lddw; int dw_f32, dw_vec, accumulate;
  int want_dh;
  int* err;
};

enum { kScores = 0, kDh = 1, kDw = 2 };
struct Item {
  int type, m0, n0;        // tile origin
  int k0;                  // first K index (dh: column of the piece)
  int nk;                  // stages of one part
  int parts;
  int slot;
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

template <int PHASE>
__device__ __forceinline__ int item_count(const Args& a, int n) {
  const int tm = cdiv(n, kTM);
  if (PHASE == 0) return tm * cdiv(a.vn, kTN);
  const int tk = cdiv(a.K, kTN);
  return (a.want_dh ? tm * tk * a.nc : 0) + (a.dW ? cdiv(a.vn, kTM) * tk : 0);
}

// dh's items come first: they are the long ones
template <int PHASE>
__device__ __forceinline__ Item item_at(const Args& a, int n, int i) {
  const int tm = cdiv(n, kTM);
  Item it;
  if (PHASE == 0) {
    it.type = kScores;
    it.m0 = (i % tm) * kTM;
    it.n0 = (i / tm) * kTN;
    it.k0 = 0;
    it.nk = a.kp / kTK;
    it.parts = 1;
    it.slot = 0;
    return it;
  }
  const int tk = cdiv(a.K, kTN);
  const int ndh = a.want_dh ? tm * tk * a.nc : 0;
  if (i < ndh) {
    const int c = i / (tm * tk), j = i % (tm * tk);
    it.type = kDh;
    it.m0 = (j / tk) * kTM;
    it.n0 = (j % tk) * kTN;
    it.k0 = c * kChunk;
    it.nk = cdiv(min(kChunk, a.vn - it.k0), kTK);
    it.parts = a.parts_h;
    it.slot = a.slots > 1 ? a.c0 + c : 0;
  } else {
    const int j = i - ndh;
    it.type = kDw;
    it.m0 = (j / tk) * kTM;
    it.n0 = (j % tk) * kTN;
    it.k0 = 0;
    it.nk = cdiv(n, kTK);
    it.parts = a.parts_w;
    it.slot = 0;
  }
  return it;
}

// PHASE 0: the scores of a piece and their dz; PHASE 1: dh and dW of it.
// Persistent pairs of CTAs (clusters of two), 320 threads each: warp 0 = TMA
// producer, warp 1 = TMEM owner and, in the pair's first CTA, MMA issuer, warps
// 2..9 = epilogue (lane quarter = warp % 4, column half = (warp - 2) / 4).  A
// tile is 256 x 256: each CTA loads its 128 rows of A and of B, the first CTA
// issues cta_group::2 MMAs over both, and each CTA's TMEM gets its 128 rows.
// full barriers live in the first CTA and count both CTAs' bytes; empty and
// tfull are signalled in both by multicast commits; both epilogues arrive on
// the first CTA's tempty.
template <int PHASE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    lm_grad_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  extern __shared__ uint8_t smem_raw[];
  // (the offset is the same in both CTAs of a pair)
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kOperand;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sB + kStages * kOperand);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kStages);
  const uint32_t tfull0 = smem_u32(bars + 2 * kStages), tempty0 = smem_u32(bars + 2 * kStages + 2);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_rank()), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(tfull0 + 8 * j, 1);
      mbar_init(tempty0 + 8 * j, 2 * kEpi);
    }
    fence_barrier_init();
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
  const int n = *a.r.n;
  const int items = item_count<PHASE>(a, n);

  int issued = 0;
  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      for (int i = pair; i < items && ok; i += pairs) {
        const Item it = item_at<PHASE>(a, n, i);
        for (int kb = 0; kb < it.nk * it.parts; ++kb) {
          const int s = issued % kStages;
          if (issued >= kStages && !mbar_wait(empty0 + 8 * s, ((issued / kStages) - 1) & 1, a.err)) {
            ok = false;
            break;
          }
          const uint32_t bar = cluster_addr(full0 + 8 * s, 0);
          const uint32_t da = smem_u32(sA + s * kOperand), db = smem_u32(sB + s * kOperand);
          if (rank == 0) mbar_expect_tx(full0 + 8 * s, 4 * kOperand);
          const int part = kb / it.nk, k = kb % it.nk;
          const int m = it.m0 + rank * 128, nn = it.n0 + rank * 128;
          if (PHASE == 0) {
            tma2_load_3d(da, &maps.h, bar, 0, m, 2 * k);
            if (a.w3) {
              tma2_load_3d(db, &maps.w, bar, 0, a.v0 + nn, 2 * k);
            } else {
              for (int q = 0; q < 2; ++q)
                tma2_load_2d(db + q * kPanel, &maps.w, bar, (2 * k + q) * 64, a.v0 + nn);
            }
          } else if (it.type == kDh) {
            const int v = it.k0 + k * kTK;
            tma2_load_3d(da, &maps.dz, bar, 0, part * a.cap + m, v / 64);
            if (a.w3) {
              tma2_load_3d(db, &maps.w, bar, 0, a.v0 + v, nn / 64);
            } else {
              for (int q = 0; q < 2; ++q)
                tma2_load_2d(db + q * kPanel, &maps.w, bar, nn + q * 64, a.v0 + v);
            }
          } else {
            tma2_load_3d(da, &maps.dz, bar, 0, part * a.cap + k * kTK, m / 64);
            tma2_load_3d(db, &maps.h, bar, 0, k * kTK, nn / 64);
          }
          ++issued;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int st = 0, j = 0;
      bool ok = true;
      for (int i = pair; i < items && ok; i += pairs) {
        const Item it = item_at<PHASE>(a, n, i);
        const int nk = it.nk * it.parts;
        if (nk == 0) continue;
        const int b = j & 1;
        if (j >= 2 && !mbar_wait(tempty0 + 8 * b, ((j >> 1) - 1) & 1, a.err)) break;
        tc_fence_after();
        const uint32_t dt = tmem + b * kTN;
        const uint32_t idesc = idesc_mma(1u, kTM, kTN) | (it.type == kDw ? 1u << 15 : 0u) |
                               (it.type != kScores ? 1u << 16 : 0u);
        for (int kb = 0; kb < nk; ++kb, ++st) {
          const int s = st % kStages;
          if (!mbar_wait(full0 + 8 * s, (st / kStages) & 1, a.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * kOperand), b0 = smem_u32(sB + s * kOperand);
#pragma unroll
          for (int kk = 0; kk < kTK / 16; ++kk) {
            // K-major panels hold 64 K elements of a row; MN-major panels 64
            // rows or columns of the output, one K index per 128 bytes
            const uint32_t ko = (kk >> 2) * kPanel + (kk & 3) * 32;
            const uint64_t ad = PHASE == 1 && it.type == kDw
                                    ? sdesc_mn_sw128(a0 + kk * 2048, kPanel, 1024)
                                    : sdesc_k_sw128(a0 + ko);
            const uint64_t bd = PHASE == 1 ? sdesc_mn_sw128(b0 + kk * 2048, kPanel, 1024)
                                           : sdesc_k_sw128(b0 + ko);
            umma2_f16(dt, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
          }
          umma2_commit(empty0 + 8 * s);
        }
        if (ok) umma2_commit(tfull0 + 8 * b);
        ++j;
      }
    }
  } else {
    const int q = warp & 3, col0 = ((warp - 2) >> 2) * (kTN / 2);
    int j = 0;
    bool ok = true;
    for (int i = pair; i < items && ok; i += pairs) {
      const Item it = item_at<PHASE>(a, n, i);
      const int nk = it.nk * it.parts;
      const int b = j & 1;
      if (nk > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(tfull0 + 8 * b, (j >> 1) & 1, a.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      const uint32_t ta = tmem + b * kTN + col0 + (uint32_t(q * 32) << 16);
      const int row = it.m0 + rank * 128 + q * 32 + lane;
      if (PHASE == 0) {
        const bool live = row < n;
        const float lse = live ? a.r.lse[row] : 0.f, cp = live ? a.r.cp[row] : 0.f;
        const int tc = live ? a.r.target[row] - a.v0 : -1;   // the target's column of the piece
        uint16_t* dst = a.r.dz + int64_t(row) * a.cols + it.n0 + col0;
        for (int g = 0; g < kTN / 64; ++g) {
          uint32_t v[32];
          tmem_ld32(ta + g * 32, v);
          tmem_ld_wait();
          const int c = it.n0 + col0 + g * 32;               // column of the piece
          float d[32];
#pragma unroll
          for (int x = 0; x < 32; ++x)
            d[x] = live && c + x < a.vn ? cp * expf(__uint_as_float(v[x]) - lse) : 0.f;
          if (tc >= c && tc < c + 32) {
            float full = a.r.dlp[row];
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (c + x == tc) {
                full += d[x];
                d[x] = 0.f;
              }
            a.r.dzt[row] = full;
          }
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) w[x] = pack_bf2(d[2 * x], d[2 * x + 1]);
          st_global_v8(dst + g * 32, w);
          st_global_v8(dst + g * 32 + 16, w + 8);
          if (a.parts == 2) {
#pragma unroll
            for (int x = 0; x < 16; ++x)
              w[x] = pack_bf2(d[2 * x] - bf2f(f2bf(d[2 * x])), d[2 * x + 1] - bf2f(f2bf(d[2 * x + 1])));
            uint16_t* lo = dst + int64_t(a.cap) * a.cols + g * 32;
            st_global_v8(lo, w);
            st_global_v8(lo + 16, w + 8);
          }
        }
      } else if (it.type == kDh) {
        float* dst = a.r.acc + (int64_t(it.slot) * a.cap + row) * a.ka + it.n0 + col0;
        const bool add = a.slots == 1 && a.c0 > 0;
        for (int g = 0; g < kTN / 64; ++g) {
          uint32_t v[32];
          tmem_ld32(ta + g * 32, v);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            if (add) {
              const float4 o0 = *reinterpret_cast<const float4*>(dst + g * 32 + x);
              const float4 o1 = *reinterpret_cast<const float4*>(dst + g * 32 + x + 4);
              const float o[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
#pragma unroll
              for (int y = 0; y < 8; ++y) v[x + y] = __float_as_uint(o[y] + __uint_as_float(v[x + y]));
            }
            st_global_v8(dst + g * 32 + x, v + x);
          }
        }
      } else {
        const int vr = a.v0 + row;                           // row of dW
        const bool live = row < a.vn;
        const int first = live && nk > 0 ? a.r.head[vr] : -1;
        for (int g = 0; g < kTN / 64; ++g) {
          uint32_t v[32];
          if (nk > 0) {
            tmem_ld32(ta + g * 32, v);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = 0u;
          }
          const int c = it.n0 + col0 + g * 32;
          if (!live || c >= a.K) continue;
          // the rows whose target this is
          for (int t = first; t >= 0; t = a.r.next[t]) {
            const float dzt = a.r.dzt[t];
            const uint4* hr = reinterpret_cast<const uint4*>(a.r.h + int64_t(t) * a.kp + c);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint4 u = hr[x];
              const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                v[8 * x + 2 * y] = __float_as_uint(
                    fmaf(dzt, __uint_as_float(uw[y] << 16), __uint_as_float(v[8 * x + 2 * y])));
                v[8 * x + 2 * y + 1] =
                    __float_as_uint(fmaf(dzt, __uint_as_float(uw[y] & 0xFFFF0000u),
                                         __uint_as_float(v[8 * x + 2 * y + 1])));
              }
            }
          }
          const bool vec = a.dw_vec && c + 32 <= a.K;
          if (a.dw_f32) {
            float* dst = static_cast<float*>(a.dW) + int64_t(vr) * a.lddw + c;
            if (vec) {
              if (a.accumulate) {
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  v[x] = __float_as_uint(dst[x] + __uint_as_float(v[x]));
              }
#pragma unroll
              for (int x = 0; x < 32; x += 8) st_global_v8(dst + x, v + x);
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (c + x < a.K)
                  dst[x] = (a.accumulate ? dst[x] : 0.f) + __uint_as_float(v[x]);
            }
          } else {
            uint16_t* dst = static_cast<uint16_t*>(a.dW) + int64_t(vr) * a.lddw + c;
            if (a.accumulate) {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (c + x < a.K) v[x] = __float_as_uint(bf2f(dst[x]) + __uint_as_float(v[x]));
            }
            if (vec) {
              uint32_t w[16];
#pragma unroll
              for (int x = 0; x < 16; ++x)
                w[x] = pack_bf2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1]));
              st_global_v8(dst, w);
              st_global_v8(dst + 16, w + 8);
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (c + x < a.K) dst[x] = f2bf(__uint_as_float(v[x]));
            }
          }
        }
      }
      if (nk > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(tempty0 + 8 * b, 0));
        ++j;
      }
    }
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

// dh of the counted rows: the chunk partials in ascending order, then the
// target's term.  One CTA per row.
__global__ void __launch_bounds__(256) dh_fold_kernel(Rows r, const uint16_t* __restrict__ W,
                                                      int64_t ldw, int K, int ka, int cap,
                                                      int slots, void* dh, int64_t lddh, int f32) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  if (i >= *r.n) return;
  const int64_t t = r.idx[i];
  const float dzt = r.dzt[i];
  const uint16_t* wr = W + int64_t(r.target[i]) * ldw;
  for (int c = threadIdx.x * 4; c < K; c += 1024) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < slots; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(r.acc + (int64_t(k) * cap + i) * ka + c);
      if (k == 0) {
        s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
      } else {
        s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
      }
    }
    for (int x = 0; x < 4 && c + x < K; ++x) {
      const float o = fmaf(dzt, bf2f(wr[c + x]), s[x]);
      if (f32)
        static_cast<float*>(dh)[t * lddh + c + x] = o;
      else
        static_cast<uint16_t*>(dh)[t * lddh + c + x] = f2bf(o);
    }
  }
}

// bf16 rows in boxes of 128, as {64, rows, K / 64} panels (two per box) or as plain rows
bool map_rows(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int64_t ld, bool panels) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint32_t es[3] = {1, 1, 1}, box[3] = {64, 128, 2};
  const cuuint64_t panel_dims[3] = {64, cuuint64_t(rows), cuuint64_t(K / 64)};
  const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
  const cuuint64_t strides[2] = {cuuint64_t(ld * 2), 128};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, panels ? 3 : 2, const_cast<void*>(base),
            panels ? panel_dims : dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int PHASE>
biv_status launch_grad(const Maps& maps, const Args& a, int64_t most_items, cudaStream_t s) {
  static bool set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (cudaFuncSetAttribute(lm_grad_kernel<PHASE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem) != cudaSuccess)
      return set_error(BIV_ERR_CUDA, "lm_head_backward: cannot set shared memory size");
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  const int sms = sm_count() > 0 ? sm_count() : 148;
  const int pairs = int(std::max<int64_t>(1, std::min<int64_t>(most_items, sms / 2)));
  launch_pdl(lm_grad_kernel<PHASE>, 2 * pairs, kThreads, kSmem, s, maps, a);
  return check_launch("lm_head_backward");
}

// --------------------------------------------------------------- forward --
constexpr int kLossRows = 8;      // rows per CTA, a warp each
constexpr int kMaxParts = 1024;   // blocks whose sums the last kernel adds up

struct LossSums { double w, nll, sq; };

// lp and lse as biv_lm_head_logprob merges the groups (lane l takes groups l,
// l + 32, ... in order, then a xor tree); sums of the counted rows of each CTA.
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
    if (tg == ignore || wt == 0.f) {
      if (lane == 0) lp[row] = lse[row] = 0.f;
      continue;
    }
    const float2* g = groups + int64_t(row) * ng;
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
      const float l = mx + logf(s);
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
  __shared__ double tot[3];
  if (threadIdx.x < 32) {
    double w = 0., nll = 0., sq = 0.;
    for (int i = threadIdx.x; i < nparts; i += 32) {
      w += parts[i].w;
      nll += parts[i].nll;
      sq += parts[i].sq;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      w += __shfl_xor_sync(0xffffffffu, w, o);
      nll += __shfl_xor_sync(0xffffffffu, nll, o);
      sq += __shfl_xor_sync(0xffffffffu, sq, o);
    }
    if (threadIdx.x == 0) {
      tot[0] = w;
      tot[1] = nll;
      tot[2] = sq;
    }
  }
  __syncthreads();
  const double over = mean ? tot[0] : double(norm);
  const double inv = over != 0. ? 1. / over : 0.;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    stats[0] = float((tot[1] + double(z_coef) * tot[2]) * inv);
    stats[1] = float(tot[1] * inv);
    stats[2] = float(tot[2] * inv);
    stats[3] = float(tot[0]);
  }
  for (int t = blockIdx.x * 256 + threadIdx.x; t < T; t += gridDim.x * 256) {
    const float wt = weight ? weight[t] : 1.f;
    const float c = target[t] == ignore || wt == 0.f ? 0.f : float(wt * inv);
    if (dlp) dlp[t] = -c;
    if (dlse) dlse[t] = c == 0.f ? 0.f : float(2. * z_coef * c * lse[t]);
  }
}

size_t loss_bytes(int T, int V) {
  size_t g = 0;
  biv_lm_head_logprob_workspace(T, V, &g);
  return (g + 255) / 256 * 256 + kMaxParts * sizeof(LossSums);
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
  int blocks = 0;
  if (d->T > 0) {
    const float2* groups;
    const float* zt;
    int ng;
    biv_status st = lm_head_groups("lm_head_loss", d->h, d->ldh, d->W, d->ldw, d->T, d->V, d->K,
                                   d->target, BIV_MODE_INVARIANT, d->workspace, gb, &groups, &zt, &ng,
                                   stream);
    if (st != BIV_OK) return st;
    blocks = int(std::min<int64_t>((d->T + kLossRows - 1) / kLossRows, kMaxParts));
    launch_pdl(lse_rows_kernel, blocks, kLossRows * 32, 0, s, groups, ng, zt, d->target, d->weight, d->T,
               d->V, d->ignore_index, d->lp, d->lse, parts, device_error_word());
    st = check_launch("lm_head_loss rows");
    if (st != BIV_OK) return st;
  }
  launch_pdl(loss_rows_kernel, std::max(1, std::min((d->T + 255) / 256, 152)), 256, 0, s,
             static_cast<const LossSums*>(parts), blocks, d->target, d->weight,
             static_cast<const float*>(d->lse), d->T, d->ignore_index, d->z_coef,
             int(d->reduce == BIV_LOSS_TOKEN_MEAN), d->norm, d->dlp, d->dlse, d->stats);
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
  *bytes = T == 0 ? 0 : layout(T, V, K, true, dh_dtype == BIV_F32 || dw_dtype == BIV_F32).bytes;
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
  const Layout l = layout(T, V, K, true, d->dh_dtype == BIV_F32 || d->dw_dtype == BIV_F32);
  if (!d->workspace || d->workspace_bytes < l.bytes)
    return set_error(BIV_ERR_WORKSPACE, "lm_head_backward: workspace of %zu bytes needed", l.bytes);
  BIV_REQUIRE((reinterpret_cast<uintptr_t>(d->workspace) & 255) == 0,
              "lm_head_backward: workspace must be 256-byte aligned");
  if (!d->dh && !d->dW) return BIV_OK;
  Args a;
  memset(&a, 0, sizeof(a));
  a.r = rows_of(l, d->workspace);
  Maps m;
  a.w3 = K % 64 == 0;
  if (!map_rows(&m.h, a.r.h, l.kp, l.cap, l.kp, true) ||
      !map_rows(&m.w, d->W, K, V, d->ldw, a.w3 != 0) ||
      !map_rows(&m.dz, a.r.dz, l.cols, int64_t(l.cap) * l.parts, l.cols, true))
    return set_error(BIV_ERR_CUDA, "lm_head_backward: tensor map encoding failed");
  a.V = V; a.K = K; a.kp = l.kp; a.ka = l.ka; a.cap = l.cap; a.cols = l.cols;
  a.slots = l.slots;
  a.parts = l.parts;
  a.parts_h = d->dh_dtype == BIV_F32 ? 2 : 1;
  a.parts_w = d->dw_dtype == BIV_F32 ? 2 : 1;
  a.dW = d->dW; a.lddw = d->lddw; a.dw_f32 = d->dw_dtype == BIV_F32;
  a.dw_vec = (reinterpret_cast<uintptr_t>(d->dW) & 31) == 0 && (d->lddw * wb) % 32 == 0;
  a.accumulate = d->accumulate;
  a.want_dh = d->dh != nullptr;
  a.err = device_error_word();
  launch_pdl(pick_rows_kernel, 1 + std::min((V + 1023) / 1024, 128), 1024, 0, s, d->target, d->dlp, d->dlse,
             T, V, a.r, a.err);
  if ((st = check_launch("lm_head_backward rows")) != BIV_OK) return st;
  launch_pdl(gather_kernel, (l.cap + 7) / 8, 256, 0, s, d->h, d->ldh, d->lse, d->dlp, d->dlse, T, K, l.kp,
             l.cap, d->dh, d->lddh, int(d->dh_dtype == BIV_F32), a.r);
  if ((st = check_launch("lm_head_backward gather")) != BIV_OK) return st;
  const int64_t tm = l.cap / kTM, tk = (K + kTN - 1) / kTN;
  for (a.c0 = 0; a.c0 < l.chunks; a.c0 += l.per_pass) {
    a.nc = std::min(l.per_pass, l.chunks - a.c0);
    a.v0 = a.c0 * kChunk;
    a.vn = std::min(V - a.v0, a.nc * kChunk);
    if ((st = launch_grad<0>(m, a, tm * ((a.vn + kTN - 1) / kTN), s)) != BIV_OK) return st;
    const int64_t items = (a.want_dh ? tm * tk * a.nc : 0) + (a.dW ? tk * ((a.vn + kTM - 1) / kTM) : 0);
    if ((st = launch_grad<1>(m, a, items, s)) != BIV_OK) return st;
  }
  if (!d->dh) return BIV_OK;
  launch_pdl(dh_fold_kernel, T, 256, 0, s, a.r, d->W, d->ldw, K, l.ka, l.cap, l.slots, d->dh,
              d->lddh, int(d->dh_dtype == BIV_F32));
  return check_launch("lm_head_backward fold");
}

}  // extern "C"
