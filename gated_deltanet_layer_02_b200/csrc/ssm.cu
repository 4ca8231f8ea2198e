// ssm.cu -- selective state space layer: entry points, the single-token step and the fp32 prompts.
// Causal depthwise conv (width 4, bias) + SiLU, then the recurrence
// S_t = exp(-exp(a_log) delta) S_{t-1} + delta x_t B_t^T, y_t = S_t C_t + D x_t with 64 rows of a
// head's state [P, N] in the registers of a CTA, and the gate silu(z) (formulas in gdn.h).  Prompts
// with bf16 activations run on the tensor cores (ssm_tc.cu).
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "args.cuh"
#include "common.cuh"
#include "ssm.cuh"
#include "tc.cuh"

namespace gdn {

constexpr int kScanThreads = 128;
constexpr int kScanRows = 64;   // rows of the state per CTA (16 per warp, 8 lanes per row)
constexpr int kConvRun = 4;    // tokens per thread of the packed conv

// The sequence that holds token t or, where none does, the first token behind it, before t1, that
// one holds; t is moved there.  For a whole block; -1: none.  `n`: the sequence that ended at t (-1:
// not known); mostly the next one holds t, else in a table without bad entries a binary search finds
// it.  Where that finds none (rows behind the last sequence; entries out of order) the block's threads
// look at every sequence: a bad entry costs no other sequence its rows.  (4096 sequences of 8192
// tokens: 176 us for the conv; 255 with as many rows behind them, 239 with the search alone.)
__device__ __forceinline__ int block_seq_of_token(const SsmArgs& a, int n, int& t, int t1, int& s,
                                                  int& end) {
  const auto holds = [&](int m) {
    s = __ldg(a.cu + m), end = __ldg(a.cu + m + 1);
    return s >= 0 && s <= t && t < end && end <= a.T;
  };
  if (n >= 0 && n + 1 < a.N && holds(n + 1)) return n + 1;
  n = seq_of_token(a.cu, a.N, t);
  if (holds(n)) return n;
  __shared__ unsigned long long first;  // (start, sequence) with the least start, from t on
  constexpr unsigned long long kNone = ~0ull;
  unsigned long long mine = kNone;
#pragma unroll 4
  for (int m = threadIdx.x; m < a.N; m += 128) {
    const int ms = __ldg(a.cu + m), me = __ldg(a.cu + m + 1);
    if (ms >= 0 && ms < t1 && t < me && ms < me && me <= a.T)
      mine = min(mine, (unsigned long long)max(ms, t) << 32 | (unsigned)m);
  }
  if (!__syncthreads_or(mine != kNone)) return -1;
  if (threadIdx.x == 0) first = kNone;
  __syncthreads();
  if (mine != kNone) atomicMin(&first, mine);
  __syncthreads();
  n = (int)(unsigned)first;
  t = (int)(first >> 32);
  s = __ldg(a.cu + n), end = __ldg(a.cu + n + 1);
  return n;
}

// Packed prompts: a thread owns 8 channels and a run of kConvRun tokens, the three rows before
// the current one in registers.
__global__ void __launch_bounds__(128, 5) ssm_conv_kernel(SsmArgs a) {
  const int c = (blockIdx.y * 128 + threadIdx.x) * 8, t0 = blockIdx.x * kConvRun;
  const bool live = c < a.Cc;
  float w[4][8], b[8];
  if (live) load_taps<float>(a, c, w, b);
  const float* x = static_cast<const float*>(a.x) + c;
  const float* c0 = static_cast<const float*>(a.conv0);
  float h[3][8];
  int n = -1, s = 0, end = 0;
  const int t1 = min(a.T, t0 + kConvRun);
  for (int t = t0; t < t1; ++t) {
    const bool fresh = t >= end;  // the history registers do not hold the rows before t
    if (fresh) n = block_seq_of_token(a, n, t, t1, s, end);
    if (n < 0) break;
    if (!live) continue;
    if (fresh) {
      const int row = state_row(a.slot, n, a.num_slots);
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int r = t - 3 + j;
        load8_or_zero(r >= s ? x + (size_t)r * a.Cc
                             : (c0 && row >= 0 ? c0 + ((size_t)row * 3 + 3 + r - s) * a.Cc + c
                                               : nullptr),
                      h[j]);
      }
    }
    float v[8], out[8];
    load8(x + (size_t)t * a.Cc, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      out[e] = silu_f(fmaf(w[3][e], v[e],
                           fmaf(w[2][e], h[2][e], fmaf(w[1][e], h[1][e], fmaf(w[0][e], h[0][e], b[e])))));
      h[0][e] = h[1][e];
      h[1][e] = h[2][e];
      h[2][e] = v[e];
    }
    store8(a.u + (size_t)t * a.Cc + c, out);
  }
}

// Four consecutive elements of an activation row (8 or 16 bytes).
__device__ __forceinline__ void load_t4(const float* p, float (&v)[4]) {
  const float4 r = *reinterpret_cast<const float4*>(p);
  v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
}
__device__ __forceinline__ void load_t4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
  const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
  v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
}
__device__ __forceinline__ void store_t4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_t4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// State rows in registers: lane `sub` of a row's eight lanes holds columns 4 sub + 32 m + e
// (m < NS / 32).  A quad is four rows, one per group of eight lanes.
//
// Raw: four elements as they are stored, so that loads stay in flight in as few registers as they
// have bytes.
template <typename TS>
struct Raw;
template <>
struct Raw<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ float4 get() const { return v; }
  static __device__ __forceinline__ void store(float* p, float4 r) {
    __stcs(reinterpret_cast<float4*>(p), r);
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    v = __ldcs(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ float4 get() const {
    const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
    const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float4 r) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(r.x, r.y), pack_bf16x2(r.z, r.w)));
  }
};

// One token of Q quads: the rows take alpha S + dx B^T; o: this lane's share of S C of its row of each
// quad (see ssm_rows_sum).  B, C: the lane's first column.
template <int Q, int M>
__device__ __forceinline__ void ssm_rows_step(float4 (&f)[Q][M], const float* B, const float* C,
                                              const float (&dx)[Q], float alpha, float (&o)[Q]) {
  float p[Q][2] = {};  // two sums: half as long a chain
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const float4 b = *reinterpret_cast<const float4*>(B + 32 * m);
    const float4 c = *reinterpret_cast<const float4*>(C + 32 * m);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float4& r = f[q][m];
      r.x = fmaf(alpha, r.x, dx[q] * b.x);
      r.y = fmaf(alpha, r.y, dx[q] * b.y);
      r.z = fmaf(alpha, r.z, dx[q] * b.z);
      r.w = fmaf(alpha, r.w, dx[q] * b.w);
      p[q][0] = fmaf(r.x, c.x, fmaf(r.y, c.y, p[q][0]));
      p[q][1] = fmaf(r.z, c.z, fmaf(r.w, c.w, p[q][1]));
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) o[q] = p[q][0] + p[q][1];
}
// Sums over the eight lanes of a row, in all of them.
template <int Q>
__device__ __forceinline__ void ssm_rows_sum(float (&o)[Q]) {
#pragma unroll
  for (int off = 4; off > 0; off >>= 1)
#pragma unroll
    for (int q = 0; q < Q; ++q) o[q] += __shfl_xor_sync(0xffffffffu, o[q], off);
}

// ------------------------------------------------------------------------- packed prompts, fp32
// Tokens of a sequence come kScanBlock at a time to shared memory (B, C, the CTA's channels of x and
// z, step and decay), the next ones in flight while these are worked through; y takes the place of
// x and leaves a block at a time.  A CTA has 16 Q rows of a head's state, 4 Q per warp.  A sequence is
// a chain of tokens, so latency bounds it: a warp takes 8 tokens (2 with Q = 4) at a time, whose sums
// over lanes overlap (one sequence of 1021 tokens: 0.29 us per token one at a time, 0.22 so), and a
// block is 32 tokens where few CTAs leave room for it (three sequences: 99 us with 16, 91 with 32).
template <int NS, int Q>
struct ScanTokens {
  static constexpr int kScanBlock = Q == 1 ? 32 : 16;
  float B[kScanBlock][NS], C[kScanBlock][NS], x[kScanBlock][16 * Q], z[kScanBlock][16 * Q];
  float2 gate[kScanBlock];  // step, decay
};

template <int NS, int Q>
__global__ void __launch_bounds__(kScanThreads, 4) ssm_scan_kernel(SsmArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  using Tokens = ScanTokens<NS, Q>;
  constexpr int kRows = 16 * Q, M = NS / 32, kScanBlock = Tokens::kScanBlock;
  Tokens* buf = reinterpret_cast<Tokens*>(smem);  // [2]
  const int blocks = a.P / kRows;
  const int pb = blockIdx.x % blocks, h = (blockIdx.x / blocks) % a.H;
  const int n = blockIdx.x / (blocks * a.H);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = lane >> 3, sub = lane & 7;
  const int row = state_row(a.slot, n, a.num_slots);
  if (row < 0 && tid == 0) report_status(a.status, GDN_ERR_INVALID_ARG);
  int s, end;
  seq_range(a, n, s, end);
  const int r0 = warp * 4 * Q + grp, p0 = pb * kRows + r0;  // this lane group's rows: p0 + 4 q
  const size_t sbase = (((size_t)(row < 0 ? 0 : row) * a.H + h) * a.P + p0) * NS + 4 * sub;
  float4 f[Q][M];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int m = 0; m < M; ++m)
      f[q][m] = a.S0 && row >= 0
                    ? __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(a.S0) + sbase +
                                                             (size_t)(4 * q) * NS + 32 * m))
                    : make_float4(0.f, 0.f, 0.f, 0.f);
  const float rate = -ssm_rate(a.a_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const float D = a.D ? a.D[h] : 0.f;
  const int cB = a.H * a.P + (h / (a.H / a.G)) * NS, cC = cB + a.G * NS;
  const int cx = h * a.P + pb * kRows;
  // 16-byte pieces of a token: NS / 4 of B, as many of C, 4 Q of x, 4 Q of z
  const bool gates = tid < kScanBlock;
  auto load_dt = [&](int t) { return gates && t < end ? a.dt[(size_t)t * a.H + h] : 0.f; };
  float raw = load_dt(s + tid);  // of the block that is fetched next
  auto fetch = [&](int t0, Tokens& b) {
    constexpr int kBC = NS / 4, kX = kRows / 4, kPieces = 2 * kBC + 2 * kX;
    for (int v = tid; v < kScanBlock * kPieces; v += kScanThreads) {
      const int t = v / kPieces, p = v % kPieces;
      if (t0 + t >= end) break;
      const float* u = a.u + (size_t)(t0 + t) * a.Cc;
      const float* src;
      float* dst;
      if (p < kBC) {
        src = u + cB + 4 * p;
        dst = &b.B[t][4 * p];
      } else if (p < 2 * kBC) {
        src = u + cC + 4 * (p - kBC);
        dst = &b.C[t][4 * (p - kBC)];
      } else if (p < 2 * kBC + kX) {
        src = u + cx + 4 * (p - 2 * kBC);
        dst = &b.x[t][4 * (p - 2 * kBC)];
      } else {
        if (!a.z) continue;
        src = static_cast<const float*>(a.z) + (size_t)(t0 + t) * a.H * a.P + cx +
              4 * (p - 2 * kBC - kX);
        dst = &b.z[t][4 * (p - 2 * kBC - kX)];
      }
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (gates) {
      const float d = ssm_step(raw + bias, a.dt_min, a.dt_max);
      b.gate[tid] = make_float2(d, expf(rate * d));
      raw = t0 + tid < end - kScanBlock ? load_dt(t0 + kScanBlock + tid) : 0.f;
    }
  };
  if (s < end) fetch(s, buf[0]);
  for (int t0 = s, k = 0; t0 < end; t0 += kScanBlock, k ^= 1) {
    if (t0 + kScanBlock < end) {
      fetch(t0 + kScanBlock, buf[k ^ 1]);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    Tokens& b = buf[k];
    const int m = min(kScanBlock, end - t0);
    // U tokens, whose sums over lanes are independent and whose results leave together
    auto tokens = [&](int i, auto count) {
      constexpr int U = decltype(count)::value;
      float xv[U][Q], o[U * Q];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float2 gt = b.gate[i + u];
        float dx[Q], part[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          xv[u][q] = b.x[i + u][r0 + 4 * q];
          dx[q] = gt.x * xv[u][q];
        }
        ssm_rows_step(f, &b.B[i + u][4 * sub], &b.C[i + u][4 * sub], dx, gt.y, part);
#pragma unroll
        for (int q = 0; q < Q; ++q) o[u * Q + q] = part[q];
      }
      ssm_rows_sum(o);
      if (sub == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < Q; ++q) b.x[i + u][r0 + 4 * q] = fmaf(D, xv[u][q], o[u * Q + q]);
      }
    };
    constexpr int U = Q == 1 ? 8 : 2;
    int i = 0;
    for (; i + U <= m; i += U) tokens(i, std::integral_constant<int, U>());
    for (; i < m; ++i) tokens(i, std::integral_constant<int, 1>());
    __syncthreads();
    for (int v = tid; v < m * (kRows / 4); v += kScanThreads) {
      const int t = v / (kRows / 4), p = 4 * (v % (kRows / 4));
      float4 y = *reinterpret_cast<const float4*>(&b.x[t][p]);
      if (a.z) {
        const float4 z = *reinterpret_cast<const float4*>(&b.z[t][p]);
        y.x *= silu_f(z.x), y.y *= silu_f(z.y), y.z *= silu_f(z.z), y.w *= silu_f(z.w);
      }
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + (size_t)(t0 + t) * a.H * a.P + cx + p) = y;
    }
    __syncthreads();  // the buffer takes the tokens after the next ones
  }
  conv_history<float>(a, n, row, s, end, blockIdx.x % (blocks * a.H), blocks * a.H);
  if (a.SN && row >= 0) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int m = 0; m < M; ++m)
        __stcs(reinterpret_cast<float4*>(static_cast<float*>(a.SN) + sbase + (size_t)(4 * q) * NS +
                                         32 * m),
               f[q][m]);
  }
}

// ------------------------------------------------------------------------------- single tokens
// One token per sequence.  A group of heads (which share B and C) is worked on by a cluster of `cl`
// CTAs, each with `nb` blocks of 64 state rows one after the other: every warp streams its rows in
// batches, the next batch in flight while one is updated, the first on its way before the conv.
// Every CTA computes the conv of its own channels of x and, again, of the group's B and C (a few KB
// beside 32 KB of state in and out per block); it shifts the history of its x, and that of B and C
// is shifted, split over the cluster, when all of it has been read.  So it is one launch without a
// workspace, from one sequence (cl = 8: all the parallelism there is) to many (cl = 1).
// Bound by memory: 256 sequences of 32 heads of 128 x 128 take 183 us, 6.05 TB/s; 83 of 48 heads of
// 64 x 128 with the state in bf16 28.5 us, 4.8 TB/s; one of 64 heads 5.4 us in a graph.
template <typename T, typename TS, int NS>
__global__ void __launch_bounds__(kScanThreads, 4) ssm_step_kernel(SsmArgs a, int cl, int nb) {
  constexpr int M = NS / 32, Q = sizeof(TS) == 4 ? 2 : 4;  // quads per batch of a warp
  constexpr int kBatches = 4 / Q;                          // batches of a block of 64 rows
  extern __shared__ __align__(16) float st_s[];
  const int blocks = a.P / kScanRows, per = a.H / a.G, R = per * blocks;
  const int rank = blockIdx.x % cl, g = (blockIdx.x / cl) % a.G, n = blockIdx.x / (cl * a.G);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = lane >> 3, sub = lane & 7;
  const int row = state_row(a.slot, n, a.num_slots);
  if (row < 0) {  // slot out of range: the sequence is skipped (by its whole clusters)
    if (tid == 0 && rank == 0) report_status(a.status, GDN_ERR_INVALID_ARG);
    return;
  }
  const int b0 = rank * nb, mine = max(0, min(nb, R - b0));  // blocks b0 .. of the group
  float* B_s = st_s;                          // [NS]
  float* C_s = B_s + NS;                      // [NS]
  float* x_s = C_s + NS;                      // [64 nb] conv outputs, then y
  float2* gate_s = reinterpret_cast<float2*>(x_s + kScanRows * nb);  // [nb] decay, step of a block's head
  const int c0 = g * per * a.P + b0 * kScanRows;  // first channel of x (and of the output)
  TS* S = static_cast<TS*>(a.SN) + ((size_t)row * a.H * a.P + c0 + warp * 16 + grp) * NS + 4 * sub;
  auto load = [&](int bt, Raw<TS> (&r)[Q][M]) {  // batch bt of this warp's rows
    const TS* p = S + ((size_t)(bt / kBatches) * kScanRows + (bt % kBatches) * (4 * Q)) * NS;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int m = 0; m < M; ++m) r[q][m].load(p + (size_t)(4 * q) * NS + 32 * m);
  };
  Raw<TS> cur[Q][M], nxt[Q][M];
  if (mine > 0) load(0, cur);
  for (int b = tid; b < mine; b += kScanThreads) {
    const int h = g * per + (b0 + b) / blocks;
    const float d = ssm_step(a.dt[(size_t)n * a.H + h] + (a.dt_bias ? a.dt_bias[h] : 0.f), a.dt_min,
                             a.dt_max);
    gate_s[b] = make_float2(expf(-ssm_rate(a.a_log[h]) * d), d);
  }
  // ---- conv + SiLU, 4 channels per item: B, C, then this CTA's x
  const int cB = a.H * a.P + g * NS;
  T* hist = static_cast<T*>(a.convN) + (size_t)row * 3 * a.Cc;
  auto conv = [&](int c, float* u, float (&v)[4][4]) {
    float w[4][4], b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 3; ++j) load_t4(hist + (size_t)j * a.Cc + c, v[j]);
    load_t4(static_cast<const T*>(a.x) + (size_t)n * a.Cc + c, v[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) load_t4(static_cast<const T*>(a.conv_w) + (size_t)(c + e) * 4, w[e]);
    if (a.conv_b) load_t4(static_cast<const T*>(a.conv_b) + c, b);
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      y[e] = silu_f(fmaf(w[e][3], v[3][e],
                         fmaf(w[e][2], v[2][e], fmaf(w[e][1], v[1][e], fmaf(w[e][0], v[0][e], b[e])))));
    *reinterpret_cast<float4*>(u) = make_float4(y[0], y[1], y[2], y[3]);
  };
  auto shift = [&](int c, const float (&v)[4][4]) {
#pragma unroll
    for (int j = 0; j < 3; ++j) store_t4(hist + (size_t)j * a.Cc + c, v[j + 1]);
  };
  static_assert(2 * NS / 4 <= kScanThreads, "an item of B or C per thread");
  {
    const int cbc = tid < NS / 4 ? cB + 4 * tid : cB + (a.G - 1) * NS + 4 * tid;
    float v[4][4];
    const bool bc = tid < 2 * NS / 4;
    if (bc) conv(cbc, B_s + 4 * tid, v);
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // has read B's and C's
    for (int it = tid; it < mine * (kScanRows / 4); it += kScanThreads) {
      float vx[4][4];
      conv(c0 + 4 * it, x_s + 4 * it, vx);
      shift(c0 + 4 * it, vx);
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (bc && tid % cl == rank) shift(cbc, v);
  }
  __syncthreads();

  // ---- the state
  for (int bt = 0; bt < mine * kBatches; ++bt) {
    if (bt + 1 < mine * kBatches) load(bt + 1, nxt);
    const int b = bt / kBatches, r0 = warp * 16 + (bt % kBatches) * (4 * Q) + grp;
    const float2 gt = gate_s[b];
    float4 f[Q][M];
    float xv[Q], dx[Q], o[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      xv[q] = x_s[b * kScanRows + r0 + 4 * q];
      dx[q] = gt.y * xv[q];
#pragma unroll
      for (int m = 0; m < M; ++m) f[q][m] = cur[q][m].get();
    }
    ssm_rows_step(f, B_s + 4 * sub, C_s + 4 * sub, dx, gt.x, o);
    ssm_rows_sum(o);
    TS* p = S + ((size_t)b * kScanRows + (bt % kBatches) * (4 * Q)) * NS;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int m = 0; m < M; ++m) Raw<TS>::store(p + (size_t)(4 * q) * NS + 32 * m, f[q][m]);
    if (sub == 0) {  // y takes the place of x (read by this group of lanes alone)
      const float D = a.D ? a.D[g * per + (b0 + b) / blocks] : 0.f;
#pragma unroll
      for (int q = 0; q < Q; ++q) x_s[b * kScanRows + r0 + 4 * q] = fmaf(D, xv[q], o[q]);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int m = 0; m < M; ++m) cur[q][m] = nxt[q][m];
  }
  __syncthreads();
  // ---- outputs
  for (int it = tid; it < mine * (kScanRows / 4); it += kScanThreads) {
    const size_t at = (size_t)n * a.H * a.P + c0 + 4 * it;
    float y[4];
    load_t4(x_s + 4 * it, y);
    if (a.z) {
      float z[4];
      load_t4(static_cast<const T*>(a.z) + at, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] *= silu_f(z[e]);
    }
    store_t4(static_cast<T*>(a.out) + at, y);
  }
}

}  // namespace gdn

namespace gdn_host {

template <typename... KArgs, typename... Args>
static cudaError_t launch_ssm(const char* name, int cluster, void (*kern)(KArgs...),
                              dim3 grid, size_t smem, cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  trace_begin(name, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  trace_end(s);
  return e;
}

cudaError_t launch_ssm_tc(gdn::SsmTcArgs g, void* workspace, cudaStream_t s);
size_t ssm_tc_workspace(int N, int T, int H, int G, int P, int NS, int Cc);

template <int NS, int Q>
static cudaError_t launch_scan(const gdn::SsmArgs& a, cudaStream_t s) {
  const size_t smem = 2 * sizeof(gdn::ScanTokens<NS, Q>);
  if (smem > 48 * 1024) {  // per call, not once: the attribute belongs to the current device
    const cudaError_t e = cudaFuncSetAttribute(
        gdn::ssm_scan_kernel<NS, Q>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  // Not before the conv has ended: CTAs that start while it runs share the SMs it has left, and the
  // recurrence takes as long as its slowest SM (1021 tokens in three sequences: 191 us and not 106).
  return launch_ssm("ssm_scan", 1, gdn::ssm_scan_kernel<NS, Q>,
                    dim3((unsigned)a.N * a.H * (a.P / (16 * Q))), smem, s, a);
}

static cudaError_t launch_ssm_prefill(bool bf16, const gdn::SsmArgs& a, int NS, cudaStream_t s) {
  if (bf16) {
    gdn::SsmTcArgs g{};
    g.a = a;
    g.NS = NS;
    return launch_ssm_tc(g, a.u, s);
  }
  if (a.T > 0) {
    const dim3 grid((a.T + gdn::kConvRun - 1) / gdn::kConvRun, (a.Cc / 8 + 127) / 128);
    cudaError_t e = launch_ssm("ssm_conv", 1, gdn::ssm_conv_kernel, grid, 0, s, a);
    if (e != cudaSuccess) return e;
  }
  // Rows per CTA: 16 while all CTAs are resident at once, three to an SM (a token costs a warp one
  // quad and not four, and a block of tokens may be twice as long), else 64 (B and C are read for four
  // quads at once).  16 and 64 rows: three sequences of 1021 tokens in all, 4 heads of 128 x 128, 91
  // and 180 us; 1000 tokens of 64 heads of 64 x 128 in two sequences 283 and 266, in four 223 and 183.
  if ((int64_t)a.N * a.H * (a.P / 64) * 4 <= 3 * 148)
    return NS == 128 ? launch_scan<128, 1>(a, s) : launch_scan<64, 1>(a, s);
  return NS == 128 ? launch_scan<128, 4>(a, s) : launch_scan<64, 4>(a, s);
}

// Blocks of 64 state rows that share a group's B and C, and what a CTA may have of them (its conv
// outputs are in shared memory).
static int step_blocks(int H, int G, int P) { return (H / G) * (P / gdn::kScanRows); }
constexpr int kStepCluster = 8, kStepMost = 128;
// CTAs per group (R blocks of 64 rows), by the time in us that N sequences take: 148 SMs hold four
// CTAs each; a block of `bytes` (in and out) takes a CTA that is alone its latency, and all of them
// together the memory bandwidth; every wave costs 2 us to begin.  Measured at 83 sequences of 48 heads
// of 64 x 128 in one group, state in bf16: 8 CTAs (a second wave of 72) 36.9 us, 6 32.8, 4 34.8, 2
// 43.0, 1 63.5; 128 sequences of 24 heads of 64 x 64 in two groups: 8 CTAs 36.9 us, 2 26.6, 1 32.8;
// 256 of 32 heads of 128 x 128 in 16 groups: 1 184 us, 2 201, 4 238.
static int step_cluster(int N, int G, int R, size_t bytes) {
  constexpr int kSlots = 148 * 4;
  const double latency = 0.55 + 2e-5 * bytes, shared = bytes / 6.5e6;
  int best = std::min(kStepCluster, R);
  double least = 1e30;
  for (int cl = 1; cl <= kStepCluster && cl <= R; ++cl) {
    const int nb = (R + cl - 1) / cl;
    if (nb > kStepMost || (cl - 1) * nb >= R) continue;  // (the latter: a CTA without a block)
    const int64_t ctas = (int64_t)N * G * cl, full = ctas / kSlots, part = ctas % kSlots;
    const double time = full * (2.0 + nb * std::max(latency, kSlots * shared)) +
                        (part ? 2.0 + nb * std::max(latency, part * shared) : 0.0);
    if (time <= least * 1.001) {  // of equal ones the most CTAs: they hide one another's start
      least = time;
      best = cl;
    }
  }
  return best;
}

template <typename T, typename TS>
static cudaError_t launch_step(const gdn::SsmArgs& a, int NS, const char* name, cudaStream_t s) {
  const int R = step_blocks(a.H, a.G, a.P);
  const int cl = step_cluster(a.N, a.G, R, 2 * sizeof(TS) * gdn::kScanRows * NS);
  const int nb = (R + cl - 1) / cl;
  const dim3 grid((unsigned)a.N * a.G * cl);
  const size_t smem = (2 * NS + (gdn::kScanRows + 2) * nb) * sizeof(float);
  return NS == 128 ? launch_ssm(name, cl, gdn::ssm_step_kernel<T, TS, 128>, grid, smem, s, a,
                                cl, nb)
                   : launch_ssm(name, cl, gdn::ssm_step_kernel<T, TS, 64>, grid, smem, s, a,
                                cl, nb);
}

static cudaError_t launch_ssm_decode(bool bf16, bool state_bf16, const gdn::SsmArgs& a, int NS,
                                     cudaStream_t s) {
  const char* name = state_bf16 ? "ssm_decode_step_bf16_state" : "ssm_decode_step";
  if (bf16)
    return state_bf16 ? launch_step<__nv_bfloat16, __nv_bfloat16>(a, NS, name, s)
                      : launch_step<__nv_bfloat16, float>(a, NS, name, s);
  return state_bf16 ? launch_step<float, __nv_bfloat16>(a, NS, name, s)
                    : launch_step<float, float>(a, NS, name, s);
}

}  // namespace gdn_host

namespace {

bool misaligned(const void* p, uintptr_t to = 16) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

int64_t ssm_channels(const gdn_ssm_dims* d) {
  return (int64_t)d->num_heads * d->head_dim + 2 * (int64_t)d->num_groups * d->state_dim;
}

int check_ssm_dims(const gdn_ssm_dims* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->num_heads <= 0 || d->num_groups <= 0 || d->head_dim <= 0 || d->state_dim <= 0 ||
      d->conv_kernel <= 0 || d->num_heads % d->num_groups != 0)
    return GDN_ERR_INVALID_ARG;
  if (!(d->dt_min >= 0.f) || !(d->dt_max >= d->dt_min)) return GDN_ERR_INVALID_ARG;
  if ((d->head_dim != 64 && d->head_dim != 128) || (d->state_dim != 64 && d->state_dim != 128) ||
      d->conv_kernel != gdn::kConvK)
    return GDN_ERR_UNSUPPORTED;
  if (ssm_channels(d) > (1 << 20)) return GDN_ERR_UNSUPPORTED;  // 32-bit channel indices
  return GDN_OK;
}

bool ssm_dtype_ok(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }

gdn::SsmArgs ssm_args(const gdn_ssm_dims* d) {
  gdn::SsmArgs a{};
  a.H = d->num_heads;
  a.G = d->num_groups;
  a.P = d->head_dim;
  a.Cc = (int)ssm_channels(d);
  a.dt_min = d->dt_min;
  a.dt_max = d->dt_max;
  return a;
}

int ssm_prefill_impl(const gdn_ssm_dims* dims, gdn_dtype dtype, const void* x, const void* conv_w,
                     const void* conv_b, const float* dt, const float* dt_bias, const float* a_log,
                     const float* D, const void* z, const int32_t* cu, int32_t N, int32_t T,
                     const int32_t* slot, int32_t num_slots, const float* S0, float* SN,
                     const void* conv0, void* convN, void* out, void* workspace,
                     size_t workspace_bytes, int32_t* dev_status, void* stream) {
  int rc = check_ssm_dims(dims);
  if (rc) return rc;
  if (!ssm_dtype_ok(dtype)) return GDN_ERR_UNSUPPORTED;
  if (N < 0 || T < 0 || (N == 0 && T > 0)) return GDN_ERR_INVALID_ARG;
  if (N > 0 && (!cu || !a_log)) return GDN_ERR_INVALID_ARG;
  if (T > 0 && (!x || !conv_w || !dt || !out)) return GDN_ERR_INVALID_ARG;
  const void* ptrs[] = {x, conv_w, conv_b, dt, dt_bias, a_log, D, z, S0, SN, conv0, convN, out};
  for (const void* p : ptrs)
    if (p && misaligned(p)) return GDN_ERR_INVALID_ARG;
  if (misaligned(cu, 4) || misaligned(slot, 4) || misaligned(dev_status, 4))
    return GDN_ERR_INVALID_ARG;
  if (workspace && misaligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
  // a grid covers every (sequence or chunk, head, 64 rows), or (chunk, group, gates of 32 heads)
  if (((int64_t)N + T / 128) * dims->num_heads * 2 > INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < gdn_ssm_prefill_workspace_size(dims, dtype, N, T))
    return GDN_ERR_WORKSPACE;
  if (N == 0) return GDN_OK;
  gdn::SsmArgs a = ssm_args(dims);
  a.x = x;
  a.conv_w = conv_w;
  a.conv_b = conv_b;
  a.dt = dt;
  a.dt_bias = dt_bias;
  a.a_log = a_log;
  a.D = D;
  a.z = z;
  a.cu = cu;
  a.S0 = S0;
  a.SN = SN;
  a.conv0 = conv0;
  a.convN = convN;
  a.out = out;
  a.slot = slot;
  a.status = dev_status;
  a.u = static_cast<float*>(workspace);
  a.num_slots = num_slots;
  a.N = N;
  a.T = T;
  return gdn_host::launch_ssm_prefill(dtype == GDN_BF16, a, dims->state_dim,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

}  // namespace

extern "C" {

int64_t gdn_ssm_conv_channels(const gdn_ssm_dims* dims) { return dims ? ssm_channels(dims) : -1; }

size_t gdn_ssm_prefill_workspace_size(const gdn_ssm_dims* dims, gdn_dtype dtype, int32_t num_seqs,
                                      int32_t num_tokens) {
  if (check_ssm_dims(dims) != GDN_OK || !ssm_dtype_ok(dtype) || num_seqs < 0 || num_tokens < 0)
    return 0;
  if (dtype == GDN_BF16)
    return 256 + gdn_host::ssm_tc_workspace(num_seqs, num_tokens, dims->num_heads,
                                            dims->num_groups, dims->head_dim, dims->state_dim,
                                            (int)ssm_channels(dims));
  return 256 + (size_t)num_tokens * ssm_channels(dims) * 4;
}

int gdn_ssm_prefill(const gdn_ssm_dims* dims, gdn_dtype dtype, const void* x, const void* conv_w,
                    const void* conv_b, const float* dt, const float* dt_bias, const float* a_log,
                    const float* D, const void* z, const int32_t* cu_seqlens, int32_t num_seqs,
                    int32_t num_tokens, const float* S0, float* SN, const void* conv0, void* convN,
                    void* out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                    void* stream) {
  return ssm_prefill_impl(dims, dtype, x, conv_w, conv_b, dt, dt_bias, a_log, D, z, cu_seqlens,
                          num_seqs, num_tokens, nullptr, num_seqs, S0, SN, conv0, convN, out,
                          workspace, workspace_bytes, dev_status, stream);
}

int gdn_ssm_prefill_slots(const gdn_ssm_dims* dims, gdn_dtype dtype, const void* x,
                          const void* conv_w, const void* conv_b, const float* dt,
                          const float* dt_bias, const float* a_log, const float* D, const void* z,
                          const int32_t* cu_seqlens, int32_t num_seqs, int32_t num_tokens,
                          const int32_t* slot_idx, int32_t num_slots, float* S_pool,
                          void* conv_pool, void* out, void* workspace, size_t workspace_bytes,
                          int32_t* dev_status, void* stream) {
  if (num_seqs > 0 && !S_pool) return GDN_ERR_INVALID_ARG;
  if (num_slots < 0 || (!slot_idx && num_slots < num_seqs)) return GDN_ERR_INVALID_ARG;
  return ssm_prefill_impl(dims, dtype, x, conv_w, conv_b, dt, dt_bias, a_log, D, z, cu_seqlens,
                          num_seqs, num_tokens, slot_idx, num_slots, S_pool, S_pool, conv_pool,
                          conv_pool, out, workspace, workspace_bytes, dev_status, stream);
}

int gdn_ssm_decode_step(const gdn_ssm_dims* dims, gdn_dtype dtype, gdn_dtype state_dtype,
                        const void* x, const void* conv_w, const void* conv_b, const float* dt,
                        const float* dt_bias, const float* a_log, const float* D, const void* z,
                        void* conv_state, void* S, const int32_t* slot_idx, int32_t num_slots,
                        int32_t batch, void* out, int32_t* dev_status, void* stream) {
  int rc = check_ssm_dims(dims);
  if (rc) return rc;
  if (!ssm_dtype_ok(dtype) || !ssm_dtype_ok(state_dtype)) return GDN_ERR_UNSUPPORTED;
  if (batch < 0) return GDN_ERR_INVALID_ARG;
  if (num_slots < 0 || (!slot_idx && num_slots < batch)) return GDN_ERR_INVALID_ARG;
  if (batch > 0 && (!x || !conv_w || !dt || !a_log || !conv_state || !S || !out))
    return GDN_ERR_INVALID_ARG;
  const void* ptrs[] = {x, conv_w, conv_b, dt, dt_bias, a_log, D, z, conv_state, S, out};
  for (const void* p : ptrs)
    if (p && misaligned(p)) return GDN_ERR_INVALID_ARG;
  if (misaligned(slot_idx, 4) || misaligned(dev_status, 4)) return GDN_ERR_INVALID_ARG;
  // the grid covers every (sequence, group, CTA of its cluster); a CTA holds its conv outputs
  if ((int64_t)batch * dims->num_groups * gdn_host::kStepCluster > INT32_MAX ||
      gdn_host::step_blocks(dims->num_heads, dims->num_groups, dims->head_dim) >
          gdn_host::kStepCluster * gdn_host::kStepMost)
    return GDN_ERR_UNSUPPORTED;
  if (batch == 0) return GDN_OK;
  gdn::SsmArgs a = ssm_args(dims);
  a.x = x;
  a.conv_w = conv_w;
  a.conv_b = conv_b;
  a.dt = dt;
  a.dt_bias = dt_bias;
  a.a_log = a_log;
  a.D = D;
  a.z = z;
  a.SN = S;
  a.convN = conv_state;
  a.out = out;
  a.slot = slot_idx;
  a.status = dev_status;
  a.num_slots = num_slots;
  a.N = a.T = batch;
  return gdn_host::launch_ssm_decode(dtype == GDN_BF16, state_dtype == GDN_BF16, a,
                                     dims->state_dim,
                                     static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

}  // extern "C"
