// ssm.cu -- selective state space layer: entry points, the single-token step and the fp32 prompts.
// Causal depthwise conv (width 4, bias) + SiLU, then the recurrence
// S_t = exp(-exp(a_log) delta) S_{t-1} + delta x_t B_t^T, y_t = S_t C_t + D x_t with 64 rows of a
// head's state [P, N] in the registers of a CTA, and the gate silu(z) (formulas in gdn.h).  Prompts
// with bf16 activations run on the tensor cores (ssm_tc.cu).
#include <cuda_runtime.h>

#include <utility>

#include "args.cuh"
#include "common.cuh"
#include "ssm.cuh"
#include "tc.cuh"

namespace gdn {

constexpr int kScanThreads = 128;
constexpr int kScanRows = 64;   // rows of the state per CTA (16 per warp, 8 lanes per row)
constexpr int kConvRun = 16;    // tokens per thread of the packed conv

// Packed prompts: a thread owns 8 channels and a run of kConvRun tokens, the three rows before
// the current one in registers.
template <typename T>
__global__ void __launch_bounds__(128) ssm_conv_kernel(SsmArgs a) {
  pdl_trigger();
  const int c = (blockIdx.y * 128 + threadIdx.x) * 8, t0 = blockIdx.x * kConvRun;
  if (c >= a.Cc) return;
  float w[4][8], b[8];
  load_taps<T>(a, c, w, b);
  const T* x = static_cast<const T*>(a.x) + c;
  const T* c0 = static_cast<const T*>(a.conv0);
  float h[3][8];
  int n = seq_of_token(a.cu, a.N, t0) - 1, s = 0, end = 0;
  const int t1 = min(a.T, t0 + kConvRun);
  bool fresh = true;  // the history registers do not hold the rows before t
  for (int t = t0; t < t1; ++t) {
    while (n < a.N && t >= end) {  // the next sequence that may hold t
      ++n;
      if (n < a.N) seq_range(a, n, s, end);
      fresh = true;
    }
    if (n >= a.N || t < s) continue;  // behind the last sequence
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
      fresh = false;
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

// One token per sequence: a thread owns 8 channels of one sequence and shifts their history.
template <typename T>
__global__ void __launch_bounds__(128) ssm_conv_step_kernel(SsmArgs a) {
  pdl_trigger();
  const int c = (blockIdx.x * 128 + threadIdx.x) * 8, n = blockIdx.y;
  if (c >= a.Cc) return;
  const int row = state_row(a.slot, n, a.num_slots);
  if (row < 0) {  // slot out of range: the sequence is skipped
    if (c == 0) report_status(a.status, GDN_ERR_INVALID_ARG);
    return;
  }
  float w[4][8], b[8], h[4][8], out[8];
  T* cs = static_cast<T*>(a.convN) + (size_t)row * 3 * a.Cc + c;
#pragma unroll
  for (int j = 0; j < 3; ++j) load8(cs + (size_t)j * a.Cc, h[j]);
  load8(static_cast<const T*>(a.x) + (size_t)n * a.Cc + c, h[3]);
  load_taps<T>(a, c, w, b);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    out[e] = silu_f(fmaf(w[3][e], h[3][e],
                         fmaf(w[2][e], h[2][e], fmaf(w[1][e], h[1][e], fmaf(w[0][e], h[0][e], b[e])))));
#pragma unroll
  for (int j = 0; j < 3; ++j) store8(cs + (size_t)j * a.Cc, h[j + 1]);
  store8(a.u + (size_t)n * a.Cc + c, out);
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

// Four consecutive elements of a state row.
__device__ __forceinline__ float4 load4(const float* p) {
  return __ldcs(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
  const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
  const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void store4(float* p, float4 v) {
  __stcs(reinterpret_cast<float4*>(p), v);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)));
}

// Lane `sub` of a row's eight lanes holds columns 4 sub + 32 m + e (m < NS / 32).  Warp w owns
// rows 16 w + 4 q + lane / 8 (q < 4) of the CTA's 64.
template <typename TS, int NS>
struct StateRows {
  static constexpr int M = NS / 32;
  float4 f[4][M];
  __device__ __forceinline__ void load(const TS* p) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int m = 0; m < M; ++m)
        f[q][m] = p ? load4(p + (size_t)(4 * q) * NS + 32 * m) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void store(TS* p) const {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int m = 0; m < M; ++m) store4(p + (size_t)(4 * q) * NS + 32 * m, f[q][m]);
  }
  // One token: the rows take alpha S + (delta x) B^T; returns S C of row q in every lane of its
  // group of eight.  B, C: the lane's first column.
  __device__ __forceinline__ void step(const float* B, const float* C, const float (&dx)[4],
                                       float alpha, float (&o)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float4 b = *reinterpret_cast<const float4*>(B + 32 * m);
      const float4 c = *reinterpret_cast<const float4*>(C + 32 * m);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float4& r = f[q][m];
        r.x = fmaf(alpha, r.x, dx[q] * b.x);
        r.y = fmaf(alpha, r.y, dx[q] * b.y);
        r.z = fmaf(alpha, r.z, dx[q] * b.z);
        r.w = fmaf(alpha, r.w, dx[q] * b.w);
        o[q] = fmaf(r.x, c.x, fmaf(r.y, c.y, fmaf(r.z, c.z, fmaf(r.w, c.w, o[q]))));
      }
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1)
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] += __shfl_xor_sync(0xffffffffu, o[q], off);
  }
};

// Lane `sub` < 4 of a group writes its row 4 sub: y = S C + D x, gated.
template <typename T>
__device__ __forceinline__ void store_y(const SsmArgs& a, int t, int h, int p0, int sub, float D,
                                        const float (&xv)[4], const float (&o)[4]) {
  if (sub < 4) {
    const float y0 = sub == 0 ? o[0] : (sub == 1 ? o[1] : (sub == 2 ? o[2] : o[3]));
    const float x0 = sub == 0 ? xv[0] : (sub == 1 ? xv[1] : (sub == 2 ? xv[2] : xv[3]));
    float y = fmaf(D, x0, y0);
    const size_t at = ((size_t)t * a.H + h) * a.P + p0 + 4 * sub;
    if (a.z) y *= silu_f(to_f(static_cast<const T*>(a.z)[at]));
    static_cast<T*>(a.out)[at] = from_f<T>(y);
  }
}

// ------------------------------------------------------------------------- packed prompts, fp32
// Tokens of a sequence come kScanBlock at a time to shared memory (B, C, the CTA's 64 channels of x,
// step and decay), the next ones in flight while these are worked through.
constexpr int kScanBlock = 16;
template <int NS>
struct ScanTokens {
  float B[kScanBlock][NS], C[kScanBlock][NS], x[kScanBlock][kScanRows];
  float2 gate[kScanBlock];  // step, decay
};

template <int NS>
__global__ void __launch_bounds__(kScanThreads, 4) ssm_scan_kernel(SsmArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  ScanTokens<NS>* buf = reinterpret_cast<ScanTokens<NS>*>(smem);  // [2]
  pdl_trigger();
  const int blocks = a.P / kScanRows;
  const int pb = blockIdx.x % blocks, h = (blockIdx.x / blocks) % a.H;
  const int n = blockIdx.x / (blocks * a.H);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = lane >> 3, sub = lane & 7;
  const int row = state_row(a.slot, n, a.num_slots);
  if (row < 0 && tid == 0) report_status(a.status, GDN_ERR_INVALID_ARG);
  int s, end;
  seq_range(a, n, s, end);
  const int p0 = pb * kScanRows + warp * 16 + grp;  // this lane group's rows: p0 + 4 q
  const size_t sbase = (((size_t)(row < 0 ? 0 : row) * a.H + h) * a.P + p0) * NS + 4 * sub;
  StateRows<float, NS> S;
  S.load(a.S0 && row >= 0 ? static_cast<const float*>(a.S0) + sbase : nullptr);
  const float rate = -expf(a.a_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const float D = a.D ? a.D[h] : 0.f;
  const int cB = a.H * a.P + (h / (a.H / a.G)) * NS, cC = cB + a.G * NS;
  const int cx = h * a.P + pb * kScanRows;
  // 16-byte pieces of a token: NS / 4 of B, as many of C, 16 of x
  auto fetch = [&](int t0, ScanTokens<NS>& b) {
    constexpr int kPieces = NS / 2 + kScanRows / 4;
    for (int v = tid; v < kScanBlock * kPieces; v += kScanThreads) {
      const int t = v / kPieces, p = v % kPieces;
      const int c = p < NS / 4 ? cB + 4 * p
                               : (p < NS / 2 ? cC + 4 * p - NS : cx + 4 * p - 2 * NS);
      float* dst = p < NS / 4 ? &b.B[t][4 * p]
                              : (p < NS / 2 ? &b.C[t][4 * p - NS] : &b.x[t][4 * p - 2 * NS]);
      if (t0 + t < end)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)),
                     "l"(a.u + (size_t)(t0 + t) * a.Cc + c)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tid < kScanBlock && t0 + tid < end) {
      const float d = ssm_step(a.dt[(size_t)(t0 + tid) * a.H + h] + bias, a.dt_min, a.dt_max);
      b.gate[tid] = make_float2(d, expf(rate * d));
    }
  };
  pdl_wait();  // the conv outputs
  if (s < end) fetch(s, buf[0]);
  for (int t0 = s, k = 0; t0 < end; t0 += kScanBlock, k ^= 1) {
    if (t0 + kScanBlock < end) {
      fetch(t0 + kScanBlock, buf[k ^ 1]);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const ScanTokens<NS>& b = buf[k];
    const int m = min(kScanBlock, end - t0);
#pragma unroll 2
    for (int i = 0; i < m; ++i) {
      float xv[4], dx[4], o[4];
      const float2 gt = b.gate[i];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        xv[q] = b.x[i][warp * 16 + grp + 4 * q];
        dx[q] = gt.x * xv[q];
      }
      S.step(&b.B[i][4 * sub], &b.C[i][4 * sub], dx, gt.y, o);
      store_y<float>(a, t0 + i, h, p0, sub, D, xv, o);
    }
    __syncthreads();  // the buffer takes the tokens after the next ones
  }
  conv_history<float>(a, n, row, s, end, blockIdx.x % (blocks * a.H), blocks * a.H);
  if (a.SN && row >= 0) S.store(static_cast<float*>(a.SN) + sbase);
}

// ------------------------------------------------------------------------------- single tokens
// One token per sequence: the rows of the state are on their way before the conv.
//   FUSED: the CTAs of a group of heads are one cluster.  Each computes the conv of its own 64
//   channels of x and of the group's B and C (a few KB beside 64 KB of state in and out), and
//   shifts the history of its x; that of B and C is shifted, split over the cluster, when all of
//   it has been read.  One launch and no workspace: 256 sequences of 32 heads of 128 x 128 take
//   the state's bytes; one sequence the latency of one launch.
//   Else (more than 8 CTAs share B and C): the conv outputs come from ssm_conv_step_kernel.
template <typename T, typename TS, int NS, bool FUSED>
__global__ void __launch_bounds__(kScanThreads, 4) ssm_step_kernel(SsmArgs a) {
  __shared__ __align__(16) float u_s[kScanRows + 2 * NS];  // x | B | C
  const int blocks = a.P / kScanRows, per = a.H / a.G;
  const int pb = blockIdx.x % blocks, h = (blockIdx.x / blocks) % a.H;
  const int n = blockIdx.x / (blocks * a.H), g = h / per;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grp = lane >> 3, sub = lane & 7;
  const int row = state_row(a.slot, n, a.num_slots);
  if (row < 0) {  // slot out of range: the sequence is skipped (by its whole clusters)
    if (tid == 0) report_status(a.status, GDN_ERR_INVALID_ARG);
    if (!FUSED) pdl_wait();
    return;
  }
  const int p0 = pb * kScanRows + warp * 16 + grp;
  const size_t sbase = (((size_t)row * a.H + h) * a.P + p0) * NS + 4 * sub;
  StateRows<TS, NS> S;
  S.load(static_cast<const TS*>(a.S0) + sbase);
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f, D = a.D ? a.D[h] : 0.f;
  const float delta = ssm_step(a.dt[(size_t)n * a.H + h] + bias, a.dt_min, a.dt_max);
  const float alpha = expf(-expf(a.a_log[h]) * delta);
  const int cx = h * a.P + pb * kScanRows, cB = a.H * a.P + g * NS, cC = cB + a.G * NS;
  constexpr int kItems = (kScanRows + 2 * NS) / 4;  // of 4 channels, one per thread
  const int rank = (h % per) * blocks + pb, ranks = per * blocks;
  const int c = tid < kScanRows / 4 ? cx + 4 * tid
                                    : (tid < (kScanRows + NS) / 4 ? cB + 4 * tid - kScanRows
                                                                  : cC + 4 * tid - kScanRows - NS);
  if (FUSED) {
    float v[4][4], w[4][4], b[4] = {0.f, 0.f, 0.f, 0.f};
    T* cs = static_cast<T*>(a.convN) + (size_t)row * 3 * a.Cc + c;
    if (tid < kItems) {
#pragma unroll
      for (int j = 0; j < 3; ++j) load_t4(cs + (size_t)j * a.Cc, v[j]);
      load_t4(static_cast<const T*>(a.x) + (size_t)n * a.Cc + c, v[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) load_t4(static_cast<const T*>(a.conv_w) + (size_t)(c + e) * 4, w[e]);
      if (a.conv_b) load_t4(static_cast<const T*>(a.conv_b) + c, b);
      float4 u;
      float* up = &u.x;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        up[e] = silu_f(fmaf(w[e][3], v[3][e],
                            fmaf(w[e][2], v[2][e], fmaf(w[e][1], v[1][e], fmaf(w[e][0], v[0][e], b[e])))));
      *reinterpret_cast<float4*>(u_s + 4 * tid) = u;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // has read the history
    const bool x_part = tid < kScanRows / 4;
    if (tid < kItems && x_part) {
#pragma unroll
      for (int j = 0; j < 3; ++j) store_t4(cs + (size_t)j * a.Cc, v[j + 1]);
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid < kItems && !x_part && tid % ranks == rank) {
#pragma unroll
      for (int j = 0; j < 3; ++j) store_t4(cs + (size_t)j * a.Cc, v[j + 1]);
    }
    __syncthreads();
  } else {
    pdl_wait();  // the conv outputs
    if (tid < kItems)
      *reinterpret_cast<float4*>(u_s + 4 * tid) =
          *reinterpret_cast<const float4*>(a.u + (size_t)n * a.Cc + c);
    __syncthreads();
  }
  float xv[4], dx[4], o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    xv[q] = u_s[warp * 16 + grp + 4 * q];
    dx[q] = delta * xv[q];
  }
  S.step(u_s + kScanRows + 4 * sub, u_s + kScanRows + NS + 4 * sub, dx, alpha, o);
  S.store(static_cast<TS*>(a.SN) + sbase);
  store_y<T>(a, n, h, p0, sub, D, xv, o);
}

}  // namespace gdn

namespace gdn_host {

template <typename K>
static cudaError_t launch_ssm(bool pdl, int cluster, K kern, dim3 grid, size_t smem, cudaStream_t s,
                              const gdn::SsmArgs& a, const char* name) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl && !trace_attached()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  trace_begin(name, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  trace_end(s);
  return e;
}

cudaError_t launch_ssm_tc(gdn::SsmTcArgs g, void* workspace, cudaStream_t s);
size_t ssm_tc_workspace(int N, int T, int H, int G, int P, int NS, int Cc);

static cudaError_t launch_ssm_prefill(bool bf16, const gdn::SsmArgs& a, int NS, cudaStream_t s) {
  if (bf16) {
    gdn::SsmTcArgs g{};
    g.a = a;
    g.NS = NS;
    return launch_ssm_tc(g, a.u, s);
  }
  if (a.T > 0) {
    const dim3 grid((a.T + gdn::kConvRun - 1) / gdn::kConvRun, (a.Cc / 8 + 127) / 128);
    cudaError_t e = launch_ssm(false, 1, gdn::ssm_conv_kernel<float>, grid, 0, s, a, "ssm_conv");
    if (e != cudaSuccess) return e;
  }
  const bool pdl = a.T > 0;  // behind a conv of this call; alone, it is an ordinary launch
  const dim3 grid((unsigned)a.N * a.H * (a.P / gdn::kScanRows));
  const size_t smem = 2 * (NS == 128 ? sizeof(gdn::ScanTokens<128>) : sizeof(gdn::ScanTokens<64>));
  return NS == 128
             ? launch_ssm(pdl, 1, gdn::ssm_scan_kernel<128>, grid, smem, s, a, "ssm_scan")
             : launch_ssm(pdl, 1, gdn::ssm_scan_kernel<64>, grid, smem, s, a, "ssm_scan");
}

// CTAs that share a group's B and C in a decode step, if they can be one cluster (8 at most, the
// portable size); 0: the conv is a kernel of its own.
static int step_cluster(int H, int G, int P) {
  const int n = (H / G) * (P / gdn::kScanRows);
  return n <= 8 ? n : 0;
}

template <typename T, typename TS, int NS>
static cudaError_t launch_step(const gdn::SsmArgs& a, const char* name, cudaStream_t s) {
  const dim3 grid((unsigned)a.N * a.H * (a.P / gdn::kScanRows));
  const int cluster = step_cluster(a.H, a.G, a.P);
  if (cluster > 0)
    return launch_ssm(false, cluster, gdn::ssm_step_kernel<T, TS, NS, true>, grid, 0, s, a, name);
  cudaError_t e = launch_ssm(false, 1, gdn::ssm_conv_step_kernel<T>,
                             dim3((a.Cc / 8 + 127) / 128, a.N), 0, s, a, "ssm_conv_step");
  if (e != cudaSuccess) return e;
  return launch_ssm(true, 1, gdn::ssm_step_kernel<T, TS, NS, false>, grid, 0, s, a, name);
}

template <typename T, typename TS>
static cudaError_t launch_step_n(const gdn::SsmArgs& a, int NS, const char* name, cudaStream_t s) {
  return NS == 128 ? launch_step<T, TS, 128>(a, name, s) : launch_step<T, TS, 64>(a, name, s);
}

static cudaError_t launch_ssm_decode(bool bf16, bool state_bf16, const gdn::SsmArgs& a, int NS,
                                     cudaStream_t s) {
  const char* name = state_bf16 ? "ssm_decode_step_bf16_state" : "ssm_decode_step";
  if (bf16)
    return state_bf16 ? launch_step_n<__nv_bfloat16, __nv_bfloat16>(a, NS, name, s)
                      : launch_step_n<__nv_bfloat16, float>(a, NS, name, s);
  return state_bf16 ? launch_step_n<float, __nv_bfloat16>(a, NS, name, s)
                    : launch_step_n<float, float>(a, NS, name, s);
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
  if (workspace && misaligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
  // a grid covers every (sequence or chunk, head, 64 rows)
  if (((int64_t)N + T / 128) * dims->num_heads * (dims->head_dim / gdn::kScanRows) > INT32_MAX)
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

size_t gdn_ssm_decode_workspace_size(const gdn_ssm_dims* dims, int32_t batch) {
  if (check_ssm_dims(dims) != GDN_OK || batch < 0) return 0;
  if (gdn_host::step_cluster(dims->num_heads, dims->num_groups, dims->head_dim) > 0) return 0;
  return (size_t)batch * ssm_channels(dims) * 4;
}

int gdn_ssm_decode_step(const gdn_ssm_dims* dims, gdn_dtype dtype, gdn_dtype state_dtype,
                        const void* x, const void* conv_w, const void* conv_b, const float* dt,
                        const float* dt_bias, const float* a_log, const float* D, const void* z,
                        void* conv_state, void* S, const int32_t* slot_idx, int32_t num_slots,
                        int32_t batch, void* out, void* workspace, size_t workspace_bytes,
                        int32_t* dev_status, void* stream) {
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
  if (workspace && misaligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
  // grids: (sequence, head, 64 rows), and the sequences as the second dimension of the conv's
  if (batch > 65535 ||
      (int64_t)batch * dims->num_heads * (dims->head_dim / gdn::kScanRows) > INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  if (batch == 0) return GDN_OK;
  const size_t need = gdn_ssm_decode_workspace_size(dims, batch);
  if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  gdn::SsmArgs a = ssm_args(dims);
  a.x = x;
  a.conv_w = conv_w;
  a.conv_b = conv_b;
  a.dt = dt;
  a.dt_bias = dt_bias;
  a.a_log = a_log;
  a.D = D;
  a.z = z;
  a.S0 = S;
  a.SN = S;
  a.convN = conv_state;
  a.out = out;
  a.slot = slot_idx;
  a.status = dev_status;
  a.u = static_cast<float*>(workspace);
  a.num_slots = num_slots;
  a.N = a.T = batch;
  return gdn_host::launch_ssm_decode(dtype == GDN_BF16, state_dtype == GDN_BF16, a,
                                     dims->state_dim,
                                     static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

}  // extern "C"
