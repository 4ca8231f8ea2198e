// ssm_tc.cu -- packed prefill of the selective state space layer on tcgen05 tensor cores (bf16
// activations, fp32 state), in chunks of 128 tokens.
//
// With cum_i the running log2 of the decay inside a chunk, delta the steps, u the conv outputs:
//   Y    = diag(2^cum) C S^T + P X,   P_ij = 2^(cum_i - cum_j) delta_j C_i.B_j  (j <= i)
//   S^T <- 2^cum_L S^T + B^T diag(2^(cum_L - cum_j) delta_j) X
// Precision.  The state is returned in fp32, so its update keeps both factors in two bf16 parts
// (three products, 2^-16 of each factor is left out); outputs are rounded to bf16, so their
// products take fp16 operands (11 bits) once.  fp16 has few exponent bits: rows of C, B and X are
// scaled by a power of two each (exponent from the row's largest value), S by one per chunk, and
// P by the row's largest weight, so that nothing overflows and what underflows is 2^-24 of what
// it is added to.  With lf_j = log2(delta_j) + the exponents of rows X_j and B_j,
//   g_j = lf_j - cum_j,  pm_i = max over j <= i of g_j:   P^_ij = (C^_i.B^_j) 2^(g_j - pm_i)
// (never above the product), and row i of the result counts 2^(cum_i + pm_i + exponent of C_i).
// cum and g are kept in fp64 (they reach thousands, and only their differences count).
//
// Kernels (programmatic dependent launch between them):
//   bc    per (chunk, group): conv of B and C; the operand tiles C^ (fp16) and B (two bf16
//         parts) in the swizzled layout the products read, C^ B^^T (tcgen05) as fp16; and a copy
//         of the initial conv history, so that the final one may overwrite it.
//   seg   per (segment of a sequence that another one follows, 128 channels): the state it adds.
//   main  per (segment, 128 channels): the state that enters it (from the segments before), then
//         chunk by chunk the outputs and the state.
// A sequence is cut into segments only to fill the GPU; the conv of X and the state update of
// all segments but the last run twice then.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "args.cuh"
#include "common.cuh"
#include "ssm.cuh"
#include "tc.cuh"

namespace gdn {

constexpr int kL = 128;                    // chunk length
constexpr uint32_t kTileB = 16384;         // one [128][64] 16-bit row tile
constexpr uint32_t kBcBytes = 6 * kTileB;  // C^ | B high | B low of a (chunk, group)
constexpr int kPipe = 256;                 // threads of one 64-channel pipeline

// idesc of idesc_bf16 with fp16 operands (format fields 0)
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_bf16(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}

__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
// v = high part + low part, both bf16 (half a step each)
__device__ __forceinline__ void split2(float2 v, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(v.x, v.y);
  const float2 h = unpack_bf16x2(hi);
  lo = pack_bf16x2(v.x - h.x, v.y - h.y);
}
// silu by one exponential and one division, each good to about 2^-22
__device__ __forceinline__ float silu_div(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// Exponent of the largest magnitude of a row (its bits), within [-100, 127]; the row is scaled
// by pow2(target - exponent).
__device__ __forceinline__ int exponent_of(uint32_t abs_bits) {
  return max((int)(abs_bits >> 23) - 127, -100);
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }
constexpr int kTargetBC = 3;   // rows of C and B below 2^4: their products stay below 2^15
constexpr int kTargetX = 13;
constexpr int kTargetS = 14;

// Unit k of the packed batch: sequences cut into units of `tokens`, numbered sequence by
// sequence; with `empty` a sequence without tokens has one unit too.  All threads of the CTA
// call it; scratch: 3 int64 per warp and a Unit in shared memory.
struct Unit {
  int n;        // sequence, or -1: no such unit
  int j;        // unit inside the sequence
  int s, e;     // its sequence's tokens
  int chunk;    // first chunk of the sequence
  int first;    // first unit of the sequence
};
// `most_units`: units the launch has room for.
__device__ __forceinline__ Unit find_unit(const SsmArgs& a, int tokens, bool empty, int k,
                                          int64_t most_units, void* scratch) {
  int64_t* wsum = reinterpret_cast<int64_t*>(scratch);  // [warps][2]
  Unit* res = reinterpret_cast<Unit*>(wsum + 64);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int64_t most = (int64_t)a.T / kL + a.N;  // chunks the workspace holds
  if (tid == 0) res->n = -1;
  int64_t u0 = 0, c0 = 0;
  for (int base = 0; base < a.N; base += blockDim.x) {
    const int n = base + tid;
    int s = 0, e = 0;
    if (n < a.N) seq_range(a, n, s, e);
    const int nc = (e - s + kL - 1) / kL;
    const int nu = n < a.N ? max((e - s + tokens - 1) / tokens, empty ? 1 : 0) : 0;
    int64_t ui = nu, ci = nc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t uu = __shfl_up_sync(0xffffffffu, ui, o);
      const int64_t cc = __shfl_up_sync(0xffffffffu, ci, o);
      if (lane >= o) {
        ui += uu;
        ci += cc;
      }
    }
    __syncthreads();
    if (lane == 31) {
      wsum[2 * warp] = ui;
      wsum[2 * warp + 1] = ci;
    }
    __syncthreads();
    int64_t ub = u0, cb = c0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) {
        ub += wsum[2 * w];
        cb += wsum[2 * w + 1];
      }
      u0 += wsum[2 * w];
      c0 += wsum[2 * w + 1];
    }
    const int64_t uf = ub + ui - nu, cf = cb + ci - nc;
    if (k >= uf && k < uf + nu) {
      Unit r{n, (int)(k - uf), s, e, (int)cf, (int)uf};
      if (cf + nc > most || uf + nu > most_units) {  // sequences that overlap: no room for it
        report_status(a.status, GDN_ERR_INVALID_ARG);
        r.e = r.s;
        if (r.j > 0 || !empty) r.n = -1;
      }
      *res = r;
    }
    if (u0 > k) break;  // uniform: every thread adds the same sums
  }
  __syncthreads();
  const Unit r = *res;
  __syncthreads();
  return r;
}

// ------------------------------------------------------------------------------------- bc
// 256 threads: lanes 0-15 hold 8 channels of B each, lanes 16-31 of C; warp w has tokens
// 16 w .. 16 w + 15 of the chunk.  State widths below 128 are padded with zero channels.
constexpr uint32_t kBcSmem = 4 * kTileB + 2048;

__global__ void __launch_bounds__(256, 2) ssm_bc_kernel(SsmTcArgs g) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const SsmArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* ctl = sm + 4 * kTileB;
  uint64_t* bar = reinterpret_cast<uint64_t*>(ctl);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(ctl + 8);
  pdl_trigger();
  const int grp = blockIdx.x % a.G;
  const Unit un = find_unit(a, kL, false, blockIdx.x / a.G, gridDim.x / a.G, sm);
  if (un.n < 0) return;
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(tslot, 128);
  const int t0 = un.s + un.j * kL, L = min(kL, un.e - t0);
  const size_t at = (size_t)(un.chunk + un.j) * a.G + grp;  // tile block
  const int part = lane >> 4, vec = lane & 15;              // 0: B, 1: C
  const bool live = vec * 8 < g.NS;
  const int c = a.H * a.P + (part * a.G + grp) * g.NS + vec * 8;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + c;
  const __nv_bfloat16* c0 = static_cast<const __nv_bfloat16*>(a.conv0);
  const int row = state_row(a.slot, un.n, a.num_slots);
  // the history the later kernels read: this group's share of the channels
  if (un.j == 0 && g.hist) {
    const int per = a.Cc / 8;
    for (int v = grp * 256 + tid; v < 3 * per; v += a.G * 256) {
      uint4 r = make_uint4(0, 0, 0, 0);
      if (c0 && row >= 0) r = reinterpret_cast<const uint4*>(c0 + (size_t)row * 3 * a.Cc)[v];
      reinterpret_cast<uint4*>(g.hist + (size_t)un.n * 3 * a.Cc)[v] = r;
    }
  }
  float w[4][8], b[8], h[3][8];
  if (live) load_taps<__nv_bfloat16>(a, c, w, b);
  const int i0 = warp * 16;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int t = t0 + i0 - 3 + j;
    const __nv_bfloat16* p = nullptr;
    if (live && i0 < L) {
      if (t >= un.s) p = x + (size_t)t * a.Cc;
      else if (c0 && row >= 0) p = c0 + ((size_t)row * 3 + 3 + t - un.s) * a.Cc + c;
    }
    load8_or_zero(p, h[j]);
  }
  uint8_t* tiles = g.tiles + at * kBcBytes;
  int8_t* ex = g.ex + at * 2 * kL;
  for (int q = 0; q < 16; ++q) {
    const int i = i0 + q;
    float v[8];
    const bool in = live && i < L;
    load8_or_zero(in ? x + (size_t)(t0 + i) * a.Cc : nullptr, v);
    float u[8];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s = 0.f;
      if (in)
        s = silu_div(fmaf(w[3][e], v[e],
                          fmaf(w[2][e], h[2][e], fmaf(w[1][e], h[1][e], fmaf(w[0][e], h[0][e], b[e])))));
      u[e] = s;
      top = max(top, __float_as_uint(s) & 0x7fffffffu);
      h[0][e] = h[1][e];
      h[1][e] = h[2][e];
      h[2][e] = v[e];
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e2 = exponent_of(top);
    const float sc = pow2(kTargetBC - e2);
    if (vec == 0) ex[part * kL + i] = (int8_t)e2;
    uint4 f;
    f.x = pack_f16x2(u[0] * sc, u[1] * sc);
    f.y = pack_f16x2(u[2] * sc, u[3] * sc);
    f.z = pack_f16x2(u[4] * sc, u[5] * sc);
    f.w = pack_f16x2(u[6] * sc, u[7] * sc);
    const uint32_t off = (vec >> 3) * kTileB + sw128_off(i, vec & 7);
    *reinterpret_cast<uint4*>(sm + part * 2 * kTileB + off) = f;
    if (part) {
      *reinterpret_cast<uint4*>(tiles + off) = f;
    } else {
      uint4 hi, lo;
      split2(make_float2(u[0], u[1]), hi.x, lo.x);
      split2(make_float2(u[2], u[3]), hi.y, lo.y);
      split2(make_float2(u[4], u[5]), hi.z, lo.z);
      split2(make_float2(u[6], u[7]), hi.w, lo.w);
      *reinterpret_cast<uint4*>(tiles + 2 * kTileB + off) = hi;
      *reinterpret_cast<uint4*>(tiles + 4 * kTileB + off) = lo;
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  if (tid == 0) {
    const uint32_t sB = smem_u32(sm), sC = sB + 2 * kTileB;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_bf16(tmem, desc_kmajor(sC, kk, kTileB), desc_kmajor(sB, kk, kTileB),
               idesc_f16(128, 128, false, false), kk > 0);
    mma_commit(bar);
  }
  __syncwarp();
  const bool ok = mbar_wait(bar, 0, g.wait_ns);
  tc_fence_after();
  if (!ok && tid == 0) report_status(a.status, GDN_ERR_TIMEOUT);
  // rows of the product: the blocks of 32 columns up to the diagonal
  const int i = (warp & 3) * 32 + lane;
  __half* cb = g.cb + (at * kL + i) * kL;
  for (int blk = warp >> 2; blk <= (warp & 3); blk += 2) {
    float v[32];
    tmem_ld32(tmem_at(tmem, (warp & 3) * 32, blk * 32), v);
    tmem_ld_wait();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 f;
      f.x = pack_f16x2(v[8 * q], v[8 * q + 1]);
      f.y = pack_f16x2(v[8 * q + 2], v[8 * q + 3]);
      f.z = pack_f16x2(v[8 * q + 4], v[8 * q + 5]);
      f.w = pack_f16x2(v[8 * q + 6], v[8 * q + 7]);
      *reinterpret_cast<uint4*>(cb + blk * 32 + 8 * q) = f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (!ok) mbar_wait(bar, 0, g.wait_ns);  // the product still in flight
    tmem_dealloc(tmem, 128);
  }
}

// -------------------------------------------------------------------- shared by seg and main
// One 64-channel slice of a head, worked on by a pipeline of 256 threads.
struct Slice {
  bool live;
  int h, c;        // head; first channel (of x and of the output)
  float rate2;     // log2(e) exp(a_log)
  float bias;
};
__device__ __forceinline__ Slice slice_of(const SsmTcArgs& g, int grp, int v, int slices) {
  const SsmArgs& a = g.a;
  Slice s;
  s.live = v < slices;
  const int blocks = a.P / 64;
  s.h = grp * (a.H / a.G) + (s.live ? v / blocks : 0);
  s.c = s.h * a.P + (s.live ? v % blocks : 0) * 64;
  s.rate2 = -1.4426950408889634f * expf(a.a_log[s.h]);
  s.bias = a.dt_bias ? a.dt_bias[s.h] : 0.f;
  return s;
}

__device__ __forceinline__ float load_dt(const SsmArgs& a, const Slice& s, int t0, int L, int i) {
  return i < L ? __ldg(a.dt + (size_t)(t0 + i) * a.H + s.h) : 0.f;
}
// Step of a token (0 behind the chunk's end) and log2 of its decay.  A decay below 2^-150 counts
// as 2^-150 (zero in fp32).
__device__ __forceinline__ float chunk_step(const SsmArgs& a, const Slice& s, float raw, bool in,
                                            double& la) {
  const float d = in ? ssm_step(raw + s.bias, a.dt_min, a.dt_max) : 0.f;
  la = (double)fmaxf(s.rate2 * d, -150.f);
  return d;
}
// 128 bytes towards L2, for the next chunk
__device__ __forceinline__ void prefetch_row(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ double warp_scan_add(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ double warp_scan_max(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = fmax(v, u);
  }
  return v;
}

// Conv + SiLU of a chunk's 64 channels.  Lane l has channels c + 2 l, c + 2 l + 1; warp w tokens
// 16 w .. 16 w + 15, walked with the three rows before them in registers; `put` gets token and
// value (zero behind the chunk's end).
template <typename Put>
__device__ __forceinline__ void conv_x(const SsmTcArgs& g, const Unit& un, const Slice& s, int t0,
                                       int L, int warp, int lane, Put&& put) {
  const SsmArgs& a = g.a;
  const int c = s.c + 2 * lane, i0 = warp * 16;
  const uint32_t* x = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.x) + c);
  const size_t pitch = (size_t)a.Cc / 2;
  const uint4 wr = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.conv_w) +
                                                   (size_t)c * 4);
  const float2 wa = unpack_bf16x2(wr.x), wb = unpack_bf16x2(wr.y);
  const float2 wc = unpack_bf16x2(wr.z), wd = unpack_bf16x2(wr.w);
  const float2 w0 = make_float2(wa.x, wc.x), w1 = make_float2(wa.y, wc.y);
  const float2 w2 = make_float2(wb.x, wd.x), w3 = make_float2(wb.y, wd.y);
  float2 b = make_float2(0.f, 0.f);
  if (a.conv_b)
    b = unpack_bf16x2(*reinterpret_cast<const uint32_t*>(
        static_cast<const __nv_bfloat16*>(a.conv_b) + c));
  uint32_t raw[19];
#pragma unroll
  for (int q = 0; q < 19; ++q) {
    const int i = i0 + q - 3, t = t0 + i;
    raw[q] = 0;
    if (i < L && i0 < L) {
      if (t >= un.s) raw[q] = __ldg(x + (size_t)t * pitch);
      else if (g.hist)
        raw[q] = *reinterpret_cast<const uint32_t*>(
            g.hist + ((size_t)un.n * 3 + 3 + t - un.s) * a.Cc + c);
    }
  }
  float2 h0 = unpack_bf16x2(raw[0]), h1 = unpack_bf16x2(raw[1]), h2 = unpack_bf16x2(raw[2]);
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const float2 v = unpack_bf16x2(raw[q + 3]);
    const float2 y = __ffma2_rn(w3, v, __ffma2_rn(w2, h2, __ffma2_rn(w1, h1, __ffma2_rn(w0, h0, b))));
    h0 = h1;
    h1 = h2;
    h2 = v;
    float2 u = make_float2(silu_div(y.x), silu_div(y.y));
    if (i0 + q >= L) u = make_float2(0.f, 0.f);
    put(i0 + q, u);
  }
}

// Byte offset of the channel pair of lane l in row i of a [128][64] row tile.
__device__ __forceinline__ uint32_t pair_off(int i, int lane) {
  return sw128_off(i, lane >> 2) + (lane & 3) * 4;
}

// B^T wX, what a chunk adds to S^T: three products of the bf16 parts (the fourth is below 2^-16 of the first).
__device__ __forceinline__ void mma_state(uint32_t tS, uint32_t sB, uint32_t sW) {
  constexpr uint32_t id = idesc_bf16(128, 64, true, true);
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t A = sB + (p == 1 ? 2 * kTileB : 0), W = sW + (p == 2 ? kTileB : 0);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_bf16(tS, desc_mnmajor(A, kk, kTileB), desc_mnmajor(W, kk, kTileB), id,
               p > 0 || kk > 0);
  }
}

// ------------------------------------------------------------------------------------ seg
// The state a segment adds, S_j = sum over its tokens of 2^(log decay from the token to the
// segment's end) delta x B^T (for the first segment: and the decayed initial state), chunk by
// chunk from its end: the decay to the end goes onto wX, the products only accumulate.
// smem: two stages of B (64 KB), one wX (32 KB) per pipeline, control.
constexpr uint32_t kSegW = 8 * kTileB, kSegCtl = kSegW + 4 * kTileB;
constexpr uint32_t kSegSmem = kSegCtl + 4096;

__global__ void __launch_bounds__(512, 1) ssm_seg_kernel(SsmTcArgs g) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const SsmArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_trigger();
  const int slices = (a.H / a.G) * (a.P / 64), pairs = (slices + 1) / 2;
  const int grp = (blockIdx.x % (a.G * pairs)) / pairs, pair = blockIdx.x % pairs;
  const Unit un = find_unit(a, g.seg * kL, true, blockIdx.x / (a.G * pairs),
                            gridDim.x / (a.G * pairs), sm);
  pdl_wait();  // before any return: the next kernel counts on this one having waited
  if (un.n < 0) return;
  const int total = (un.e - un.s + kL - 1) / kL;  // chunks of the sequence
  const int c0 = un.j * g.seg, c1 = c0 + g.seg;
  if (c1 >= total) return;  // no segment follows

  const int pipe = tid >> 8, pt = tid & 255, pw = pt >> 5;
  uint8_t* ctl = sm + kSegCtl;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctl);      // [2] B stages landed
  uint64_t* done = full + 2;                              // [2] a pipeline's products
  int* count = reinterpret_cast<int*>(ctl + 32);          // [2] uses of a stage, both pipelines
  int* loads = count + 2;                                 // [2] copies into it
  uint32_t* tslot = reinterpret_cast<uint32_t*>(ctl + 48);
  double* tot = reinterpret_cast<double*>(ctl + 64) + pipe * 4;
  float* w_s = reinterpret_cast<float*>(ctl + 256) + pipe * kL;
  if (tid == 0) {
    for (int k = 0; k < 4; ++k) {
      mbar_init(full + k, 1);
      count[k] = 0;  // and loads
    }
    fence_barrier_init();
  }
  if (tid < 32) tmem_alloc(tslot, 128);
  fence_proxy_async_smem();  // find_unit's scratch is overwritten by bulk copies
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = *tslot + pipe * 64;
  const Slice s = slice_of(g, grp, 2 * pair + pipe, slices);
  const int users = min(2, slices - 2 * pair);
  const int nch = c1 - c0;
  auto load_b = [&](int k) {  // k-th chunk from the end
    const size_t at = (size_t)(un.chunk + c1 - 1 - k) * a.G + grp;
    mbar_arrive_expect_tx(full + (k & 1), 4 * kTileB);
    bulk_load(sm + (k & 1) * 4 * kTileB, g.tiles + at * kBcBytes + 2 * kTileB, 4 * kTileB,
              full + (k & 1));
    loads[k & 1]++;
  };
  if (tid == 0) {
    load_b(0);
    if (nch > 1) load_b(1);
  }
  float v[32];  // row n = lane of the state, 32 of the slice's channels
#pragma unroll
  for (int q = 0; q < 32; ++q) v[q] = 0.f;
  double R = 0.0;  // log2 decay of the chunks behind the current one
  bool ok = true;
  int mmas = 0;
  uint8_t* W = sm + kSegW + pipe * 2 * kTileB;
  // adds the products of chunk k (they have read wX and the stage then); the last pipeline
  // through with a stage fetches the next chunk but one into it
  auto take = [&](int k) {
    ok = mbar_wait(done + pipe, k & 1, g.wait_ns) && ok;
    tc_fence_after();
    if (pt == 0 && ok) {
      __threadfence_block();
      if (atomicAdd(count + (k & 1), 1) == users * ((k >> 1) + 1) - 1 && k + 2 < nch) {
        __threadfence_block();
        load_b(k + 2);
      }
    }
    __syncwarp();
    float u[32];
    tmem_ld32(tmem_at(tS, (pw & 3) * 32, (pw >> 2) * 32), u);
    tmem_ld_wait();
    tc_fence_before();
#pragma unroll
    for (int q = 0; q < 32; ++q) v[q] += u[q];
  };
  if (s.live) {
    const int i = pt & 127;
    float raw = load_dt(a, s, un.s + (c1 - 1) * kL, kL, i);
    for (int k = 0; k < nch; ++k) {
      const int t0 = un.s + (c1 - 1 - k) * kL;
      double la;
      const float d = chunk_step(a, s, raw, i < kL, la);
      if (k + 1 < nch) {
        raw = load_dt(a, s, t0 - kL, kL, i);
        if (pt < 128) prefetch_row(static_cast<const __nv_bfloat16*>(a.x) +
                                   (size_t)(t0 - kL + i) * a.Cc + s.c);
      }
      double cum = warp_scan_add(la, lane);
      if (pt < 128 && lane == 31) tot[pw] = cum;
      if (bar_or_n(1 + pipe, kPipe, !ok)) break;
      double all = 0.0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q < (i >> 5)) cum += tot[q];
        all += tot[q];
      }
      if (pt < 128) w_s[i] = d * exp2f((float)(R + all - cum));
      R += all;
      if (k > 0) take(k - 1);
      bar_sync_n(1 + pipe, kPipe);
      conv_x(g, un, s, t0, kL, pw, lane, [&](int q, float2 u) {
        const float wq = w_s[q];
        uint32_t hi, lo;
        split2(make_float2(u.x * wq, u.y * wq), hi, lo);
        const uint32_t off = pair_off(q, lane);
        *reinterpret_cast<uint32_t*>(W + off) = hi;
        *reinterpret_cast<uint32_t*>(W + kTileB + off) = lo;
      });
      fence_proxy_async_smem();
      bar_sync_n(1 + pipe, kPipe);
      if (pt == 0) {
        const bool got = mbar_wait(full + (k & 1), (k >> 1) & 1, g.wait_ns);
        tc_fence_after();
        if (got) {
          mma_state(tS, smem_u32(sm + (k & 1) * 4 * kTileB), smem_u32(W));
          mma_commit(done + pipe);
          ++mmas;
        }
        ok = ok && got;
      }
      __syncwarp();
    }
    if (bar_or_n(1 + pipe, kPipe, !ok)) ok = false;
    if (ok) take(nch - 1);
    if (ok) {
      // [p][n] fp32, like the caller's states; lane = n
      const int n = (pw & 3) * 32 + lane, p0 = (pw >> 2) * 32;
      if (n < g.NS) {
        const size_t base = (size_t)(s.c + p0) * g.NS + n;
        const size_t pitch = (size_t)a.H * a.P * g.NS;
        float* out = g.seg_state + (size_t)(un.first + un.j) * pitch + base;
        const int row = state_row(a.slot, un.n, a.num_slots);
        if (un.j == 0) {
          // with the initial state, which is also kept for the first segment (in the place of
          // the last one): the final state may overwrite it
          const float* S0 = a.S0 && row >= 0
                                ? static_cast<const float*>(a.S0) + (size_t)row * pitch + base
                                : nullptr;
          float* keep = g.seg_state + (size_t)(un.first + (total - 1) / g.seg) * pitch + base;
          const float dec = exp2f((float)R);
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const float s0 = S0 ? S0[(size_t)q * g.NS] : 0.f;
            keep[(size_t)q * g.NS] = s0;
            v[q] = fmaf(dec, s0, v[q]);
          }
        }
#pragma unroll
        for (int q = 0; q < 32; ++q) out[(size_t)q * g.NS] = v[q];
      }
      if (pt == 0 && s.c % a.P == 0) g.seg_decay[(size_t)(un.first + un.j) * a.H + s.h] = R;
    }
    if (!ok && pt == 0) {
      report_status(a.status, GDN_ERR_TIMEOUT);
      if (mmas > 0) mbar_wait(done + pipe, (mmas - 1) & 1, g.wait_ns);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0)  // copies in flight, after a wait that ran out
    for (int k = 0; k < 2; ++k)
      if (loads[k] > 0) mbar_wait(full + k, (loads[k] - 1) & 1, g.wait_ns);
  if (tid < 32) tmem_dealloc(*tslot, 128);
}

// ----------------------------------------------------------------------------------- main
// smem: C^ | B high | B low (96 KB, shared by both pipelines), then per pipeline X^ | wX high |
// wX low | S^ (64 KB), and 3 KB of control: with no more to be had, the base has to be aligned.
// TMEM, per pipeline: what the chunk adds to S^T (64 columns), C S^T and P X (128), P (64).  S^T
// itself stays in registers (32 of a row per thread): fp32 sums there round to nearest.
constexpr uint32_t kMainPipe = 6 * kTileB, kMainCtl = kMainPipe + 8 * kTileB;
constexpr uint32_t kMainSmem = kMainCtl + 3072;

__global__ void __launch_bounds__(512, 1) ssm_main_kernel(SsmTcArgs g) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const SsmArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_trigger();
  const int slices = (a.H / a.G) * (a.P / 64), pairs = (slices + 1) / 2;
  const int grp = (blockIdx.x % (a.G * pairs)) / pairs, pair = blockIdx.x % pairs;
  const Unit un = find_unit(a, g.seg * kL, true, blockIdx.x / (a.G * pairs),
                            gridDim.x / (a.G * pairs), sm);
  if (un.n < 0) {
    pdl_wait();
    return;
  }
  const int pipe = tid >> 8, pt = tid & 255, pw = pt >> 5;
  uint8_t* ctl = sm + kMainCtl;
  uint64_t* c_full = reinterpret_cast<uint64_t*>(ctl);
  uint64_t* b_full = c_full + 1;
  uint64_t* done = c_full + 2;  // [2] a pipeline's products of a chunk
  int* count = reinterpret_cast<int*>(ctl + 32);  // chunks finished, over both pipelines
  int* loads = count + 1;                         // chunks whose tiles were fetched
  uint32_t* tslot = reinterpret_cast<uint32_t*>(ctl + 40);
  uint8_t* mine = ctl + 64 + pipe * 1408;
  double* tot = reinterpret_cast<double*>(mine);           // [4] sums of la over 32 tokens
  double* ref_s = tot + 4;                                 // [4] maxima of g over them
  uint32_t* top_s = reinterpret_cast<uint32_t*>(mine + 64);  // [8]
  float* wf_s = reinterpret_cast<float*>(mine + 128);      // [128] weights of wX, then F
  float* g_s = wf_s + kL;                                  // [128]
  int8_t* ex_s = reinterpret_cast<int8_t*>(g_s + kL);      // [128]
  if (tid == 0) {
    for (int k = 0; k < 4; ++k) mbar_init(c_full + k, 1);
    *count = *loads = 0;
    fence_barrier_init();
  }
  if (tid < 32) tmem_alloc(tslot, 512);
  fence_proxy_async_smem();  // find_unit's scratch is overwritten by bulk copies
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tS = tmem + pipe * 64, tI = tmem + 128 + pipe * 128, tX = tI + 64;
  const uint32_t tP = tmem + 384 + pipe * 64;
  const Slice s = slice_of(g, grp, 2 * pair + pipe, slices);
  const int users = min(2, slices - 2 * pair);
  const int total = (un.e - un.s + kL - 1) / kL;
  const int c0 = un.j * g.seg, c1 = min(total, c0 + g.seg), nch = c1 - c0;
  const int row = state_row(a.slot, un.n, a.num_slots);
  if (row < 0 && tid == 0) report_status(a.status, GDN_ERR_INVALID_ARG);
  const float D = a.D ? a.D[s.h] : 0.f;
  const int quad = pw & 3, half = pw >> 2;
  const int i = quad * 32 + lane;   // row of this thread: token of the chunk, or n of the state
  const int p0 = half * 32;         // its channels
  const size_t pitch = (size_t)a.H * a.P * g.NS, sbase = (size_t)(s.c + p0) * g.NS + i;
  pdl_wait();
  auto load_tiles = [&](int c) {
    const uint8_t* src = g.tiles + ((size_t)(un.chunk + c) * a.G + grp) * kBcBytes;
    mbar_arrive_expect_tx(c_full, 2 * kTileB);
    bulk_load(sm, src, 2 * kTileB, c_full);
    mbar_arrive_expect_tx(b_full, 4 * kTileB);
    bulk_load(sm + 2 * kTileB, src + 2 * kTileB, 4 * kTileB, b_full);
    ++*loads;
  };
  if (tid == 0 && nch > 0) load_tiles(c0);

  // ---- the state that enters (row i of S^T, this thread's channels)
  float sv[32];
#pragma unroll
  for (int q = 0; q < 32; ++q) sv[q] = 0.f;
  {
    if (s.live && i < g.NS) {
      if (un.j == 0) {
        const float* S0 = total > g.seg
                              ? g.seg_state + (size_t)(un.first + (total - 1) / g.seg) * pitch
                              : (a.S0 && row >= 0
                                     ? static_cast<const float*>(a.S0) + (size_t)row * pitch
                                     : nullptr);
        if (S0) {
#pragma unroll
          for (int q = 0; q < 32; ++q) sv[q] = S0[sbase + (size_t)q * g.NS];
        }
      } else {
        for (int j = 0; j < un.j; ++j) {
          const float* S = g.seg_state + (size_t)(un.first + j) * pitch + sbase;
          const float dec = exp2f((float)g.seg_decay[(size_t)(un.first + j) * a.H + s.h]);
#pragma unroll
          for (int q = 0; q < 32; ++q) sv[q] = fmaf(dec, sv[q], S[(size_t)q * g.NS]);
        }
      }
    }
    // P above the diagonal blocks is zero throughout
    float zero[32];
#pragma unroll
    for (int q = 0; q < 32; ++q) zero[q] = 0.f;
    tmem_st32(tmem_at(tP, quad * 32, half * 32), zero);
    tmem_st_wait();
  }
  uint8_t* X = sm + kMainPipe + pipe * 4 * kTileB;
  uint8_t* W = X + kTileB;
  uint8_t* S16 = X + 3 * kTileB;
  bool ok = true;
  int mmas = 0;
  if (s.live) {
    float raw = nch > 0 ? load_dt(a, s, un.s + c0 * kL, un.e - un.s - c0 * kL, i) : 0.f;
    for (int k = 0; k < nch; ++k) {
      const int t0 = un.s + (c0 + k) * kL, L = min(kL, un.e - t0);
      const size_t at = (size_t)(un.chunk + c0 + k) * a.G + grp;
      // ---- steps and decays of the chunk's tokens (thread i: token i)
      double la;
      const float d = chunk_step(a, s, raw, i < L, la);
      if (k + 1 < nch) {  // the next chunk's inputs on their way
        const int t1 = t0 + kL;
        raw = load_dt(a, s, t1, un.e - t1, i);
        if (t1 + i < un.e) {
          if (half == 0)
            prefetch_row(static_cast<const __nv_bfloat16*>(a.x) + (size_t)(t1 + i) * a.Cc + s.c);
          else if (a.z)
            prefetch_row(static_cast<const __nv_bfloat16*>(a.z) + (size_t)(t1 + i) * a.H * a.P +
                         s.c);
        }
      }
      double cum = warp_scan_add(la, lane);
      if (pt < 128 && lane == 31) tot[quad] = cum;
      // ---- S^T: its largest magnitude
      uint32_t top = 0;
#pragma unroll
      for (int q = 0; q < 32; ++q) top = max(top, __float_as_uint(sv[q]) & 0x7fffffffu);
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) top_s[pw] = top;
      tc_fence_before();
      if (bar_or_n(1 + pipe, kPipe, !ok)) break;
      double all = 0.0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q < quad) cum += tot[q];
        all += tot[q];
      }
      if (half == 0) wf_s[i] = d * exp2f((float)(all - cum));
#pragma unroll
      for (int q = 0; q < 8; ++q) top = max(top, top_s[q]);
      const int eS = exponent_of(top);
      // ---- S^ = fp16 operand of C S^T
      {
        const float sc = pow2(kTargetS - eS);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 f;
          f.x = pack_f16x2(sv[8 * q] * sc, sv[8 * q + 1] * sc);
          f.y = pack_f16x2(sv[8 * q + 2] * sc, sv[8 * q + 3] * sc);
          f.z = pack_f16x2(sv[8 * q + 4] * sc, sv[8 * q + 5] * sc);
          f.w = pack_f16x2(sv[8 * q + 6] * sc, sv[8 * q + 7] * sc);
          *reinterpret_cast<uint4*>(S16 + sw128_off(i, half * 4 + q)) = f;
        }
      }
      bar_sync_n(1 + pipe, kPipe);  // the weights
      // ---- X^ and wX
      conv_x(g, un, s, t0, L, pw, lane, [&](int q, float2 u) {
        const uint32_t m = __reduce_max_sync(
            0xffffffffu,
            max(__float_as_uint(u.x) & 0x7fffffffu, __float_as_uint(u.y) & 0x7fffffffu));
        const int e = exponent_of(m);
        if (lane == 0) ex_s[q] = (int8_t)e;
        const float sc = pow2(kTargetX - e), wq = wf_s[q];
        uint32_t hi, lo;
        split2(make_float2(u.x * wq, u.y * wq), hi, lo);
        const uint32_t off = pair_off(q, lane);
        *reinterpret_cast<uint32_t*>(X + off) = pack_f16x2(u.x * sc, u.y * sc);
        *reinterpret_cast<uint32_t*>(W + off) = hi;
        *reinterpret_cast<uint32_t*>(W + kTileB + off) = lo;
      });
      fence_proxy_async_smem();
      tc_fence_before();
      bar_sync_n(1 + pipe, kPipe);
      if (pt == 0) {
        const bool got = mbar_wait(c_full, k & 1, g.wait_ns) && mbar_wait(b_full, k & 1, g.wait_ns);
        tc_fence_after();
        if (got) {
          const uint32_t sC = smem_u32(sm), sS = smem_u32(S16);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16(tI, desc_kmajor(sC, kk, kTileB), desc_mnmajor(sS, kk, kTileB),
                     idesc_f16(128, 64, false, true), kk > 0);
          mma_state(tS, sC + 2 * kTileB, smem_u32(W));
        }
        ok = ok && got;
      }
      __syncwarp();
      // ---- weights of P: g, its running maximum, the factors of whole blocks
      const int8_t* ex = g.ex + at * 2 * kL;
      const float eC = (float)__ldg(ex + kL + i);
      const float lf = fmaxf(log2f(d), -1000.f) + (float)ex_s[i] + (float)__ldg(ex + i);
      const double gi = (double)lf - cum;
      double pm = warp_scan_max(gi, lane);
      if (half == 0 && lane == 31) ref_s[quad] = pm;
      bar_sync_n(1 + pipe, kPipe);
      double ref[4];
      ref[0] = ref_s[0];
#pragma unroll
      for (int q = 1; q < 4; ++q) ref[q] = fmax(ref[q - 1], ref_s[q]);
      double mine_ref = ref[0];
#pragma unroll
      for (int q = 1; q < 4; ++q) {
        if (q == quad) {
          pm = fmax(pm, ref[q - 1]);
          mine_ref = ref[q];
        }
      }
      if (half == 0) {
        g_s[i] = (float)(gi - mine_ref);
        wf_s[i] = exp2f((float)(gi - mine_ref));
      }
      bar_sync_n(1 + pipe, kPipe);
      // ---- P^ (fp16) into TMEM, block by block; this thread has 16 of each block's 32 columns
      {
        const __half* cb = g.cb + (at * kL + i) * kL + half * 16;
        const float pmd = (float)(pm - mine_ref);
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) {
          if (blk > quad) break;
          const uint4 r0 = __ldg(reinterpret_cast<const uint4*>(cb + blk * 32));
          const uint4 r1 = __ldg(reinterpret_cast<const uint4*>(cb + blk * 32 + 8));
          const uint32_t raw[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
          uint32_t out[8];
          const int j0 = blk * 32 + half * 16;
          const float rf = blk < quad ? exp2f((float)(ref[blk] - pm)) : 0.f;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&raw[q]));
            const int j = j0 + 2 * q;
            float2 f;
            if (blk < quad) {
              f = *reinterpret_cast<const float2*>(wf_s + j);
              f.x *= rf;
              f.y *= rf;
            } else {
              const float2 e = *reinterpret_cast<const float2*>(g_s + j);
              f.x = j <= i ? exp2f(fminf(e.x - pmd, 0.f)) : 0.f;
              f.y = j + 1 <= i ? exp2f(fminf(e.y - pmd, 0.f)) : 0.f;
            }
            out[q] = pack_f16x2(j <= i ? v.x * f.x : 0.f, j + 1 <= i ? v.y * f.y : 0.f);
          }
          tmem_st8(tmem_at(tP, quad * 32, j0 / 2), out);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      bar_sync_n(1 + pipe, kPipe);
      if (pt == 0 && ok) {
        tc_fence_after();
        const uint32_t sX = smem_u32(X);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tX, tP + kk * 8, desc_mnmajor(sX, kk, kTileB), idesc_f16(128, 64, false, true),
                 kk > 0);
        mma_commit(done + pipe);
        ++mmas;
      }
      __syncwarp();
      // ---- outputs
      const bool in = i < L;
      const size_t o_at = ((size_t)(t0 + i) * a.H) * a.P + s.c + p0;
      uint4 zr[4];
      if (a.z && in) {
        const uint4* zp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.z) + o_at);
#pragma unroll
        for (int q = 0; q < 4; ++q) zr[q] = __ldg(zp + q);
      }
      ok = mbar_wait(done + pipe, k & 1, g.wait_ns) && ok;
      tc_fence_after();
      if (pt == 0 && ok) {  // the last pipeline through with the tiles fetches the next ones
        __threadfence_block();
        if (atomicAdd(count, 1) == users * (k + 1) - 1 && k + 1 < nch) {
          __threadfence_block();
          load_tiles(c0 + k + 1);
        }
      }
      __syncwarp();
      const float si = exp2f((float)cum + eC + (float)(eS - kTargetS - kTargetBC));
      const float sx = exp2f((float)(cum + pm) + eC - (float)(2 * kTargetBC + kTargetX));
      const float dx = D * pow2((int)ex_s[i] - kTargetX), dec = exp2f((float)all);
      __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + o_at;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float yi[16], yx[16];
        tmem_ld16(tmem_at(tI, quad * 32, p0 + 16 * r), yi);
        tmem_ld16(tmem_at(tX, quad * 32, p0 + 16 * r), yx);
        tmem_ld_wait();
        if (in) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint4 xr = *reinterpret_cast<const uint4*>(X + sw128_off(i, half * 4 + 2 * r + q));
            const uint32_t xw[4] = {xr.x, xr.y, xr.z, xr.w};
            const uint4 zv = zr[2 * r + q];
            const uint32_t zw[4] = {zv.x, zv.y, zv.z, zv.w};
            uint32_t ow[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int m = 8 * q + 2 * e;
              const float2 xf = __half22float2(*reinterpret_cast<const __half2*>(&xw[e]));
              float2 y;
              y.x = fmaf(si, yi[m], fmaf(sx, yx[m], dx * xf.x));
              y.y = fmaf(si, yi[m + 1], fmaf(sx, yx[m + 1], dx * xf.y));
              if (a.z) {
                const float2 zf = unpack_bf16x2(zw[e]);
                y.x *= silu_div(zf.x);
                y.y *= silu_div(zf.y);
              }
              ow[e] = pack_bf16x2(y.x, y.y);
            }
            *reinterpret_cast<uint4*>(op + 16 * r + 8 * q) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
          }
        }
        // ---- S^T <- 2^cum_L S^T + what the chunk adds
        float ds[16];
        tmem_ld16(tmem_at(tS, quad * 32, p0 + 16 * r), ds);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 16; ++q) sv[16 * r + q] = fmaf(dec, sv[16 * r + q], ds[q]);
      }
      tc_fence_before();
    }
    if (bar_or_n(1 + pipe, kPipe, !ok)) ok = false;
    // ---- the state behind the sequence
    if (ok && c1 == total && a.SN && row >= 0 && i < g.NS) {
      float* SN = static_cast<float*>(a.SN) + (size_t)row * pitch + sbase;
#pragma unroll
      for (int q = 0; q < 32; ++q) SN[(size_t)q * g.NS] = sv[q];
    }
    if (!ok && pt == 0) {
      report_status(a.status, GDN_ERR_TIMEOUT);
      if (mmas > 0) mbar_wait(done + pipe, (mmas - 1) & 1, g.wait_ns);
    }
  }
  if (c1 == total)
    conv_history<__nv_bfloat16>(a, un.n, row, un.s, un.e, blockIdx.x % (a.G * pairs), a.G * pairs);
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *loads > 0) {  // copies in flight, after a wait that ran out
    mbar_wait(c_full, (*loads - 1) & 1, g.wait_ns);
    mbar_wait(b_full, (*loads - 1) & 1, g.wait_ns);
  }
  if (tid < 32) tmem_dealloc(tmem, 512);
}

}  // namespace gdn

namespace gdn_host {

cudaError_t launch_ssm_tc(gdn::SsmTcArgs g, void* workspace, cudaStream_t s);
size_t ssm_tc_workspace(int N, int T, int H, int G, int P, int NS, int Cc);

namespace {

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Chunks per segment.  A CTA works on 128 channels of one segment, so a call has pairs x units
// CTAs, one per SM; the units are chosen so that they fill whole waves of the GPU, with the least
// total of chunks one after the other.
int ssm_segment(int N, int T, int pairs) {
  constexpr int kSms = 148;
  const int chunks = std::max(1, T / gdn::kL + N);
  int best = chunks, cost = INT32_MAX;
  for (int waves = 1; waves <= 4; ++waves) {
    const int units = kSms * waves / pairs;
    if (units < 1) continue;
    const int seg = (chunks + units - 1) / units;
    if (seg * waves < cost) {
      cost = seg * waves;
      best = seg;
    }
  }
  return best;
}

struct TcLayout {
  int seg, units;
  size_t tiles, cb, ex, hist, state, decay, total;
};

TcLayout tc_layout(int N, int T, int H, int G, int P, int NS, int Cc) {
  TcLayout l{};
  const int pairs = G * (((H / G) * (P / 64) + 1) / 2);
  const size_t blocks = ((size_t)T / gdn::kL + N) * G;
  l.seg = ssm_segment(N, T, pairs);
  l.units = T / (l.seg * gdn::kL) + N;
  size_t o = 0;
  l.tiles = o; o = up256(o + blocks * gdn::kBcBytes);
  l.cb = o; o = up256(o + blocks * gdn::kL * gdn::kL * 2);
  l.ex = o; o = up256(o + blocks * 2 * gdn::kL);
  l.hist = o; o = up256(o + (size_t)N * 3 * Cc * 2);
  l.state = o; o = up256(o + (size_t)l.units * H * P * NS * 4);
  l.decay = o; o = up256(o + (size_t)l.units * H * 8);
  l.total = o;
  return l;
}

cudaError_t launch_tc(bool pdl, void (*kern)(gdn::SsmTcArgs), unsigned grid, unsigned block,
                      size_t smem, cudaStream_t s, const gdn::SsmTcArgs& g, const char* name) {
  // per call, not once: the attribute belongs to the current device
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (pdl && !trace_attached()) ? 1 : 0;
  trace_begin(name, s);
  e = cudaLaunchKernelEx(&cfg, kern, g);
  trace_end(s);
  return e;
}

}  // namespace

size_t ssm_tc_workspace(int N, int T, int H, int G, int P, int NS, int Cc) {
  return tc_layout(N, T, H, G, P, NS, Cc).total;
}

cudaError_t launch_ssm_tc(gdn::SsmTcArgs g, void* workspace, cudaStream_t s) {
  const gdn::SsmArgs& a = g.a;
  const TcLayout l = tc_layout(a.N, a.T, a.H, a.G, a.P, g.NS, a.Cc);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  g.tiles = w + l.tiles;
  g.cb = reinterpret_cast<__half*>(w + l.cb);
  g.ex = reinterpret_cast<int8_t*>(w + l.ex);
  g.hist = a.conv0 ? reinterpret_cast<__nv_bfloat16*>(w + l.hist) : nullptr;
  g.seg_state = reinterpret_cast<float*>(w + l.state);
  g.seg_decay = reinterpret_cast<double*>(w + l.decay);
  g.seg = l.seg;
  g.wait_ns = debug_opts().wait_limit_us ? (uint64_t)debug_opts().wait_limit_us * 1000ull
                                         : gdn::kWaitLimitNs;
  const unsigned pairs = a.G * (((a.H / a.G) * (a.P / 64) + 1) / 2);
  cudaError_t e = launch_tc(false, gdn::ssm_bc_kernel, (unsigned)(a.T / gdn::kL + a.N) * a.G, 256,
                            gdn::kBcSmem, s, g, "ssm_bc");
  if (e == cudaSuccess && a.T > l.seg * gdn::kL)  // a sequence may have several segments
    e = launch_tc(true, gdn::ssm_seg_kernel, (unsigned)l.units * pairs, 512, gdn::kSegSmem, s, g,
                  "ssm_seg");
  if (e == cudaSuccess)
    e = launch_tc(true, gdn::ssm_main_kernel, (unsigned)l.units * pairs, 512, gdn::kMainSmem, s, g,
                  "ssm_main");
  return e;
}

}  // namespace gdn_host
