// ssm_tc.cu -- packed prefill of the selective state space layer on tcgen05 tensor cores (bf16
// activations, fp32 state), in chunks of 128 tokens.
//
// With cum_i the running log2 of the decay inside a chunk, delta the steps, u the conv outputs:
//   Y    = diag(2^cum) C S^T + P X,   P_ij = 2^(cum_i - cum_j) delta_j C_i.B_j  (j <= i)
//   S^T <- 2^cum_L S^T + B^T diag(w) X,   w_j = 2^(cum_L - cum_j) delta_j
// Precision.  All products take fp16 operands (11 bits) and sum in fp32.  Outputs are rounded to
// bf16, so what forms them is rounded to fp16 wherever it becomes an operand or is stored: C, B, C B^T,
// P, X for P X, C and S for C S^T, X for D X.  The state is returned in fp32, so its update keeps both
// factors in two fp16 parts (three products; what is left out is 2^-22 of them).  fp16 has few exponent
// bits: rows of C, B and X are scaled by a power of two each (exponent from the row's largest value), S
// and wX by one per chunk, and P by the row's largest weight.  Nothing overflows then.  What underflows
// is small beside the largest value of its scale: 2^-28 of it for C, 2^-38 for B and X, 2^-30 for a
// token's share of P X beside the largest token's (fp32 weights; the sums of gdn.h).  It may still be
// all that a channel has: 64 channels of X share a scale.  With the exponents eX, eB of
// rows of X and B: g_j = log2(delta_j) - cum_j + eX_j + eB_j, pm_i = max over j <= i of g_j,
//   P^_ij = (C^_i.B^_j) 2^(g_j - pm_i)
// (never above the product), and row i of the result counts 2^(cum_i + pm_i + exponent of C_i).
// Non-finite values.  Zero weights would not remove them, and as a row's largest value they would
// scale its other values away.  So a row of X that holds one counts as zero in X^, and the token's
// weights in P and wX as NaN: the 64 channels of such a token are NaN from it on, what came before
// stays.  A row of B that holds one is NaN throughout; C only concerns its own token.
//
// Kernels (programmatic dependent launch between them):
//   bc    per (chunk, group): conv of B and C; the operand tiles C^ and B (two parts) in the
//         swizzled layout the products read, and C^ B^^T (tcgen05) as fp16.  Further CTAs per
//         (chunk, 32 heads): steps, decays (summed in fp64) and weights of the chunk's tokens.
//         The initial conv history is copied, so that the final one may overwrite it.
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
constexpr int kTok = 16;                   // tokens per warp (8 warps a pipeline)

// idesc of idesc_bf16 with fp16 operands (format fields 0)
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_bf16(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}
// tcgen05.mma issued by the lane with `lead` of a whole warp that runs this code together.
// Operands by the low words of their descriptors (address and LBO); the high words (SBO, version,
// swizzle) are the same for all.  ss: both operands in shared memory; ts: A in TMEM (row i in lane
// i, two fp16 per 32-bit column).
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo_bytes >> 4) << 16);
}
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (kLayoutSW128 << 29);
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint32_t a_low,
                                       uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %6};\n\t"
      "mov.b64 db, {%2, %6};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(lead), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem,
                                       uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %6};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(lead), "n"(kDescHigh)
      : "memory");
}
// Bounded wait for phase `parity` of `bar`; a try sleeps in hardware up to 20 us before it returns
// (polling threads would take issue slots from the others).
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  uint64_t t0 = 0;
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000)
        : "memory");
    if (done) return true;
    const uint64_t t = global_timer_ns();
    if (t0 == 0) t0 = t;
    else if (t - t0 > limit_ns) return false;
  }
}
// Read-only loads that stay where they are written: the compiler would move them up, or out of the
// chunk loop, and spill (with 227 KB of shared memory the L1 cache holds no spills).
__device__ __forceinline__ uint32_t ldg32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float ldgf(const float* p) { return __uint_as_float(ldg32(p)); }
__device__ __forceinline__ int ldg8(const int8_t* p) {
  int v;
  asm volatile("ld.global.nc.s8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ldg128(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float4 ldgf4(const void* p) {
  const uint4 v = ldg128(p);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                     __uint_as_float(v.w));
}
// The same value in every lane, in a uniform register (the reduction's result is one): the chunk
// loops keep their indices there and all vector registers for data.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Arrive at named barrier `id` of n threads without waiting.
__device__ __forceinline__ void bar_arrive_n(int id, int n) {
  asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// One instruction each; results below 2^-126 are zero.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}
__device__ __forceinline__ uint32_t pack_f16x2(float2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 mul2(float2 v, float s) {
  return __fmul2_rn(v, make_float2(s, s));
}
// v = high part + low part, both fp16 (half a step each)
__device__ __forceinline__ void split2(float2 v, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2(v);
  const float2 h = unpack_f16x2(hi);
  lo = pack_f16x2(__ffma2_rn(h, make_float2(-1.f, -1.f), v));
}
// silu of two values, x / (1 + exp(-x)): relative precision down to where the reciprocal underflows
// (-87), zero behind it.  (One reciprocal for both divisors would save a special-function result,
// but has to bound the exponents and takes three instructions more: 40,677 tokens in eight
// sequences 848 us so, 837 with two.)
__device__ __forceinline__ float2 silu2(float2 x) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float2 v = mul2(x, -kLog2e);
  const float2 d = __fadd2_rn(make_float2(ex2(v.x), ex2(v.y)), make_float2(1.f, 1.f));
  return __fmul2_rn(x, make_float2(rcp(d.x), rcp(d.y)));
}

// Exponent of the largest magnitude of a row (its bits), within [-100, 127], or 128 for a row that
// holds an infinity or NaN (kept as the int8 -128); the row is scaled by pow2(target - exponent).
constexpr int kNotFinite = 128;
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ int exponent_of(uint32_t bits) {
  return max((int)(bits >> 23) - 127, -100);
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }
// v 2^e for any e a call can form
__device__ __forceinline__ float scale2(float v, int e) {
  const int h = max(min(e, 250), -250) >> 1;
  return v * pow2(h) * pow2(max(min(e, 250), -250) - h);
}
constexpr int kTargetC = 3;    // C below 2^4
constexpr int kTargetB = 13;   // B below 2^14: C B^T below 2^25, kept as fp16 scaled by 2^-10
constexpr int kScaleCB = -10;
constexpr int kTargetX = 13;
constexpr int kTargetS = 14;
constexpr int kTargetW = 12;   // wX below 2^14 (two factors, each below 2 of its exponent)

// Unit k of the packed batch: sequences cut into units of `tokens`, numbered sequence by
// sequence.  A sequence without tokens has no chunk (kChunks) but one segment (kSegments: its state
// is written too); kFollowed numbers the segments that another one follows, one fewer than a
// sequence's segments, so that a batch of short sequences starts no CTA for them (96 sequences, 24
// heads of 64: a call 169 -> 148 us when it came in).  Every warp finds its unit by itself, 128
// sequences at a time (4 per lane).  `most_units`: units the launch has room for.
enum UnitKind { kChunks, kSegments, kFollowed };
struct Unit {
  int n;        // sequence, or -1: no such unit
  int j;        // unit inside the sequence
  int s, e;     // its sequence's tokens
  int chunk;    // first chunk of the sequence
  int first;    // first segment of the sequence (kChunks: first chunk)
};
__device__ __forceinline__ Unit find_unit(const SsmArgs& a, int tokens, UnitKind kind, int k,
                                          int most_units) {
  const int lane = threadIdx.x & 31;
  const int64_t most = (int64_t)a.T / kL + a.N;  // chunks the workspace holds
  Unit r{-1, 0, 0, 0, 0, 0};
  int64_t u0 = 0, c0 = 0;
  for (int base = 0; base < a.N && u0 <= k; base += 128) {
    int s[4], e[4];
    uint32_t nu[4], nc[4], us = 0, cs = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = base + 4 * lane + q;
      s[q] = e[q] = 0;
      if (n < a.N) seq_range(a, n, s[q], e[q]);
      nc[q] = (uint32_t)(e[q] - s[q] + kL - 1) / kL;
      const uint32_t followed = ((uint32_t)max(e[q] - s[q], 1) - 1) / (uint32_t)tokens;
      nu[q] = n >= a.N             ? 0u
              : kind == kSegments  ? followed + 1
              : kind == kFollowed  ? followed
                                   : (uint32_t)(e[q] - s[q] + tokens - 1) / (uint32_t)tokens;
      us += nu[q];
      cs += nc[q];
    }
    uint32_t ui = us, ci = cs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t uu = __shfl_up_sync(0xffffffffu, ui, o);
      const uint32_t cc = __shfl_up_sync(0xffffffffu, ci, o);
      if (lane >= o) {
        ui += uu;
        ci += cc;
      }
    }
    int64_t uf = u0 + ui - us, cf = c0 + ci - cs;
    bool mine = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (k >= uf && k < uf + nu[q]) {
        mine = true;
        const int n = base + 4 * lane + q;
        r = Unit{n, (int)(k - uf), s[q], e[q], (int)cf, (int)uf + (kind == kFollowed ? n : 0)};
        if (cf + nc[q] > most || uf + nu[q] > most_units) {
          // sequences that overlap: no room for this one, it counts as empty
          report_status(a.status, GDN_ERR_INVALID_ARG);
          r.e = r.s;
          if (r.j > 0 || kind != kSegments) r.n = -1;
        }
      }
      uf += nu[q];
      cf += nc[q];
    }
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    if (who) {
      const int l = __ffs(who) - 1;
      const bool it = lane == l;
      return Unit{uniform(it ? r.n : -1), uniform(it ? r.j : 0),     uniform(it ? r.s : 0),
                  uniform(it ? r.e : 0),  uniform(it ? r.chunk : 0), uniform(it ? r.first : 0)};
    }
    u0 += __shfl_sync(0xffffffffu, ui, 31);
    c0 += __shfl_sync(0xffffffffu, ci, 31);
  }
  return r;
}

// find_unit for up to 32 sequences (one per lane) with the units in descending order of length: the
// whole segments (`seg` chunks) first, then the sequences' last units by length.  Long work begins
// first then, and 8 sequences of 20 to 56 chunks leave no SM alone at the end.
__device__ __forceinline__ Unit find_unit_by_length(const SsmArgs& a, int seg, int k,
                                                    int most_units) {
  const int lane = threadIdx.x & 31;
  int s = 0, e = 0;
  if (lane < a.N) seq_range(a, lane, s, e);
  const uint32_t nc = (uint32_t)(e - s + kL - 1) / kL, whole = nc / (uint32_t)seg;
  const uint32_t rest = nc - whole * seg;
  const bool last = lane < a.N && (rest > 0 || nc == 0);
  const uint32_t nu = whole + (last ? 1 : 0);
  // sums over the sequences before: chunks (64 bits: sequences may overlap), units, whole segments
  uint64_t cs = nc;
  uint32_t us = nu, ws = whole;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t c = __shfl_up_sync(0xffffffffu, cs, o);
    const uint32_t u = __shfl_up_sync(0xffffffffu, us, o), w = __shfl_up_sync(0xffffffffu, ws, o);
    if (lane >= o) {
      cs += c;
      us += u;
      ws += w;
    }
  }
  const uint32_t all = __shfl_sync(0xffffffffu, ws, 31);
  uint32_t rank = all;  // place of the sequence's last unit
  for (int m = 0; m < a.N; ++m) {
    const uint32_t r = __shfl_sync(0xffffffffu, rest, m);
    const bool l = __shfl_sync(0xffffffffu, (int)last, m);
    if (l && (r > rest || (r == rest && m < lane))) ++rank;
  }
  const uint32_t w0 = ws - whole, kk = (uint32_t)k;
  const bool in_whole = kk >= w0 && kk < ws, mine = in_whole || (last && kk == rank);
  Unit r{lane, (int)(in_whole ? kk - w0 : whole), s, e, (int)(cs - nc), (int)(us - nu)};
  if (mine && (cs > (uint64_t)(a.T / kL + a.N) || us > (uint32_t)most_units)) {
    report_status(a.status, GDN_ERR_INVALID_ARG);  // sequences that overlap: see find_unit
    r.e = r.s;
    if (r.j > 0) r.n = -1;
  }
  const uint32_t who = __ballot_sync(0xffffffffu, mine);
  if (!who) return Unit{-1, 0, 0, 0, 0, 0};
  const bool it = lane == __ffs(who) - 1;
  return Unit{uniform(it ? r.n : -1), uniform(it ? r.j : 0),     uniform(it ? r.s : 0),
              uniform(it ? r.e : 0),  uniform(it ? r.chunk : 0), uniform(it ? r.first : 0)};
}

// C B^T in memory: for 32 rows, a block of 32 columns and a half of it, 16 columns of each row after
// one another, so that a warp (a row per lane) reads and writes 1 KB in one piece.
__device__ __forceinline__ int cb_off(int blk, int half) { return (blk * 2 + half) * 32 * 16; }

// ------------------------------------------------------------------------------------- bc
// 512 threads: warp w has tokens 8 w .. 8 w + 7 of the chunk, first of B, then of C; a lane holds 4
// channels of a row.  State widths below 128 are padded with zero channels.
// Bound by instructions: 63 % of issue slots, 1.5 TB/s.  4096 tokens of 16 groups 33 us, 65,536 of
// 8 groups 230 us; one chunk 14 us, of which an empty launch is 6.
constexpr uint32_t kBcSmem = 4 * kTileB + 2048;
constexpr int kGateHeads = 32;  // heads per gates CTA

// Steps, decays and weights of the chunk's tokens for 32 heads.  Rows of [chunk][H][3][128]: w,
// log2(delta) - cum, cum, the latter two with cum counted from the start of the token's block of
// 32; the log2 decay of each block; and that of the chunk in fp64.  The sums run in fp64: cum may
// reach thousands while only its differences count, to 2^-22 in w.
__device__ __forceinline__ void gates(const SsmTcArgs& g, const Unit& un, int part, float* d_s) {
  const SsmArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = un.s + un.j * kL, L = min(kL, un.e - t0), h0 = part * kGateHeads;
  {
    const int h = h0 + lane;
    const float bias = h < a.H && a.dt_bias ? a.dt_bias[h] : 0.f;
    float raw[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int i = warp + 16 * q;
      raw[q] = h < a.H && i < L ? __ldg(a.dt + (size_t)(t0 + i) * a.H + h) : 0.f;
    }
#pragma unroll 1
    for (int q = 0; q < 8; ++q) {
      const int i = warp + 16 * q;
      d_s[lane * 132 + i] = h < a.H && i < L ? ssm_step(raw[q] + bias, a.dt_min, a.dt_max) : 0.f;
    }
  }
  __syncthreads();
  for (int hh = warp; hh < kGateHeads; hh += 16) {
    const int h = h0 + hh;
    if (h >= a.H) break;
    const float rate2 = -1.4426950408889634f * ssm_rate(a.a_log[h]);
    const float4 d4 = *reinterpret_cast<const float4*>(d_s + hh * 132 + 4 * lane);
    const float d[4] = {d4.x, d4.y, d4.z, d4.w};
    double c[4], sum = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // a decay below 2^-150 counts as 2^-150 (zero in fp32); a NaN stays one
      const float l = rate2 * d[e];
      sum += (double)(l < -150.f ? -150.f : l);
      c[e] = sum;
    }
    double inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    const double all = __shfl_sync(0xffffffffu, inc, 31);
    const double up = __shfl_up_sync(0xffffffffu, inc, 1), before = lane ? up : 0.0;
    const double start = __shfl_sync(0xffffffffu, before, lane & 24);  // of the block of 32 tokens
    const double stop = __shfl_sync(0xffffffffu, inc, lane | 7);
    float4 w, lf, cum;
    float* pw = &w.x;
    float* pl = &lf.x;
    float* pc = &cum.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double ce = before + c[e];
      pw[e] = d[e] * exp2f((float)(all - ce));
      const float l = log2f(d[e]);
      pl[e] = (float)((double)(l < -1000.f ? -1000.f : l) - (ce - start));
      pc[e] = (float)(ce - start);
    }
    const size_t at = (size_t)(un.chunk + un.j) * a.H + h;
    float4* out = reinterpret_cast<float4*>(g.gate + at * 3 * kL) + lane;
    out[0] = w;
    out[32] = lf;
    out[64] = cum;
    if (lane == 0) g.decay[at] = all;
    if ((lane & 7) == 0) g.block[at * 4 + (lane >> 3)] = (float)(stop - start);
  }
}

__global__ void __launch_bounds__(512, 2) ssm_bc_kernel(const __grid_constant__ SsmTcArgs g) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const SsmArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  uint8_t* ctl = sm + 4 * kTileB;
  uint64_t* bar = reinterpret_cast<uint64_t*>(ctl);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(ctl + 8);
  pdl_trigger();
  const int roles = a.G + (a.H + kGateHeads - 1) / kGateHeads;
  const int grp = blockIdx.x % roles;
  const Unit un = find_unit(a, kL, kChunks, blockIdx.x / roles, gridDim.x / roles);
  if (un.n < 0) return;
  if (grp >= a.G) {
    gates(g, un, grp - a.G, reinterpret_cast<float*>(sm));
    return;
  }
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(tslot, 128);
  const int t0 = un.s + un.j * kL, L = min(kL, un.e - t0);
  const size_t at = (size_t)(un.chunk + un.j) * a.G + grp;  // tile block
  const __nv_bfloat16* c0 = static_cast<const __nv_bfloat16*>(a.conv0);
  const int row = uniform(state_row(a.slot, un.n, a.num_slots));
  // the history the later kernels read: this group's share of the channels
  if (un.j == 0 && g.hist) {
    const int per = a.Cc / 8;
    for (int v = grp * 512 + tid; v < 3 * per; v += a.G * 512) {
      uint4 r = make_uint4(0, 0, 0, 0);
      if (c0 && row >= 0) r = reinterpret_cast<const uint4*>(c0 + (size_t)row * 3 * a.Cc)[v];
      reinterpret_cast<uint4*>(g.hist + (size_t)un.n * 3 * a.Cc)[v] = r;
    }
  }
  const int i0 = warp * 8;
  uint8_t* tiles = g.tiles + at * kBcBytes;
  int8_t* ex = g.ex + at * 2 * kL;
  const bool live = lane * 4 < g.NS;
  const bool inside = t0 + i0 - 3 >= un.s && t0 + i0 + 8 <= un.e;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {  // B, then C
    const int c = a.H * a.P + (part * a.G + grp) * g.NS + lane * 4;
    uint2 raw[11];  // the warp's rows and the three before them
    if (inside) {  // all of the sequence: no checks per row (65,536 tokens: 248 us with them, 228 without)
      const __nv_bfloat16* r =
          static_cast<const __nv_bfloat16*>(a.x) + (size_t)(t0 + i0 - 3) * a.Cc + c;
#pragma unroll
      for (int q = 0; q < 11; ++q) {
        raw[q] = make_uint2(0, 0);
        if (live) raw[q] = *reinterpret_cast<const uint2*>(r);
        r += a.Cc;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 11; ++q) {  // (row addresses are the same for the whole warp)
        const int t = t0 + i0 + q - 3;
        const __nv_bfloat16* r =
            t >= un.s ? static_cast<const __nv_bfloat16*>(a.x) + (size_t)t * a.Cc
                      : (c0 && row >= 0 ? c0 + ((size_t)row * 3 + 3 + t - un.s) * a.Cc : nullptr);
        raw[q] = make_uint2(0, 0);
        if (r && i0 < L && t < un.e && live) raw[q] = *reinterpret_cast<const uint2*>(r + c);
      }
    }
    uint4 wr[2] = {};
    uint2 br = make_uint2(0, 0);
    if (live) {
      const __nv_bfloat16* cw = static_cast<const __nv_bfloat16*>(a.conv_w) + (size_t)c * 4;
      wr[0] = __ldg(reinterpret_cast<const uint4*>(cw));
      wr[1] = __ldg(reinterpret_cast<const uint4*>(cw + 8));
      if (a.conv_b)
        br = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.conv_b) + c));
    }
    float2 w[4][2], b[2];  // taps and bias of the channel pairs
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float2 wa = unpack_bf16x2(wr[p].x), wb = unpack_bf16x2(wr[p].y);
      const float2 wc = unpack_bf16x2(wr[p].z), wd = unpack_bf16x2(wr[p].w);
      w[0][p] = make_float2(wa.x, wc.x), w[1][p] = make_float2(wa.y, wc.y);
      w[2][p] = make_float2(wb.x, wd.x), w[3][p] = make_float2(wb.y, wd.y);
      b[p] = unpack_bf16x2(p ? br.y : br.x);
    }
    float2 h[3][2];  // the three rows before the current one
#pragma unroll
    for (int q = 0; q < 3; ++q)
      h[q][0] = unpack_bf16x2(raw[q].x), h[q][1] = unpack_bf16x2(raw[q].y);
    uint32_t tops = 0;
    uint8_t* hi_out = tiles + (part ? 0 : 2 * kTileB);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float2 u[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 v = unpack_bf16x2(p ? raw[q + 3].y : raw[q + 3].x);
        float2 y = __ffma2_rn(w[0][p], h[0][p], b[p]);
        y = __ffma2_rn(w[1][p], h[1][p], y);
        y = __ffma2_rn(w[2][p], h[2][p], y);
        u[p] = silu2(__ffma2_rn(w[3][p], v, y));
        h[0][p] = h[1][p], h[1][p] = h[2][p], h[2][p] = v;
        if (i0 + q >= L) u[p] = make_float2(0.f, 0.f);
      }
      const uint32_t top = __reduce_max_sync(
          0xffffffffu, __float_as_uint(max_nan(max_nan(fabsf(u[0].x), fabsf(u[0].y)),
                                               max_nan(fabsf(u[1].x), fabsf(u[1].y)))));
      if (lane == q) tops = top;
      const float sc = pow2((part ? kTargetC : kTargetB) - exponent_of(top));
      uint2 hi, lo;
      split2(mul2(u[0], sc), hi.x, lo.x);
      split2(mul2(u[1], sc), hi.y, lo.y);
      // row i0 + q of two row tiles (i0 is a multiple of 8: the swizzle goes by q)
      const uint32_t off = ((lane >> 4) * kTileB + i0 * 128 + (((lane & 15) >> 1) << 4) +
                            (lane & 1) * 8 ^ (q << 4)) + q * 128;
      *reinterpret_cast<uint2*>(sm + part * 2 * kTileB + off) = hi;
      *reinterpret_cast<uint2*>(hi_out + off) = hi;
      if (!part) *reinterpret_cast<uint2*>(hi_out + 2 * kTileB + off) = lo;
    }
    if (lane < 8) ex[part * kL + i0 + lane] = (int8_t)exponent_of(tops);
    uint32_t lost = __ballot_sync(0xffffffffu, lane < 8 && exponent_of(tops) == kNotFinite);
    for (; lost; lost &= lost - 1) {  // such a row: NaN throughout (the lane rewrites its own)
      const int q = __ffs(lost) - 1;
      const uint32_t off = ((lane >> 4) * kTileB + (i0 + q) * 128 +
                            (((((lane & 15) >> 1) ^ q) << 4) | (lane & 1) * 8));
      const uint2 nan2 = make_uint2(0x7fff7fffu, 0x7fff7fffu);
      *reinterpret_cast<uint2*>(sm + part * 2 * kTileB + off) = nan2;
      *reinterpret_cast<uint2*>(hi_out + off) = nan2;
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  if (tid == 0 && (blockIdx.x != 0 || g.skip_bc != 0)) {
    const uint32_t sB = smem_u32(sm), sC = sB + 2 * kTileB;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_bf16(tmem, desc_kmajor(sC, kk, kTileB), desc_kmajor(sB, kk, kTileB),
               idesc_f16(128, 128, false, false), kk > 0);
    mma_commit(bar);
  }
  __syncwarp();
  const bool ok = wait_long(bar, 0, g.wait_ns);
  tc_fence_after();
  if (!ok && tid == 0) report_status(a.status, GDN_ERR_TIMEOUT);
  // rows of the product: the blocks of 32 columns up to the diagonal
  __half* cb = g.cb + (at * kL + (warp & 3) * 32) * kL + lane * 16;
  {
    const int blk = warp >> 2;
    if (blk <= (warp & 3)) {
    float v[32];
    tmem_ld32(tmem_at(tmem, (warp & 3) * 32, blk * 32), v);
    tmem_ld_wait();
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      uint4 f[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float* w = v + 8 * (q + p);
        f[p].x = pack_f16x2(mul2(make_float2(w[0], w[1]), pow2(kScaleCB)));
        f[p].y = pack_f16x2(mul2(make_float2(w[2], w[3]), pow2(kScaleCB)));
        f[p].z = pack_f16x2(mul2(make_float2(w[4], w[5]), pow2(kScaleCB)));
        f[p].w = pack_f16x2(mul2(make_float2(w[6], w[7]), pow2(kScaleCB)));
      }
      store32(cb + cb_off(blk, q >> 1), f[0], f[1]);
    }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    if (!ok) wait_long(bar, 0, kWaitLimitNs);  // the product still in flight
    tmem_dealloc(tmem, 128);
  }
}

// -------------------------------------------------------------------- shared by seg and main
// One 64-channel slice of a head, worked on by a pipeline of 256 threads.
struct Slice {
  bool live;
  int h, c;        // head; first channel (of x and of the output)
};
__device__ __forceinline__ Slice slice_of(const SsmTcArgs& g, int grp, int v, int slices) {
  const SsmArgs& a = g.a;
  Slice s;
  s.live = v < slices;
  const int blocks = a.P / 64;
  s.h = grp * (a.H / a.G) + (s.live ? v / blocks : 0);
  s.c = s.h * a.P + (s.live ? v % blocks : 0) * 64;
  return s;
}
// 128 bytes towards L2, for the next chunk
__device__ __forceinline__ void prefetch_row(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The rows of a chunk's 64 channels on their way to shared memory: every warp fetches its own 16
// tokens (so that no barrier orders them, only its own wait), and the three rows before them to
// registers.
__device__ __forceinline__ void load_x(const SsmTcArgs& g, const Unit& un, const Slice& s, int t0,
                                       int warp, int lane, uint8_t* dst, uint32_t (&halo)[3]) {
  const SsmArgs& a = g.a;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + s.c;
  const int tw = t0 + warp * kTok;
#pragma unroll
  for (int q = 0; q < kTok / 4; ++q) {
    const int r = 4 * q + (lane >> 3);
    const bool in = tw + r < un.e;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     smem_u32(dst) + (warp * kTok + r) * 128 + (lane & 7) * 16),
                 "l"(x + (size_t)(in ? tw + r : un.s) * a.Cc + (lane & 7) * 8), "r"(in ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const int t = tw - 3 + q;
    halo[q] = 0;
    if (t >= un.s && t < un.e)
      halo[q] = ldg32(reinterpret_cast<const uint32_t*>(x + (size_t)t * a.Cc) + lane);
    else if (t < un.s && g.hist)
      halo[q] = *(reinterpret_cast<const uint32_t*>(
                      g.hist + ((size_t)un.n * 3 + 3 + t - un.s) * a.Cc + s.c) + lane);
  }
}
__device__ __forceinline__ void wait_x() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

// Conv + SiLU of 64 channels of the warp's 16 tokens, lane l with channels c + 2 l and c + 2 l + 1:
// put(q, u) takes token q's values (zero behind the chunk's end, L); the exponents of the token
// rows go to ex_s, and lane q returns that of its token.  `raw`: the chunk's rows.
// The taps and the bias of a lane's two channels stay packed (5 registers, not 10).
struct Taps {
  uint4 w;
  uint32_t b;
};
__device__ __forceinline__ Taps load_taps2(const SsmArgs& a, const Slice& s, int lane) {
  const int c = s.c + 2 * lane;
  Taps t{make_uint4(0, 0, 0, 0), 0};
  t.w = ldg128(static_cast<const __nv_bfloat16*>(a.conv_w) + (size_t)c * 4);
  if (a.conv_b) t.b = ldg32(static_cast<const __nv_bfloat16*>(a.conv_b) + c);
  return t;
}
template <typename Put>
__device__ __forceinline__ int conv_x(const Taps& tp, int L, int warp, int lane, const uint8_t* raw,
                                      const uint32_t (&halo)[3], int8_t* ex_s, Put&& put) {
  uint4 wr = tp.w;
  uint32_t br = tp.b;
  asm volatile("" : "+r"(wr.x), "+r"(wr.y), "+r"(wr.z), "+r"(wr.w), "+r"(br));
  const float2 wa = unpack_bf16x2(wr.x), wb = unpack_bf16x2(wr.y);
  const float2 wc = unpack_bf16x2(wr.z), wd = unpack_bf16x2(wr.w);
  const float2 w0 = make_float2(wa.x, wc.x), w1 = make_float2(wa.y, wc.y);
  const float2 w2 = make_float2(wb.x, wd.x), w3 = make_float2(wb.y, wd.y);
  const float2 b = unpack_bf16x2(br);
  const uint32_t* at = reinterpret_cast<const uint32_t*>(raw + warp * kTok * 128) + lane;
  const int live = L - warp * kTok;  // tokens of this warp
  float2 h0 = unpack_bf16x2(halo[0]), h1 = unpack_bf16x2(halo[1]), h2 = unpack_bf16x2(halo[2]);
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < kTok; ++q) {
    const float2 v = unpack_bf16x2(at[q * 32]);
    float2 u =
        silu2(__ffma2_rn(w3, v, __ffma2_rn(w2, h2, __ffma2_rn(w1, h1, __ffma2_rn(w0, h0, b)))));
    h0 = h1;
    h1 = h2;
    h2 = v;
    if (q >= live) u = make_float2(0.f, 0.f);
    put(q, u);
    const uint32_t m =
        __reduce_max_sync(0xffffffffu, __float_as_uint(max_nan(fabsf(u.x), fabsf(u.y))));
    if (lane == q) top = m;
  }
  const int e = exponent_of(top);
  if (lane < kTok) ex_s[warp * kTok + lane] = (int8_t)e;
  return e;
}

// B^T wX, what a chunk adds to S^T: three products of the two parts of each (the fourth is below
// 2^-22 of the first).
// (In these three the base addresses are made opaque: as loop invariants all descriptors would be
// computed before the chunk loop, and spill.)
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}
__device__ __forceinline__ void mma_state(uint32_t lead, uint32_t tS, uint32_t sB, uint32_t sW) {
  const uint32_t A = opaque(desc_low(sB, kTileB)), W = opaque(desc_low(sW, kTileB));
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_ss(lead, tS, A + (((p == 1 ? 2 * kTileB : 0) + kk * 2048) >> 4),
             W + (((p == 2 ? kTileB : 0) + kk * 2048) >> 4), idesc_f16(128, 64, true, true),
             (p | kk) != 0);
}
// C S^T: C^ by rows (two row tiles of 64 columns), S^ by columns.
__device__ __forceinline__ void mma_in(uint32_t lead, uint32_t tI, uint32_t sC, uint32_t sS) {
  const uint32_t A = opaque(desc_low(sC, 16)), B = opaque(desc_low(sS, kTileB));
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ss(lead, tI, A + (((kk >> 2) * kTileB + (kk & 3) * 32) >> 4), B + ((kk * 2048) >> 4),
           idesc_f16(128, 64, false, true), kk != 0);
}
// P X: P^ in TMEM.
__device__ __forceinline__ void mma_px(uint32_t lead, uint32_t tX, uint32_t tP, uint32_t sX) {
  const uint32_t B = opaque(desc_low(sX, kTileB));
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(lead, tX, tP + kk * 8, B + ((kk * 2048) >> 4), idesc_f16(128, 64, false, true), kk != 0);
}

// Exponent of the largest value row i of wX may hold (w, and the rows of X and B).  A weight of zero
// (a token masked by its step) counts for nothing, however large its rows.
__device__ __forceinline__ int weight_exponent(float w, int eX, int eB) {
  return w == 0.f ? -1000 : (int)(abs_bits(w) >> 23) - 127 + eX + eB;
}

// The chunk's exponent of wX, by a whole warp (lane l: tokens 4 l .. 4 l + 3; every warp of the
// pipeline finds the same one).
__device__ __forceinline__ int chunk_exponent(const float4& w4, uint32_t ex4, uint32_t eB4) {
  const float w[4] = {w4.x, w4.y, w4.z, w4.w};
  int top = INT32_MIN;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    top = max(top, weight_exponent(w[e], (int)(int8_t)(ex4 >> (8 * e)), (int)(int8_t)(eB4 >> (8 * e))));
  return __reduce_max_sync(0xffffffffu, top);
}

// Byte offset of the warp's token q and the lane's channel pair in a [128][64] row tile; the 16-byte
// pieces of row r are swizzled by r % 8.
__device__ __forceinline__ uint32_t pair_off(int warp, int lane, int q) {
  return ((warp * kTok * 128 + ((lane >> 2) << 4) + (lane & 3) * 4) ^ ((q & 7) << 4)) + q * 128;
}
// w 2^e, the weight of a token whose row of X has exponent eX
__device__ __forceinline__ float token_weight(float w, int eX, int e) {
  return eX == kNotFinite ? __int_as_float(0x7fffffff) : scale2(w, e);
}
// Two parts of u w into the tiles at W (high) and W + kTileB (low).
__device__ __forceinline__ void store_parts(float2 u, float w, uint8_t* W, uint32_t at) {
  uint32_t hi, lo;
  split2(mul2(u, w), hi, lo);
  *reinterpret_cast<uint32_t*>(W + at) = hi;
  *reinterpret_cast<uint32_t*>(W + at + kTileB) = lo;
}

// ------------------------------------------------------------------------------------ seg
// The state a segment adds, the sum over its tokens of 2^(log decay from the token to the
// segment's end) delta x B^T (for the first segment: and the decayed initial state), chunk by
// chunk from its end; the chunks' contributions are added in fp32 registers.
// 3.7 us per chunk of 128 channels; 65,536 tokens of 64 heads of 64 412 us, 52 % of issue slots busy.
// smem: two stages of B (64 KB), wX (32 KB) and a chunk of x rows (16 KB) per pipeline, control.
constexpr uint32_t kSegW = 8 * kTileB, kSegCtl = kSegW + 6 * kTileB;
constexpr uint32_t kSegSmem = kSegCtl + 3072;

__global__ void __launch_bounds__(512, 1) ssm_seg_kernel(const __grid_constant__ SsmTcArgs g) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const SsmArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_trigger();
  const int slices = (a.H / a.G) * (a.P / 64), pairs = (slices + 1) / 2;
  const int grp = (blockIdx.x % (a.G * pairs)) / pairs, pair = blockIdx.x % pairs;
  const Unit un = find_unit(a, g.seg * kL, kFollowed, blockIdx.x / (a.G * pairs),
                            gridDim.x / (a.G * pairs));
  pdl_wait();  // before any return: the next kernel counts on this one having waited
  if (un.n < 0) return;
  const int c0 = un.j * g.seg, c1 = c0 + g.seg;  // whole: another segment follows

  const int wid = uniform(tid >> 5), pipe = wid >> 3, pw = wid & 7, pt = tid & 255;
  uint8_t* ctl = sm + kSegCtl;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctl);      // [2] B stages landed
  uint64_t* done = full + 2;                              // [2] a pipeline's products
  int* count = reinterpret_cast<int*>(ctl + 48);          // [2] uses of a stage, both pipelines
  int* loads = count + 2;                                 // [2] copies into it
  uint32_t* tslot = reinterpret_cast<uint32_t*>(ctl + 64);
  // exponents of the rows of X, of two chunks: a warp may begin the next one's conv while another
  // has yet to read this one's
  int8_t* ex2_s = reinterpret_cast<int8_t*>(ctl + 128) + pipe * 2 * kL;
  if (tid == 0) {
    for (int k = 0; k < 4; ++k) {
      mbar_init(full + k, 1);
      count[k] = 0;  // and loads
    }
    fence_barrier_init();
  }
  if (tid < 32) tmem_alloc(tslot, 128);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tslot), tS = tmem + pipe * 64;
  const Slice s = slice_of(g, grp, 2 * pair + pipe, slices);
  const int users = min(2, slices - 2 * pair);
  const int nch = c1 - c0;
  auto load_b = [&](int k) {  // k-th chunk from the end
    if (k == g.skip_seg && blockIdx.x == 0) return;
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
  float scale = 0.f;  // of the products in flight
  bool ok = true;
  int mmas = 0;
  uint8_t* W = sm + kSegW + pipe * 3 * kTileB;
  uint8_t* raw = W + 2 * kTileB;
  const uint32_t sB = smem_u32(sm), sW = smem_u32(W);
  const int warp = pw;
  // adds the products of chunk k (they have read wX and the stage then); the last pipeline
  // through with a stage fetches the next chunk but one into it
  auto take = [&](int k) {
    ok = wait_long(done + pipe, k & 1, g.wait_ns) && ok;
    tc_fence_after();
    if (pt == 0 && ok) {
      __threadfence_block();
      if (atomicAdd(count + (k & 1), 1) == users * ((k >> 1) + 1) - 1 && k + 2 < nch) {
        __threadfence_block();
        load_b(k + 2);
      }
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float d[16];
      tmem_ld16(tmem_at(tS, (pw & 3) * 32, (pw >> 2) * 32 + 16 * r), d);
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 16; ++q) v[16 * r + q] = fmaf(scale, d[q], v[16 * r + q]);
    }
    tc_fence_before();
  };
  if (s.live) {
    uint32_t halo[3];
    const Taps taps = load_taps2(a, s, lane);
    load_x(g, un, s, un.s + (c1 - 1) * kL, warp, lane, raw, halo);
    for (int k = 0; k < nch; ++k) {
      const int ch = c1 - 1 - k, t0 = un.s + ch * kL, own = warp * kTok + (lane & (kTok - 1));
      const size_t at = (size_t)(un.chunk + ch) * a.H + s.h;
      const float* gate = g.gate + at * 3 * kL;
      const int8_t* ex = g.ex + ((size_t)(un.chunk + ch) * a.G + grp) * 2 * kL;
      const float4 w4 = ldgf4(gate + 4 * lane);
      const uint32_t eB4 = ldg32(ex + 4 * lane);
      const float w = ldgf(gate + own);  // of this lane's token
      const int eB = ldg8(ex + own);
      const double all = __ldg(g.decay + at);
      if (k + 2 < nch && pt < 128)
        prefetch_row(static_cast<const __nv_bfloat16*>(a.x) + (size_t)(t0 - 2 * kL + pt) * a.Cc + s.c);
      wait_x();
      float2 u[kTok];
      int8_t* ex_s = ex2_s + (k & 1) * kL;
      const int eq =
          conv_x(taps, kL, warp, lane, raw, halo, ex_s, [&](int q, float2 v) { u[q] = v; });
      __syncwarp();  // the warp has read its rows
      if (k + 1 < nch) load_x(g, un, s, t0 - kL, warp, lane, raw, halo);
      if (bar_or_n(1 + pipe, kPipe, !ok)) break;
      const int top = chunk_exponent(w4, reinterpret_cast<const uint32_t*>(ex_s)[lane], eB4);
      const float wq = token_weight(w, eq, eB + kTargetW - top);
      if (k > 0) take(k - 1);
      scale = scale2(exp2f((float)R), top - kTargetW - kTargetB);
      R += all;
#pragma unroll
      for (int q = 0; q < kTok; ++q)
        store_parts(u[q], __shfl_sync(0xffffffffu, wq, q), W, pair_off(warp, lane, q));
      fence_proxy_async_smem();
      if (warp != 0) {
        bar_arrive_n(3 + pipe, kPipe);
      } else {
        bar_sync_n(3 + pipe, kPipe);
        const bool got = wait_long(full + (k & 1), (k >> 1) & 1, g.wait_ns);
        tc_fence_after();
        if (__all_sync(0xffffffffu, got)) {
          const uint32_t lead = elect_one();
          mma_state(lead, tS, sB + (k & 1) * 4 * kTileB, sW);
          if (lead) mma_commit(done + pipe);
          ++mmas;
        } else {
          ok = false;
        }
        __syncwarp();
      }
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
          const int last = ((un.e - un.s + kL - 1) / kL - 1) / g.seg;  // segment of the sequence
          float* keep = g.seg_state + (size_t)(un.first + last) * pitch + base;
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
      if (mmas > 0) wait_long(done + pipe, (mmas - 1) & 1, kWaitLimitNs);
    }
    wait_x();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0)  // copies in flight, after a wait that ran out
    for (int k = 0; k < 2; ++k)
      if (loads[k] > 0) wait_long(full + k, (loads[k] - 1) & 1, kWaitLimitNs);
  if (tid < 32) tmem_dealloc(tmem, 128);
}

// ----------------------------------------------------------------------------------- main
// smem: C^ | B high | B low (96 KB, shared by both pipelines), then per pipeline X^ | wX high |
// wX low | S^ (64 KB), and 3 KB of control: with no more to be had, the base has to be aligned.
// The place of S^ also takes the next chunk's x rows, from the end of the products of one chunk
// until the conv of the next has read them.
// TMEM, per pipeline: what the chunk adds to S^T (64 columns), C S^T and P X (128), P (64).  S^T
// itself stays in registers (32 of a row per thread): fp32 sums there round to nearest.
// Bound by the chain of a chunk's phases (conv, scales, weights, products, epilogue): 9 us for the
// two pipelines, with 44 % of issue slots and 11 % of the tensor pipe busy.
// 4096 tokens of 32 heads of 128 89 us, 65,536 of 64 heads of 64 1045 us, 40,677 in eight 791 us.
constexpr uint32_t kMainPipe = 6 * kTileB, kMainCtl = kMainPipe + 8 * kTileB;
constexpr uint32_t kMainSmem = kMainCtl + 3072;

__global__ void __launch_bounds__(512, 1) ssm_main_kernel(const __grid_constant__ SsmTcArgs g) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const SsmArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_trigger();
  const int slices = (a.H / a.G) * (a.P / 64), pairs = (slices + 1) / 2;
  const int grp = (blockIdx.x % (a.G * pairs)) / pairs, pair = blockIdx.x % pairs;
  const int unit = blockIdx.x / (a.G * pairs), units = gridDim.x / (a.G * pairs);
  const Unit un = a.N <= 32 ? find_unit_by_length(a, g.seg, unit, units)
                            : find_unit(a, g.seg * kL, kSegments, unit, units);
  if (un.n < 0) {
    pdl_wait();
    return;
  }
  const int wid = uniform(tid >> 5), pipe = wid >> 3, pw = wid & 7, pt = tid & 255;
  uint8_t* ctl = sm + kMainCtl;
  uint64_t* c_full = reinterpret_cast<uint64_t*>(ctl);
  uint64_t* b_full = c_full + 1;
  uint64_t* done = c_full + 2;  // [2] a pipeline's products of a chunk
  int* count = reinterpret_cast<int*>(ctl + 48);  // chunks finished, over both pipelines
  int* loads = count + 1;                         // chunks whose tiles were fetched
  uint32_t* tslot = reinterpret_cast<uint32_t*>(ctl + 56);
  uint8_t* mine = ctl + 64 + pipe * 1408;
  uint32_t* top_s = reinterpret_cast<uint32_t*>(mine);      // [8] largest magnitudes of S
  float* m_s = reinterpret_cast<float*>(mine + 64);         // [4] maxima of g of the blocks
  float* pm_s = reinterpret_cast<float*>(mine + 128);       // [128] running maximum of g
  float* f_s = pm_s + kL;                                   // [128] F: 2^(g - maximum of the block)
  int8_t* ex_s = reinterpret_cast<int8_t*>(f_s + kL);       // [128] exponents of the rows of X
  if (tid == 0) {
    for (int k = 0; k < 4; ++k) mbar_init(c_full + k, 1);
    *count = *loads = 0;
    fence_barrier_init();
  }
  if (tid < 32) tmem_alloc(tslot, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tslot);
  const uint32_t tS = tmem + pipe * 64, tI = tmem + 128 + pipe * 128, tX = tI + 64;
  const uint32_t tP = tmem + 384 + pipe * 64;
  const Slice s = slice_of(g, grp, 2 * pair + pipe, slices);
  const int users = min(2, slices - 2 * pair);
  const int total = (un.e - un.s + kL - 1) / kL;
  const int c0 = un.j * g.seg, c1 = min(total, c0 + g.seg), nch = c1 - c0;
  const int row = uniform(state_row(a.slot, un.n, a.num_slots));
  if (row < 0 && tid == 0) report_status(a.status, GDN_ERR_INVALID_ARG);
  const float D = a.D ? a.D[s.h] : 0.f;
  // whole sectors of z and of the output, where their addresses allow it (40,677 tokens in eight
  // sequences: a call 837 us; with z in 16-byte pieces 848)
  const bool wide =
      ((reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.z)) & 31u) == 0;
  auto load_z = [&](const __nv_bfloat16* p, uint4& lo, uint4& hi) {
    if (wide) {
      load32_nc(p, lo, hi);
    } else {
      lo = ldg128(p);
      hi = ldg128(p + 8);
    }
  };
  const int quad = pw & 3, half = pw >> 2;
  const int i = quad * 32 + lane;   // row of this thread: token of the chunk, or n of the state
  const int p0 = half * 32;         // its channels
  const size_t pitch = (size_t)a.H * a.P * g.NS, sbase = (size_t)(s.c + p0) * g.NS + i;
  pdl_wait();
  auto load_tiles = [&](int c) {
    if (c - c0 == g.skip_main && blockIdx.x == 0) return;
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
  {
    // P above the diagonal blocks is zero throughout
    const uint32_t zero[16] = {};
    tmem_st16(tmem_at(tP, quad * 32, p0), zero);
    tmem_st16(tmem_at(tP, quad * 32, p0 + 16), zero);
    tmem_st_wait();
  }
  uint8_t* X = sm + kMainPipe + pipe * 4 * kTileB;
  uint8_t* W = X + kTileB;
  uint8_t* S16 = X + 3 * kTileB;  // and the next chunk's rows of x
  const uint32_t sC = smem_u32(sm), sX = smem_u32(X), sW = smem_u32(W), sS = smem_u32(S16);
  const int warp = pw;
  bool ok = true;
  int mmas = 0;
  float smax = 0.f;  // largest magnitude of this thread's part of S
#pragma unroll
  for (int q = 0; q < 32; ++q) smax = fmaxf(smax, fabsf(sv[q]));
  if (s.live) {
    uint32_t halo[3];
    Taps taps{};
    if (nch > 0) {  // (a call without a token may have neither taps nor rows)
      taps = load_taps2(a, s, lane);
      load_x(g, un, s, un.s + c0 * kL, warp, lane, S16, halo);
    }
    for (int k = 0; k < nch; ++k) {
      const int t0 = un.s + (c0 + k) * kL, L = min(kL, un.e - t0);
      const size_t chunk = (size_t)(un.chunk + c0 + k), at = chunk * a.G + grp;
      const float* gate = g.gate + (chunk * a.H + s.h) * 3 * kL;
      const int8_t* ex = g.ex + at * 2 * kL;
      if (t0 + kL + i < un.e && k + 1 < nch) {  // the next chunk's inputs on their way
        const size_t t1 = (size_t)t0 + kL + i;
        if (half == 0) prefetch_row(static_cast<const __nv_bfloat16*>(a.x) + t1 * a.Cc + s.c);
        else if (a.z)
          prefetch_row(static_cast<const __nv_bfloat16*>(a.z) + t1 * a.H * a.P + s.c);
      }
      // ---- conv of X; the largest magnitude of S
      const float4 w4 = ldgf4(gate + 4 * lane);
      const uint32_t eB4 = ldg32(ex + 4 * lane);
      const float w = ldgf(gate + warp * kTok + (lane & (kTok - 1)));
      const float lfi = ldgf(gate + kL + i);
      const int eBi = ldg8(ex + i);
      const float4 bt = ldgf4(g.block + (chunk * a.H + s.h) * 4);
      wait_x();
      // u stays in the place of its two parts of wX until their scale is known (in registers
      // beside S it would spill)
      const int eq = conv_x(taps, L, warp, lane, S16, halo, ex_s, [&](int q, float2 u) {
        const uint32_t at = pair_off(warp, lane, q);
        *reinterpret_cast<float*>(W + at) = u.x;
        *reinterpret_cast<float*>(W + at + kTileB) = u.y;
      });
      uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(smax));
      if (lane == 0) top_s[warp] = top;
      if (bar_or_n(1 + pipe, kPipe, !ok)) break;
      // ---- S^ = fp16 operand of C S^T
      top = __reduce_max_sync(0xffffffffu, top_s[lane & 7]);
      const int eS = exponent_of(top);
      {
        // (an infinity in the state: as a row of X that holds one)
        const float sc = eS == kNotFinite ? __int_as_float(0x7fffffff) : pow2(kTargetS - eS);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 f;
          f.x = pack_f16x2(mul2(make_float2(sv[8 * q], sv[8 * q + 1]), sc));
          f.y = pack_f16x2(mul2(make_float2(sv[8 * q + 2], sv[8 * q + 3]), sc));
          f.z = pack_f16x2(mul2(make_float2(sv[8 * q + 4], sv[8 * q + 5]), sc));
          f.w = pack_f16x2(mul2(make_float2(sv[8 * q + 6], sv[8 * q + 7]), sc));
          *reinterpret_cast<uint4*>(S16 + sw128_off(i, half * 4 + q)) = f;
        }
      }
      // ---- weights of wX; X^ and wX
      const uint32_t ex4 = reinterpret_cast<const uint32_t*>(ex_s)[lane];
      const int wt = chunk_exponent(w4, ex4, eB4);
      {
        const int own = warp * kTok + (lane & (kTok - 1));
        const uint32_t e4 = __shfl_sync(0xffffffffu, eB4, own >> 2);
        const int eB = (int)(int8_t)(e4 >> (8 * (own & 3)));
        const float wq = token_weight(w, eq, eB + kTargetW - wt);
        const float xs = pow2(kTargetX - eq);
#pragma unroll
        for (int q0 = 0; q0 < kTok; q0 += 8) {  // eight loads, then their stores
          float2 u[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t at = pair_off(warp, lane, q0 + q);
            u[q] = make_float2(*reinterpret_cast<const float*>(W + at),
                               *reinterpret_cast<const float*>(W + at + kTileB));
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t at = pair_off(warp, lane, q0 + q);
            *reinterpret_cast<uint32_t*>(X + at) =
                pack_f16x2(mul2(u[q], __shfl_sync(0xffffffffu, xs, q0 + q)));
            store_parts(u[q], __shfl_sync(0xffffffffu, wq, q0 + q), W, at);
          }
        }
      }
      uint32_t lost = __ballot_sync(0xffffffffu, lane < kTok && eq == kNotFinite);
      for (; lost; lost &= lost - 1)  // zero rows of X^ (the lane rewrites its own)
        *reinterpret_cast<uint32_t*>(X + pair_off(warp, lane, __ffs(lost) - 1)) = 0u;
      // ---- g of token i, in units of its block's start
      const int eX = ex_s[i];
      const float gi = eX == -kNotFinite ? __int_as_float(0x7fffffff) : lfi + (float)(eX + eBi);
      if (half == 0) {
        // its running maximum, and the maxima M of the blocks (lane l: tokens 4 l ..)
        const float4 lf4 = ldgf4(gate + kL + 4 * lane);
        float pm = gi;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float up = __shfl_up_sync(0xffffffffu, pm, o);
          if (lane >= o) pm = fmaxf(pm, up);
        }
        const float l4[4] = {lf4.x, lf4.y, lf4.z, lf4.w};
        float gm = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          gm = fmaxf(gm, l4[e] + (float)((int)(int8_t)(ex4 >> (8 * e)) + (int)(int8_t)(eB4 >> (8 * e))));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
        const float M0 = __shfl_sync(0xffffffffu, gm, 0);
        const float M1 = fmaxf(M0 + bt.x, __shfl_sync(0xffffffffu, gm, 8));
        const float M2 = fmaxf(M1 + bt.y, __shfl_sync(0xffffffffu, gm, 16));
        const float M3 = fmaxf(M2 + bt.z, __shfl_sync(0xffffffffu, gm, 24));
        if (quad == 1) pm = fmaxf(pm, M0 + bt.x);
        if (quad == 2) pm = fmaxf(pm, M1 + bt.y);
        if (quad == 3) pm = fmaxf(pm, M2 + bt.z);
        pm_s[i] = pm;
        f_s[i] = ex2(gi - (quad == 0 ? M0 : (quad == 1 ? M1 : (quad == 2 ? M2 : M3))));
        if (pt == 0) *reinterpret_cast<float4*>(m_s) = make_float4(M0, M1, M2, M3);
      }
      // C B^T of this thread's columns: 16 of each block of 32 up to the diagonal
      // (two blocks ahead)
      const __half* cb = g.cb + (at * kL + quad * 32) * kL + lane * 16;
      uint4 cbr[2][2];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        if (blk <= quad) {
          load32_nc(cb + cb_off(blk, half), cbr[blk][0], cbr[blk][1]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      bar_sync_n(1 + pipe, kPipe);
      if (warp == 0) {
        const bool got = wait_long(c_full, k & 1, g.wait_ns) && wait_long(b_full, k & 1, g.wait_ns);
        tc_fence_after();
        if (__all_sync(0xffffffffu, got)) {
          const uint32_t lead = elect_one();
          mma_in(lead, tI, sC, sS);
          mma_state(lead, tS, sC + 2 * kTileB, sW);
        } else {
          ok = false;
        }
        __syncwarp();
      }
      // ---- P^ (fp16) into TMEM, its weights in fp32: one token with a large channel makes those of
      // the others small for all channels.  ref: the blocks' maxima from this block's start on; cs:
      // decay up to this block
      const float pm = pm_s[i];
      float cs = 0.f;
      {
        const float4 M = *reinterpret_cast<const float4*>(m_s);
        float ref[3] = {0.f, 0.f, 0.f};
        if (quad == 1) {
          cs = bt.x, ref[0] = M.x + bt.x;
        } else if (quad == 2) {
          cs = bt.x + bt.y, ref[0] = M.x + (bt.x + bt.y), ref[1] = M.y + bt.y;
        } else if (quad == 3) {
          cs = bt.x + (bt.y + bt.z), ref[0] = M.x + cs, ref[1] = M.y + (bt.y + bt.z);
          ref[2] = M.z + bt.z;
        }
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) {
          if (blk <= quad) {
            const uint4 r0 = cbr[blk & 1][0], r1 = cbr[blk & 1][1];
            const uint32_t in[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
            if (blk + 2 <= quad) {
              load32_nc(cb + cb_off(blk + 2, half), cbr[blk & 1][0], cbr[blk & 1][1]);
            }
            uint32_t out[8];
            const int j0 = blk * 32 + half * 16;
            if (blk < quad) {
              const float rf = ex2(ref[blk < 3 ? blk : 2] - pm);
#pragma unroll
              for (int q = 0; q < 8; q += 2) {
                const float4 f = *reinterpret_cast<const float4*>(f_s + j0 + 2 * q);
                out[q] = pack_f16x2(__fmul2_rn(unpack_f16x2(in[q]), mul2(make_float2(f.x, f.y), rf)));
                out[q + 1] =
                    pack_f16x2(__fmul2_rn(unpack_f16x2(in[q + 1]), mul2(make_float2(f.z, f.w), rf)));
              }
            } else {
              // the diagonal block: g of its tokens is in the lanes of this warp
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const int j = half * 16 + 2 * q;
                const float ea = __shfl_sync(0xffffffffu, gi, j) - pm;
                const float eb = __shfl_sync(0xffffffffu, gi, j + 1) - pm;
                const float2 v = unpack_f16x2(in[q]);
                out[q] = pack_f16x2(make_float2(j <= lane ? v.x * ex2(ea) : 0.f,
                                                j + 1 <= lane ? v.y * ex2(eb) : 0.f));
              }
            }
            tmem_st8(tmem_at(tP, quad * 32, j0 / 2), out);
          }
        }
        tmem_st_wait();
      }
      tc_fence_before();
      if (warp != 0) {
        bar_arrive_n(3 + pipe, kPipe);
      } else {
        bar_sync_n(3 + pipe, kPipe);
        tc_fence_after();
        if (__all_sync(0xffffffffu, ok)) {
          const uint32_t lead = elect_one();
          mma_px(lead, tX, tP, sX);
          if (lead) mma_commit(done + pipe);
          ++mmas;
        }
        __syncwarp();
      }
      // ---- outputs
      const bool in = i < L;
      const size_t o_at = ((size_t)(t0 + i) * a.H) * a.P + s.c + p0;
      const __nv_bfloat16* zp = static_cast<const __nv_bfloat16*>(a.z) + o_at;
      uint4 zr[2] = {};  // of two quarters
      if (a.z && in) load_z(zp, zr[0], zr[1]);
      const float cum = ldgf(gate + 2 * kL + i);
      const int eC = ldg8(ex + kL + i);
      const float dec = exp2f((float)__ldg(g.decay + chunk * a.H + s.h));
      const float si = ex2(cs + cum + (float)(eC + eS - kTargetS - kTargetC));
      const float sx = ex2((cum + pm) + (float)(eC - kTargetC - kTargetB - kScaleCB - kTargetX));
      const float dx = D * pow2(eX - kTargetX);
      const float ds = scale2(1.f, wt - kTargetW - kTargetB);
      ok = wait_long(done + pipe, k & 1, g.wait_ns) && ok;
      tc_fence_after();
      if (pt == 0 && ok) {  // the last pipeline through with the tiles fetches the next ones
        __threadfence_block();
        if (atomicAdd(count, 1) == users * (k + 1) - 1 && k + 1 < nch) {
          __threadfence_block();
          load_tiles(c0 + k + 1);
        }
      }
      __syncwarp();
      if (k + 1 < nch) load_x(g, un, s, t0 + kL, warp, lane, S16, halo);
      __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + o_at;
      smax = 0.f;
      uint4 even = {};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float yi[8], yx[8], add[8];
        tmem_ld8(tmem_at(tI, quad * 32, p0 + 8 * r), yi);
        tmem_ld8(tmem_at(tX, quad * 32, p0 + 8 * r), yx);
        tmem_ld8(tmem_at(tS, quad * 32, p0 + 8 * r), add);
        tmem_ld_wait();
        // S^T <- 2^cum_L S^T + what the chunk adds
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
          const float2 n2 = __ffma2_rn(make_float2(dec, dec),
                                       make_float2(sv[8 * r + q], sv[8 * r + q + 1]),
                                       mul2(make_float2(add[q], add[q + 1]), ds));
          sv[8 * r + q] = n2.x;
          sv[8 * r + q + 1] = n2.y;
          smax = fmaxf(smax, fmaxf(fabsf(n2.x), fabsf(n2.y)));
        }
        if (in) {
          const uint4 xr = *reinterpret_cast<const uint4*>(X + sw128_off(i, half * 4 + r));
          const uint4 zv = zr[r & 1];
          if (r == 1 && a.z) load_z(zp + 16, zr[0], zr[1]);
          const uint32_t xw[4] = {xr.x, xr.y, xr.z, xr.w};
          const uint32_t zw[4] = {zv.x, zv.y, zv.z, zv.w};
          uint32_t ow[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 y = mul2(unpack_f16x2(xw[e]), dx);
            y = __ffma2_rn(make_float2(sx, sx), make_float2(yx[2 * e], yx[2 * e + 1]), y);
            y = __ffma2_rn(make_float2(si, si), make_float2(yi[2 * e], yi[2 * e + 1]), y);
            if (a.z) y = __fmul2_rn(y, silu2(unpack_bf16x2(zw[e])));
            ow[e] = pack_bf16x2(y.x, y.y);
          }
          // two quarters leave together (with 16-byte stores, in the case above, 837 us become 869)
          const uint4 now = make_uint4(ow[0], ow[1], ow[2], ow[3]);
          if ((r & 1) == 0) {
            even = now;
          } else if (wide) {
            store32(op + 8 * (r - 1), even, now);
          } else {
            *reinterpret_cast<uint4*>(op + 8 * (r - 1)) = even;
            *reinterpret_cast<uint4*>(op + 8 * r) = now;
          }
        }
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
      if (mmas > 0) wait_long(done + pipe, (mmas - 1) & 1, kWaitLimitNs);
    }
    wait_x();
  }
  if (c1 == total)
    conv_history<__nv_bfloat16>(a, un.n, row, un.s, un.e, blockIdx.x % (a.G * pairs), a.G * pairs);
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *loads > 0) {  // copies in flight, after a wait that ran out
    wait_long(c_full, (*loads - 1) & 1, kWaitLimitNs);
    wait_long(b_full, (*loads - 1) & 1, kWaitLimitNs);
  }
  if (tid < 32) tmem_dealloc(tmem, 512);
}

}  // namespace gdn

namespace gdn_host {

cudaError_t launch_ssm_tc(gdn::SsmTcArgs g, void* workspace, cudaStream_t s);
size_t ssm_tc_workspace(int N, int T, int H, int G, int P, int NS, int Cc);

namespace {

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Chunks per segment.  A CTA works on 128 channels of one segment, so a call has pairs x units CTAs,
// one per SM, the longest first.
// One sequence: the length with the least time, counted in chunks of main: a CTA's chunks and half a
// one to begin, whole segments over the SMs and then the shorter last ones, and 0.36 for a chunk of
// the segments that seg goes over first.  Measured at 65,536 tokens of 64 heads: segments of 29
// chunks 1694 us, of 37 1826 and of 64 1762 us, 1.08 and 1.04 times as long (the count says 1.11 and
// 1.09); of 56, which it chooses, 1604 to 1689 us by the clocks.  4096 tokens of 32 heads of 128: 8
// chunks, which it chooses, 147 us, 4 167, 16 248.
// Several (whose lengths only the device knows): an SM's even share of the chunks, so that a sequence
// is cut only if it alone would keep its SMs longer than the whole call should take; every other cut
// costs a second conv and state update.  8 sequences of 20 to 56 chunks (bf16, 64 heads of 64): a
// call takes 837 us so, 959 in segments of 19 (four waves), and 885 with the units in order.
constexpr int kSms = 148, kMostWaves = 4;
// Until the last SM is through with n CTAs of `a` and then m of `b` <= a.
double makespan(int64_t n, double a, int64_t m, double b) {
  const int64_t over = n % kSms, left = kSms - over, rounds = (m + left - 1) / left;
  const double low = (double)(n / kSms) * a, high = over ? low + a : low;
  const double even = ((double)n * a + (double)m * b) / kSms + b;
  return std::max(high, std::min(low + (double)rounds * b, even));
}
int64_t ssm_segment(int N, int T, int pairs) {
  if (N > 1) {
    const int64_t chunks = (int64_t)T / gdn::kL + N;
    const int units = std::max(1, kSms / pairs);
    return (chunks + units - 1) / units;
  }
  const int64_t chunks = std::max<int64_t>(1, ((int64_t)T + gdn::kL - 1) / gdn::kL);
  int64_t best = chunks;
  double least = makespan(0, 0.0, pairs, chunks + 0.5);
  for (int quarters = 5; quarters <= 4 * (kSms * kMostWaves / pairs); ++quarters) {
    const int64_t seg = (4 * chunks + quarters - 1) / quarters;
    if (seg >= chunks) continue;
    const int64_t whole = chunks / seg, rest = chunks % seg;
    const double time = makespan(whole * pairs, seg + 0.5, rest ? pairs : 0, rest + 0.5) +
                        0.36 * makespan((whole - (rest ? 0 : 1)) * pairs, seg + 0.5, 0, 0.0);
    if (time < least) {
      least = time;
      best = seg;
    }
    if (seg == 1) break;
  }
  return best;
}

struct TcLayout {
  int64_t seg, units;  // chunks per segment, segments
  size_t tiles, cb, ex, hist, gate, block, decay, seg_state, seg_decay, total;
};

TcLayout tc_layout(int N, int T, int H, int G, int P, int NS, int Cc) {
  TcLayout l{};
  const int pairs = G * (((H / G) * (P / 64) + 1) / 2);
  const size_t chunks = (size_t)T / gdn::kL + N, blocks = chunks * G;
  l.seg = ssm_segment(N, T, pairs);
  l.units = T / (l.seg * gdn::kL) + N;
  // room for the states of as many segments as any rule of ssm_segment makes: the size grows with N
  // and with T, so a workspace for a server's largest batch takes the others too
  const size_t room = std::min(T / gdn::kL, kSms * kMostWaves / pairs) + (size_t)N;
  size_t o = 0;
  l.tiles = o; o = up256(o + blocks * gdn::kBcBytes);
  l.cb = o; o = up256(o + blocks * gdn::kL * gdn::kL * 2);
  l.ex = o; o = up256(o + blocks * 2 * gdn::kL);
  l.hist = o; o = up256(o + (size_t)N * 3 * Cc * 2);
  l.gate = o; o = up256(o + chunks * H * 3 * gdn::kL * 4);
  l.block = o; o = up256(o + chunks * H * 4 * 4);
  l.decay = o; o = up256(o + chunks * H * 8);
  l.seg_state = o; o = up256(o + room * H * P * NS * 4);
  l.seg_decay = o; o = up256(o + room * H * 8);
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
  g.gate = reinterpret_cast<float*>(w + l.gate);
  g.block = reinterpret_cast<float*>(w + l.block);
  g.decay = reinterpret_cast<double*>(w + l.decay);
  g.seg_state = reinterpret_cast<float*>(w + l.seg_state);
  g.seg_decay = reinterpret_cast<double*>(w + l.seg_decay);
  g.seg = (int)l.seg;
  g.wait_ns = debug_opts().wait_limit_us ? (uint64_t)debug_opts().wait_limit_us * 1000ull
                                         : gdn::kWaitLimitNs;
  const auto skip = [](int fault) {
    return debug_opts().fault == fault ? debug_opts().fault_chunk : -1;
  };
  g.skip_bc = skip(GDN_FAULT_SKIP_SSM_PRODUCT);
  g.skip_seg = skip(GDN_FAULT_SKIP_SSM_SEG_LOAD);
  g.skip_main = skip(GDN_FAULT_SKIP_SSM_LOAD);
  const unsigned pairs = a.G * (((a.H / a.G) * (a.P / 64) + 1) / 2);
  const unsigned roles = a.G + (a.H + gdn::kGateHeads - 1) / gdn::kGateHeads;
  cudaError_t e = launch_tc(false, gdn::ssm_bc_kernel, (unsigned)(a.T / gdn::kL + a.N) * roles, 512,
                            gdn::kBcSmem, s, g, "ssm_bc");
  if (e == cudaSuccess && a.T > l.seg * gdn::kL)  // a sequence may have several segments
    e = launch_tc(true, gdn::ssm_seg_kernel, (unsigned)(a.T / (l.seg * gdn::kL)) * pairs, 512,
                  gdn::kSegSmem, s, g, "ssm_seg");
  if (e == cudaSuccess)
    e = launch_tc(true, gdn::ssm_main_kernel, (unsigned)l.units * pairs, 512, gdn::kMainSmem, s, g,
                  "ssm_main");
  return e;
}

}  // namespace gdn_host
