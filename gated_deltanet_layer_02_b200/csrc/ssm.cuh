// ssm.cuh -- parts shared by the kernels of the state space layer (ssm.cu, ssm_tc.cu).
#pragma once
#include <cuda_fp16.h>

#include "args.cuh"
#include "common.cuh"

namespace gdn {

// Selective state space layer: packed prefill, and one token per sequence (N = T).
struct SsmArgs {
  const void* x;         // [T][Cc] pre-conv rows [x | B | C]
  const void* conv_w;    // [Cc][4]
  const void* conv_b;    // [Cc] or NULL
  const float* dt;       // [T][H]
  const float* dt_bias;  // [H] or NULL
  const float* a_log;    // [H]
  const float* D;        // [H] or NULL
  const void* z;         // [T][H][P] or NULL
  const int32_t* cu;     // [N+1] (prompts)
  const void* S0;        // initial states, or NULL
  void* SN;              // final states, or NULL (may be S0)
  const void* conv0;
  void* convN;
  void* out;
  const int32_t* slot;   // [N] state-pool rows, or NULL (= n)
  int32_t* status;
  float* u;              // workspace: [T][Cc] conv outputs, fp32
  int num_slots;
  int N, T, H, G, P, Cc;
  float dt_min, dt_max;
};

// 32 bytes in one store (p 32-byte aligned).
__device__ __forceinline__ void store32(void* p, const uint4& lo, const uint4& hi) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(lo.x), "r"(lo.y),
               "r"(lo.z), "r"(lo.w), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
               : "memory");
}

// Tokens [s, e) of sequence n.  Entries of cu that are out of order or past T give an empty range
// and GDN_ERR_INVALID_ARG.
__device__ __forceinline__ void seq_range(const SsmArgs& a, int n, int& s, int& e) {
  s = __ldg(a.cu + n);
  e = __ldg(a.cu + n + 1);
  if (s < 0 || e < s || e > a.T) {
    report_status(a.status, GDN_ERR_INVALID_ARG);
    s = e = 0;
  }
}

// softplus(v) = max(v, 0) + log1p(exp(-|v|)), within [lo, hi]; a NaN stays one
__device__ __forceinline__ float ssm_step(float v, float lo, float hi) {
  const float sp = fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
  return sp < lo ? lo : (sp > hi ? hi : sp);
}

// exp(a_log), held at 2.3e38 (finite in log2 too): past it a token with a step forgets all before
// it, and one without a step nothing (0 times an infinity would be NaN).  A NaN stays one.
__device__ __forceinline__ float ssm_rate(float a_log) {
  const float r = expf(a_log);
  return r > 2.3e38f ? 2.3e38f : r;
}

template <typename T>
__device__ __forceinline__ void load8_or_zero(const T* p, float (&v)[8]) {
  if (p) {
    load8(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  }
}

// Taps of 8 channels ([c][4] in memory) by tap, and their bias.
template <typename T>
__device__ __forceinline__ void load_taps(const SsmArgs& a, int c, float (&w)[4][8],
                                          float (&b)[8]) {
  const T* p = static_cast<const T*>(a.conv_w) + (size_t)c * 4;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
    load8(p + 8 * q, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e & 3][2 * q + (e >> 2)] = v[e];
  }
  load8_or_zero(a.conv_b ? static_cast<const T*>(a.conv_b) + c : nullptr, b);
}

// Final conv history of sequence n (tokens [s, end), pool row `row`): the last three rows of its
// history followed by its tokens.  Block k of the sequence's nb blocks takes its share of the
// channels; a thread reads its 8 channels before it writes them, so convN may be conv0 (the conv,
// which reads conv0 too, has finished).
template <typename T>
__device__ __forceinline__ void conv_history(const SsmArgs& a, int n, int row, int s, int end,
                                             int k, int nb) {
  if (!a.convN || row < 0) return;
  const T* c0 = static_cast<const T*>(a.conv0);
  for (int c = (k * (int)blockDim.x + (int)threadIdx.x) * 8; c < a.Cc;
       c += nb * (int)blockDim.x * 8) {
    float r[3][8];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int t = end - 3 + j;  // may lie before the sequence
      load8_or_zero(t >= s ? static_cast<const T*>(a.x) + (size_t)t * a.Cc + c
                           : (c0 ? c0 + ((size_t)row * 3 + 3 + t - s) * a.Cc + c : nullptr),
                    r[j]);
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
      store8(static_cast<T*>(a.convN) + ((size_t)row * 3 + j) * a.Cc + c, r[j]);
  }
}

// Arguments of the tensor-core prefill (ssm_tc.cu).  Per chunk of 128 tokens and group:
struct SsmTcArgs {
  SsmArgs a;
  uint8_t* tiles;        // C, B high, B low (fp16): [128][128] each, as swizzled row tiles
  __half* cb;            // [128][128] C B^T (see cb_off), blocks of 32 columns up to the diagonal
  int8_t* ex;            // [2][128] exponents of the rows of B and of C
  __nv_bfloat16* hist;   // [N][3][Cc] initial conv history (NULL: zeros)
  float* gate;           // per chunk and head: [3][128] w, log2(delta) - cum, cum (see gates)
  float* block;          // per chunk and head: [4] log2 decays of the blocks of 32 tokens
  double* decay;         // per chunk and head: log2 of its decay
  float* seg_state;      // [segments][H][P][NS] state added by each segment
  double* seg_decay;     // [segments][H] log2 of its decay
  uint64_t wait_ns;
  int NS, seg;           // state width; chunks per segment
  int skip_bc, skip_seg, skip_main;  // debug fault injection: the product (bc) or the tiles' copy that
                                     // the first CTA leaves out, counted in its own, or -1
};

}  // namespace gdn
