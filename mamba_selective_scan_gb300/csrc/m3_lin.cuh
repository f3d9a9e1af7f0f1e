// m3_lin.cuh -- linear attention with a decay for each head: argument structs
// and the entry points the translation units provide to each other.
//
// Per batch row and value head, S in R^{head_k x head_v}, lam = exp(log_decay):
//
//   S_t = lam S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// The gradients are three passes of the same form, two of them backwards in
// time (dS_t the adjoint of S_t):
//
//   dq_t = scale S_t d_o_t                                 S^T from keys v, values k, queries d_o
//   dS_t = lam dS_{t+1} + scale q_t d_o_t^T,  dv_t = dS_t^T k_t,  dk_t = dS_t v_t
//
// so every kernel here runs a list of passes (queries, keys, values, outputs).
// A pass in time takes its start state as S_{-1}, the state before the first
// token; one backwards takes d S_{T-1} without its last token's own share, so
// that the start enters the first token's output with lam^0, and it ends with
// lam dS_0, the gradient of S_{-1}.
#pragma once

#include "m3_common.cuh"

namespace m3 {

constexpr int LIN_DMAX = 128;         // head_k and head_v, at most
constexpr float LIN_LD_MIN = -150.0f; // exp(-150) is 0 in f32: lower log decays (and -inf) count as this

struct LinPass {
  const void *q, *k, *v;
  void* out;
  const float* s_in;     // NULL = zero
  float* s_out;          // NULL = not wanted
  int64_t qs, ks, vs, os;  // elements between tokens
  int qh, kh, vh;          // value heads that share a head of each (outputs have one of their own)
  int DK, DV;              // sizes of the pass's keys and values
  bool rev;                // backwards in time
  bool st;                 // states are given transposed, [DV][DK]
  bool out_f32;            // outputs are f32 whatever the activations
};

struct LinArgs {
  LinPass p[3];
  const float* ld;  // [Hv] log decays
  int np, B, T, Hv;
  float scale;
  unsigned* status;
  int nc;                // chunks of a sequence
  bool stream;           // tensor-core kernels: equal shares of all items' chunks, one block per SM
  unsigned* flags;       // stream: per block, set once it handed on its state (in seg_start)
  int segs, seg_chunks;  // else: time segments, chunks per segment
  float *seg_end, *seg_start;  // [items][segs][128][128]: ends from a zero start, start states; stream: seg_start [blocks][128][128]
};
constexpr int LIN_C = 64;  // tokens per chunk
// The SMs of a GB300.  Plans are made for them, without a device, so that a
// plan's bytes are the same wherever it is made; a launch takes the SMs that
// there are, and no more blocks of equal shares than these.
constexpr int LIN_SMS = 152;

// (a comparison, not fmaxf: a decay that is NaN stays one)
__device__ __forceinline__ float lin_ld(float x) { return x < LIN_LD_MIN ? LIN_LD_MIN : x; }

// A decay over n tokens as near + off.  Rounded to one f32 value, a slow decay
// is off by up to 2^-25 of the state each time it is applied, always the same
// way: 16384 tokens that hardly fade were off by 2e-4.  So a decay above a half
// is 1 + (exp - 1), the second term with f32's relative precision.
struct LinDecay {
  float near, off;
};
__device__ __forceinline__ LinDecay lin_decay(float ld, int n) {
  const float x = lin_ld(ld) * (float)n;
  return x > -0.6f && x < 0.6f ? LinDecay{1.0f, expm1f(x)} : LinDecay{expf(x), 0.0f};
}

// Token after token, any type and length: m3_lin_rec.cu
template <typename T> cudaError_t launch_lin_rec(LinArgs a, cudaStream_t st, int sms);
// The start states of time segments from the ends that the kernel before left: m3_lin_tc.cu
cudaError_t launch_lin_seg(const LinArgs& a, cudaStream_t st);

// bf16, chunks of 64 on the tensor cores: m3_lin_tc.cu
cudaError_t launch_lin_tc(const LinArgs& a, cudaStream_t st, int sms);
cudaError_t take_lin_status(unsigned* out);

// f32 shares of shared heads, added in order: m3_lin_rec.cu
struct LinShare {
  const float* part[2];  // [B T][Hv][D], of dq and dk
  void* out[2];
  int64_t os[2];
  int64_t tokens;
  int Hk, share, D;
};
template <typename T> cudaError_t launch_lin_share(const LinShare& a, cudaStream_t st);

}  // namespace m3
