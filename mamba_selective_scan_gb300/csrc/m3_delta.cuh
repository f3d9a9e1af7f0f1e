// m3_delta.cuh -- gated delta rule: argument structs, the launch plan and the
// entry points the translation units provide to each other.
//
// Per batch row and value head, S in R^{head_k x head_v}:
//
//   S' = exp(g_t) S_{t-1};  u = beta_t (v_t - S'^T k_t);  S_t = S' + k_t u^T
//   o_t = scale S_t^T q_t
//
// Over a chunk of C tokens with gam = cumsum(g), D_ij = exp(gam_i - gam_j):
//
//   A_ij = beta_i D_ij k_i.k_j (j < i),  T = (I + A)^-1
//   E = V - exp(gam) (K S0),  U = T (beta E)
//   O = scale (exp(gam) (Q S0) + (D o Q K^T) U)
//   S_end = exp(gam_C) S0 + (exp(gam_C - gam) K)^T U
#pragma once

#include "m3_common.cuh"

namespace m3 {

// Per chunk and head, bf16 [16-byte unit][128 rows (head_v)][8], a layout of
// shared-memory operands, so that one bulk copy brings them in ready to use:
constexpr size_t TC_PREP = 33920;  // T, P and the per-token factors (TcPrep)
constexpr size_t TC_CKPT = 65536 + TC_PREP;  // the forward's: S^T, U^T hi, U^T lo, TcPrep
constexpr size_t TC_BWD = 98304;   // the reverse pass's: dS^T hi, lo, dR^T hi, lo
constexpr size_t F32_KEPT = 155904;  // per chunk of 32 and head, between the kernels of the f32 backward
constexpr int TC = 64;             // tokens per chunk of the tensor-core kernels
constexpr int TC_BLOCKS = 152;     // persistent blocks of the gradients' kernel, at most (the SMs of a GB300)
constexpr int DMAX = 128;          // head_k and head_v, at most
constexpr float DELTA_L2_EPS = 1e-6f;  // added to the sum of squares of q and of k
constexpr float G_MIN = -110.0f;       // exp(-110) is 0 in f32: lower log decays (and -inf) count as this

struct DeltaArgs {
  const void *q, *k, *v, *g, *beta, *d_o;
  const float *s_in, *ckpt_in, *ds_out;  // state in, checkpoints and d(state out) of the backward
  void *o, *dq, *dk, *dv, *dg, *dbeta;
  float *s_out, *ckpt, *ds_in;
  float *pdq, *pdk;  // f32, shared heads: per-value-head shares of dq, dk [B, T, Hv, dk]
  int64_t qs, ks, vs, dqs, dks, dvs;  // elements between tokens
  int B, T, Hk, Hv, DK, DV, share;
  int chunk, nc;
  float scale;
  int l2;
  bool stream;           // tensor-core kernels: equal shares of all heads' chunks, one block per SM
  unsigned* flags;       // stream: [B Hv], set once a head's state was handed over (in seg_start)
  int segs, seg_chunks;  // else: time segments, chunks per segment
  float *seg_end, *seg_phi, *seg_start;  // [B Hv][segs][128][128]: zero-start ends, transitions, start states
  float* seg_keep;     // with checkpoints: the transitions' transposes, which are the adjoint's transitions
  unsigned char* bwd;  // [B Hv][nc] of TC_BWD (f32: F32_KEPT) bytes
  unsigned char* tp;   // TcPrep of every chunk, tp_stride bytes apart (in the checkpoints, or the workspace)
  size_t tp_stride;
  unsigned* status;
};

struct DeltaPlan {
  int B, T, Hk, Hv, DK, DV, chunk, nc;
  size_t ckpt_bytes, fwd_ws_bytes, ws_bytes;  // (the forward's part comes first)
  size_t o_pdq, o_pdk, o_end, o_phi, o_start, o_bwd, o_flags, o_tp;  // workspace offsets
  size_t o_keep;  // in the checkpoints
  bool stream;           // more heads than SMs: equal shares instead of segments
  int segs, seg_chunks;  // time segments
  int fwd_launches, bwd_launches;
};

// SM count of the current device (a property that never changes: kept)
cudaError_t sm_count(int* sms);

// (a comparison, not fmaxf: a gate that is NaN stays one)
__device__ __forceinline__ float clamp_g(float g) { return g < G_MIN ? G_MIN : g; }

// A chunk's gates are summed in two f32 terms: each forgetting token brings up
// to 110, so that in one term the small decays between such tokens would be
// differences of numbers in the thousands (errors to 2e-4).  A decay is then
// e^{h_i - h_j} (1 + l_i) (1 - l_j): h_i - h_j is exact where it is small, and
// |l| stays below 2^-10, so the linear factor is good to f32's rounding (l in
// powers of e) and goes into the tokens' own factors.
struct GateSum {
  float h, l;
};
__device__ __forceinline__ GateSum gate_add(GateSum a, GateSum b) {
  const float s = a.h + b.h, t = s - a.h, e = ((a.h - (s - t)) + (b.h - t)) + (a.l + b.l), h = s + e;
  return {h, e - (h - s)};
}
// lane i's sum over the lanes up to i
__device__ __forceinline__ GateSum gate_scan(GateSum v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const GateSum up = {__shfl_up_sync(~0u, v.h, o), __shfl_up_sync(~0u, v.l, o)};
    if (lane >= o) v = gate_add(up, v);
  }
  return v;
}

// Forward by the recurrence itself, token after token (any length and type;
// decoding): provided by m3_delta_rec.cu
template <typename T> cudaError_t launch_delta_rec(const DeltaArgs& a, cudaStream_t st, int sms);
// Backward of f32 activations from the checkpoints: m3_delta_bwd.cu
cudaError_t launch_delta_bwd(const DeltaArgs& a, cudaStream_t st);
// and the sum of its per-value-head shares of dq and dk
cudaError_t launch_delta_share(const DeltaArgs& a, cudaStream_t st);

// bf16 activations, chunks of 64 on the tensor cores: T, P and factors of
// every chunk, then the forward
cudaError_t launch_delta_tc_prep(const DeltaArgs& a, cudaStream_t st);
cudaError_t take_delta_prep_status(unsigned* out);
cudaError_t launch_delta_tc_fwd(const DeltaArgs& a, cudaStream_t st);
// Tensor map of a [B, T, H, D] bf16 tensor (`stride` elements between
// tokens) read in tiles of 64 tokens x 64 columns, 128-byte swizzle
// (of an f32 tensor: 64 tokens x 32 columns)
bool delta_tile_map(CUtensorMap* map, const void* ptr, int D, int H, int64_t T, int64_t B, int64_t stride, bool f32 = false);
cudaError_t launch_delta_seg(const DeltaArgs& a, const float* first, bool rev, cudaStream_t st);
cudaError_t take_delta_fwd_status(unsigned* out);
// Its backward: the reverse pass over the chunks, then every chunk's gradients
cudaError_t launch_delta_tc_rev(const DeltaArgs& a, cudaStream_t st);
cudaError_t launch_delta_tc_grad(const DeltaArgs& a, cudaStream_t st);
cudaError_t take_delta_bwd_status(unsigned* out);

}  // namespace m3
