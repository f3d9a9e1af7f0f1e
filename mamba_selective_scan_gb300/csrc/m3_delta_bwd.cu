// m3_delta_bwd.cu -- backward of the gated delta rule in f32 arithmetic, and
// the sum over the value heads that share a key head.
//
// With a chunk's start state S0 from the checkpoint, gam, D as in
// m3_delta.cuh, k and q normalised, P = scale D o QK^T and the adjoint dS of
// the state after it:
//
//   prep    E = V - e^gam (K S0), T = (I + A)^-1, U = T (beta E)
//   rev     dU = P^T dO + (e^{gam_C - gam} K) dS,   dR = T^T dU,   dV = beta dR
//           dS0 = e^{gam_C} dS + scale (e^gam Q)^T dO - (beta e^gam K)^T dR
//   grad    dA = -(dR U^T) below the diagonal,      dP = dO U^T on and below it
//           dQ = scale e^gam dO S0^T + (scale dP o D) K
//           dK = e^{gam_C - gam} U dS^T - beta e^gam dR S0^T
//                + (scale dP o D)^T Q + (dA beta D) K + (dA beta D)^T K
//
// and each exponent gam_i that a term carries takes that term's share; dg is
// their sum from the end of the chunk.  Only rev goes from chunk to chunk:
// prep and grad run over all chunks at once, what they share with rev is in
// the workspace.  8 x 128 x 4 heads of 128 x 128: 17, 50 and 43 us, bound by
// latency (128 blocks, four chunks one after the other in rev).  With 128
// columns per block in rev (32 blocks) the training pass took 174 us instead of
// 141.
#include "m3_delta.cuh"

namespace m3 {

namespace {
constexpr int C = 32;         // tokens per chunk (the checkpoint interval)
constexpr int LD = DMAX + 4;  // row length of the [C][128] arrays: float4 columns, rows 4 banks apart
constexpr int LS = C + 1;     // row length of the [C][C] arrays

// what the kernels hand on, per chunk and head
struct Kept {
  float K[C][DMAX], Q[C][DMAX], E[C][DMAX], U[C][DMAX], dR[C][DMAX];  // K, Q normalised
  float T[C][C], P[C][C];
  float nk[C], nq[C];
  float dS[DMAX][DMAX];
};
static_assert(sizeof(Kept) == F32_KEPT, "the workspace's share");

struct Gates {
  float gam[C], lo[C], beta[C], eg[C], el[C];  // gam + lo: the gates' sum; el = e^{gam_C - gam}
  __device__ __forceinline__ float decay(int i, int j) const { return expf(gam[i] - gam[j]) * (1.0f + (lo[i] - lo[j])); }
};
struct PrepSmem {
  float K[C][LD], Q[C][LD], E[C][LD];
  float S0[64][LD];
  float A[C][LS], P[C][LS], Ti[C][LS];
  Gates g;
};
constexpr int RV = 32, LR = RV + 4;  // columns of dS per block of the reverse pass
struct RevSmem {
  float K[C][LD], Q[C][LD];
  float dO[C][LR], dU[C][LR], dR[C][LR], dS[DMAX][LR];
  float P[C][LS], Ti[C][LS];
  Gates g;
};
struct GradSmem {
  float K[C][LD], Q[C][LD], dO[C][LD], U[C][LD], dR[C][LD], E[C][LD];
  float S0[64][LD], dS[64][LD];
  float A[C][LS], P[C][LS], X[C][LS];
  float dgam[C], dbeta[C], nq[C], nk[C];
  float red[8];
  Gates g;
};

__device__ __forceinline__ float wsum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}
__device__ __forceinline__ const float4& f4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4& f4(float* p) { return *reinterpret_cast<float4*>(p); }
__device__ __forceinline__ void axpy4(float4& o, float s, float4 x) {
  o.x = fmaf(s, x.x, o.x); o.y = fmaf(s, x.y, o.y); o.z = fmaf(s, x.z, o.z); o.w = fmaf(s, x.w, o.w);
}

// where a block's chunk is
struct Place {
  int bh, b, h, hk, ch, n;
  int64_t tok0;
  __device__ __forceinline__ Place(const DeltaArgs& a, int bh_, int ch_) : bh(bh_), ch(ch_) {
    b = bh / a.Hv;
    h = bh % a.Hv;
    hk = h / a.share;
    n = min(C, a.T - ch * C);
    tok0 = (int64_t)b * a.T + ch * C;
  }
};
__device__ __forceinline__ Kept& kept(const DeltaArgs& a, const Place& p) {
  return reinterpret_cast<Kept*>(a.bwd)[(size_t)p.bh * a.nc + p.ch];
}
// rows [C][width <= 128] of a [.., H, D] array, zeros past the sequence and
// the head (256 threads)
__device__ __forceinline__ void load_rows(float (*to)[LD], const float* from, int64_t stride, int D, int n, int tid) {
#pragma unroll
  for (int i = 0; i < C * DMAX / 4 / 256; ++i) {
    const int e = tid + i * 256, r = e >> 5, c = (e & 31) * 4;
    f4(&to[r][c]) = r < n && c < D ? f4(from + r * stride + c) : make_float4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void load_kept(float (*to)[LD], const float (*from)[DMAX], int rows, int tid) {
  for (int e = tid; e < rows * DMAX / 4; e += 256) f4(&to[e >> 5][(e & 31) * 4]) = f4(&from[e >> 5][(e & 31) * 4]);
}
__device__ __forceinline__ void store_kept(float (*to)[DMAX], const float (*from)[LD], int tid) {
  for (int e = tid; e < C * DMAX / 4; e += 256) f4(&to[e >> 5][(e & 31) * 4]) = f4(&from[e >> 5][(e & 31) * 4]);
}
// 64 rows of a state [head_k][head_v]
__device__ __forceinline__ void load_half(float (*to)[LD], const float* S, int half, const DeltaArgs& a, int tid) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = tid + i * 256, k = e >> 5, v = (e & 31) * 4, kk = half * 64 + k;
    f4(&to[k][v]) = kk < a.DK && v < a.DV ? f4(S + (size_t)kk * a.DV + v) : make_float4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void load_gates(Gates& s, const DeltaArgs& a, const Place& p, int lane) {  // one warp
  const bool ok = lane < p.n;
  const int64_t at = (p.tok0 + lane) * a.Hv + p.h;
  const GateSum g = gate_scan({ok ? clamp_g(static_cast<const float*>(a.g)[at]) : 0.0f, 0.0f}, lane);
  s.beta[lane] = ok ? static_cast<const float*>(a.beta)[at] : 0.0f;
  s.gam[lane] = g.h;
  s.lo[lane] = g.l;
  s.eg[lane] = expf(g.h) * (1.0f + g.l);
  s.el[lane] = expf(__shfl_sync(~0u, g.h, 31) - g.h) * (1.0f + (__shfl_sync(~0u, g.l, 31) - g.l));
}
__device__ __forceinline__ const float* start_state(const DeltaArgs& a, const Place& p) {
  return a.ckpt_in + ((size_t)p.bh * a.nc + p.ch) * a.DK * a.DV;
}
}  // namespace

// Blocks of 8 warps.  Every warp owns four rows of a chunk; a lane four
// columns, side by side where a product's sum runs over rows, 32 apart where
// it runs along a row.
__global__ void __launch_bounds__(256) m3_delta_bwd_prep_kernel(const __grid_constant__ DeltaArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  PrepSmem& s = *reinterpret_cast<PrepSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = warp * 4, c0 = lane * 4;
  const Place p(a, blockIdx.x / a.nc, blockIdx.x % a.nc);
  Kept& out = kept(a, p);
  const float* S0 = start_state(a, p);
  load_rows(s.K, static_cast<const float*>(a.k) + p.tok0 * a.ks + (int64_t)p.hk * a.DK, a.ks, a.DK, p.n, tid);
  load_rows(s.Q, static_cast<const float*>(a.q) + p.tok0 * a.qs + (int64_t)p.hk * a.DK, a.qs, a.DK, p.n, tid);
  load_rows(s.E, static_cast<const float*>(a.v) + p.tok0 * a.vs + (int64_t)p.h * a.DV, a.vs, a.DV, p.n, tid);
  load_half(s.S0, S0, 0, a, tid);
  if (warp == 0) load_gates(s.g, a, p, lane);
  __syncthreads();
  // normalise the rows of K and Q
#pragma unroll
  for (int r = r0; r < r0 + 4; ++r) {
    float4& k4 = f4(&s.K[r][c0]);
    float4& q4 = f4(&s.Q[r][c0]);
    float nk = 1.0f, nq = 1.0f;
    if (a.l2) {
      nk = rsqrtf(wsum(dot4(k4, k4, 0.0f)) + DELTA_L2_EPS);
      nq = rsqrtf(wsum(dot4(q4, q4, 0.0f)) + DELTA_L2_EPS);
      k4.x *= nk; k4.y *= nk; k4.z *= nk; k4.w *= nk;
      q4.x *= nq; q4.y *= nq; q4.z *= nq; q4.w *= nq;
    }
    f4(&out.K[r][c0]) = k4;
    f4(&out.Q[r][c0]) = q4;
    if (lane == 0) {
      out.nk[r] = nk;
      out.nq[r] = nq;
    }
  }
  __syncthreads();
  {  // A, P: row i of a warp, column j = lane
    float kk[4] = {0, 0, 0, 0}, qk[4] = {0, 0, 0, 0};
    for (int c = 0; c < DMAX; c += 4) {
      const float4 kj = f4(&s.K[lane][c]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kk[i] = dot4(f4(&s.K[r0 + i][c]), kj, kk[i]);
        qk[i] = dot4(f4(&s.Q[r0 + i][c]), kj, qk[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i;
      const float D = lane <= r ? s.g.decay(r, lane) : 0.0f;
      const float P = a.scale * D * qk[i];
      s.P[r][lane] = P;
      out.P[r][lane] = P;
      s.A[r][lane] = lane < r ? s.g.beta[r] * D * kk[i] : 0.0f;
    }
  }
  {  // E -= e^gam (K S0)
    float4 acc[4] = {};
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      if (half) {
        __syncthreads();
        load_half(s.S0, S0, 1, a, tid);
        __syncthreads();
      }
#pragma unroll 8
      for (int k = 0; k < 64; ++k) {
        const float4 sv = f4(&s.S0[k][c0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) axpy4(acc[i], s.K[r0 + i][half * 64 + k], sv);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 e = f4(&s.E[r0 + i][c0]);
      axpy4(e, -s.g.eg[r0 + i], acc[i]);
      f4(&s.E[r0 + i][c0]) = e;
      f4(&out.E[r0 + i][c0]) = e;
    }
  }
  __syncthreads();
  // T = (I + A)^-1 by forward substitution, a column per lane
  if (warp == 0) {
    float x[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float t0 = i == lane ? 1.0f : 0.0f, t1 = 0.0f;
#pragma unroll
      for (int l = 0; l < i; ++l) (l & 1 ? t1 : t0) = fmaf(-s.A[i][l], x[l], l & 1 ? t1 : t0);
      x[i] = t0 + t1;
      s.Ti[i][lane] = x[i];
      out.T[i][lane] = x[i];
    }
  }
  __syncthreads();
  {  // U = T (beta E)
    float4 u[4] = {};
    for (int j = 0; j < C; ++j) {
      const float4 e = f4(&s.E[j][c0]);
      const float bj = s.g.beta[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) axpy4(u[i], s.Ti[r0 + i][j] * bj, e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f4(&out.U[r0 + i][c0]) = u[i];
  }
}

// Chunks last to first, 32 of dS's columns per block in shared memory (the
// columns never meet).  A thread has a row of the chunk, and four rows of dS,
// in four columns.
__global__ void __launch_bounds__(256) m3_delta_bwd_rev_kernel(const __grid_constant__ DeltaArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  RevSmem& s = *reinterpret_cast<RevSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x, v0 = blockIdx.y * RV;
  const int r = tid >> 3, c0 = (tid & 7) * 4, k0 = r * 4;
  const bool vok = v0 + c0 < a.DV;
  float4 d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d[i] = a.ds_out && vok && k0 + i < a.DK ? f4(a.ds_out + ((size_t)bh * a.DK + k0 + i) * a.DV + v0 + c0)
                                            : make_float4(0, 0, 0, 0);
    f4(&s.dS[k0 + i][c0]) = d[i];
  }
  for (int ch = a.nc - 1; ch >= 0; --ch) {
    const Place p(a, bh, ch);
    Kept& kp = kept(a, p);
    __syncthreads();
    load_kept(s.K, kp.K, C, tid);
    load_kept(s.Q, kp.Q, C, tid);
    f4(&s.dO[r][c0]) = r < p.n && vok ? f4(static_cast<const float*>(a.d_o) + ((p.tok0 + r) * a.Hv + p.h) * a.DV + v0 + c0)
                                      : make_float4(0, 0, 0, 0);
    for (int e = tid; e < C * C; e += 256) {
      s.P[e >> 5][e & 31] = kp.P[e >> 5][e & 31];
      s.Ti[e >> 5][e & 31] = kp.T[e >> 5][e & 31];
    }
    if (warp == 0) load_gates(s.g, a, p, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) f4(&kp.dS[k0 + i][v0 + c0]) = d[i];
    __syncthreads();
    {  // dU = P^T dO + (e^{gam_C - gam} K) dS
      float4 u = make_float4(0, 0, 0, 0), w = u;
#pragma unroll 8
      for (int j = 0; j < C; ++j) axpy4(u, s.P[j][r], f4(&s.dO[j][c0]));
#pragma unroll 4
      for (int k = 0; k < DMAX; k += 4) {
        const float4 kr = f4(&s.K[r][k]);
        axpy4(w, kr.x, f4(&s.dS[k][c0]));
        axpy4(w, kr.y, f4(&s.dS[k + 1][c0]));
        axpy4(w, kr.z, f4(&s.dS[k + 2][c0]));
        axpy4(w, kr.w, f4(&s.dS[k + 3][c0]));
      }
      axpy4(u, s.g.el[r], w);
      f4(&s.dU[r][c0]) = u;
    }
    __syncthreads();
    {  // dR = T^T dU;  dV = beta dR
      float4 x = make_float4(0, 0, 0, 0);
#pragma unroll 8
      for (int j = 0; j < C; ++j) axpy4(x, s.Ti[j][r], f4(&s.dU[j][c0]));
      f4(&kp.dR[r][v0 + c0]) = x;
      const float bt = s.g.beta[r];
      x = make_float4(bt * x.x, bt * x.y, bt * x.z, bt * x.w);
      f4(&s.dR[r][c0]) = x;  // beta dR
      if (r < p.n && vok) f4(static_cast<float*>(a.dv) + (p.tok0 + r) * a.dvs + (int64_t)p.h * a.DV + v0 + c0) = x;
    }
    __syncthreads();
    {  // dS0
      const float ec = s.g.eg[C - 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = make_float4(ec * d[i].x, ec * d[i].y, ec * d[i].z, ec * d[i].w);
#pragma unroll 4
      for (int j = 0; j < C; ++j) {
        const float4 o = f4(&s.dO[j][c0]), x = f4(&s.dR[j][c0]);
        const float4 q = f4(&s.Q[j][k0]), k = f4(&s.K[j][k0]);
        const float fq = a.scale * s.g.eg[j], fk = -s.g.eg[j];
        axpy4(d[0], fq * q.x, o); axpy4(d[1], fq * q.y, o); axpy4(d[2], fq * q.z, o); axpy4(d[3], fq * q.w, o);
        axpy4(d[0], fk * k.x, x); axpy4(d[1], fk * k.y, x); axpy4(d[2], fk * k.z, x); axpy4(d[3], fk * k.w, x);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) f4(&s.dS[k0 + i][c0]) = d[i];
    }
  }
  if (a.ds_in && vok) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i < a.DK) f4(a.ds_in + ((size_t)bh * a.DK + k0 + i) * a.DV + v0 + c0) = d[i];
  }
}

__global__ void __launch_bounds__(256) m3_delta_bwd_grad_kernel(const __grid_constant__ DeltaArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  GradSmem& s = *reinterpret_cast<GradSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = warp * 4, c0 = lane * 4;
  const Place p(a, blockIdx.x / a.nc, blockIdx.x % a.nc);
  const Kept& kp = kept(a, p);
  const float* S0 = start_state(a, p);
  load_kept(s.K, kp.K, C, tid);
  load_kept(s.Q, kp.Q, C, tid);
  load_kept(s.U, kp.U, C, tid);
  load_kept(s.dR, kp.dR, C, tid);
  load_kept(s.E, kp.E, C, tid);
  load_rows(s.dO, static_cast<const float*>(a.d_o) + (p.tok0 * a.Hv + p.h) * a.DV, (int64_t)a.Hv * a.DV, a.DV, p.n, tid);
  for (int e = tid; e < C * C; e += 256) s.P[e >> 5][e & 31] = kp.P[e >> 5][e & 31];
  if (warp == 0) {
    load_gates(s.g, a, p, lane);
    s.nk[lane] = kp.nk[lane];
    s.nq[lane] = kp.nq[lane];
  }
  __syncthreads();
  // dA and dP (row i of a warp, column j = lane); A and P become dA beta D
  // and scale dP D
  {
    float kk[4] = {0, 0, 0, 0}, da[4] = {0, 0, 0, 0}, dp[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int c = 0; c < DMAX; c += 4) {
      const float4 uj = f4(&s.U[lane][c]), kj = f4(&s.K[lane][c]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        da[i] = dot4(f4(&s.dR[r0 + i][c]), uj, da[i]);
        dp[i] = dot4(f4(&s.dO[r0 + i][c]), uj, dp[i]);
        kk[i] = dot4(f4(&s.K[r0 + i][c]), kj, kk[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i;
      const float D = lane <= r ? s.g.decay(r, lane) : 0.0f, be = s.g.beta[r];
      const float xa = lane < r ? -da[i] : 0.0f, xp = lane <= r ? dp[i] : 0.0f;
      const float dk = xa * D * kk[i], m = dk * be + xp * s.P[r][lane];
      // A carries beta_r: its derivative is taken with A / beta_r = D k_r.k_j
      const float db = wsum(dk) + wsum(dot4(f4(&s.dR[r][c0]), f4(&s.E[r][c0]), 0.0f));
      const float row = wsum(m);
      if (lane == 0) {
        s.dbeta[r] = db;
        s.dgam[r] = row;
      }
      s.X[r][lane] = m;
      s.A[r][lane] = xa * be * D;
      s.P[r][lane] = xp * a.scale * D;
    }
  }
  __syncthreads();
  if (warp == 0) {
    float col = 0.0f;
    for (int i = lane; i < C; ++i) col += s.X[i][lane];
    s.dgam[lane] -= col;
  }
  // the products with the states (rows of a warp; columns lane + 32 m) and <dS, S0>
  float os[4][4] = {}, us[4][4] = {}, rs[4][4] = {};
  float inner = 0.0f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncthreads();
    load_half(s.S0, S0, half, a, tid);
    for (int e = tid; e < 64 * DMAX / 4; e += 256) {
      const int k = e >> 5, v = (e & 31) * 4;
      const float4 d = f4(&kp.dS[half * 64 + k][v]);
      f4(&s.dS[k][v]) = d;
      inner = dot4(d, f4(&s.S0[k][v]), inner);  // (this thread's own element of S0)
    }
    __syncthreads();
#pragma unroll 2
    for (int v = 0; v < DMAX; v += 4) {
      float4 sv[2], dv[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        sv[m] = f4(&s.S0[lane + 32 * m][v]);
        dv[m] = f4(&s.dS[lane + 32 * m][v]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 o = f4(&s.dO[r0 + i][v]), u = f4(&s.U[r0 + i][v]), r = f4(&s.dR[r0 + i][v]);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          os[i][half * 2 + m] = dot4(o, sv[m], os[i][half * 2 + m]);
          us[i][half * 2 + m] = dot4(u, dv[m], us[i][half * 2 + m]);
          rs[i][half * 2 + m] = dot4(r, sv[m], rs[i][half * 2 + m]);
        }
      }
    }
  }
  // dQ, dK, the rest of dgam
  float dqr[4][4], dkr[4][4];
  float wtot = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i;
    float dq_ = 0.0f, dk_ = 0.0f, dw_ = 0.0f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int k = lane + 32 * m;
      dqr[i][m] = a.scale * s.g.eg[r] * os[i][m];
      const float x = -s.g.beta[r] * s.g.eg[r] * rs[i][m], w = s.g.el[r] * us[i][m];
      dkr[i][m] = x + w;
      dq_ = fmaf(dqr[i][m], s.Q[r][k], dq_);
      dk_ = fmaf(x, s.K[r][k], dk_);
      dw_ = fmaf(w, s.K[r][k], dw_);
    }
    const float own = wsum(dq_ + dk_), w = wsum(dw_);
    wtot += w;
    if (lane == 0) s.dgam[r] += own - w;
  }
#pragma unroll 2
  for (int j = 0; j < C; ++j) {
    float kj[4], qj[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      kj[m] = s.K[j][lane + 32 * m];
      qj[m] = s.Q[j][lane + 32 * m];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i;
      const float pq = s.P[r][j], pk = s.P[j][r], ak = s.A[r][j] + s.A[j][r];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        dqr[i][m] = fmaf(pq, kj[m], dqr[i][m]);
        dkr[i][m] = fmaf(pk, qj[m], fmaf(ak, kj[m], dkr[i][m]));
      }
    }
  }
  // through the normalisation, and out
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + i;
    float pq = 0.0f, pk = 0.0f;
    if (a.l2) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        pq = fmaf(dqr[i][m], s.Q[r][lane + 32 * m], pq);
        pk = fmaf(dkr[i][m], s.K[r][lane + 32 * m], pk);
      }
      pq = wsum(pq);
      pk = wsum(pk);
    }
    if (r < p.n) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int k = lane + 32 * m;
        if (k < a.DK) {
          const float q = s.nq[r] * (dqr[i][m] - s.Q[r][k] * pq), kx = s.nk[r] * (dkr[i][m] - s.K[r][k] * pk);
          if (a.share == 1) {
            static_cast<float*>(a.dq)[(p.tok0 + r) * a.dqs + (int64_t)p.h * a.DK + k] = q;
            static_cast<float*>(a.dk)[(p.tok0 + r) * a.dks + (int64_t)p.h * a.DK + k] = kx;
          } else {
            const size_t at = ((size_t)(p.tok0 + r) * a.Hv + p.h) * a.DK + k;
            a.pdq[at] = q;
            a.pdk[at] = kx;
          }
        }
      }
    }
  }
  inner = wsum(inner);
  if (lane == 0) s.red[warp] = fmaf(s.g.eg[C - 1], inner, wtot);
  __syncthreads();
  if (warp == 0) {
    float d = s.dgam[lane];
    if (lane == C - 1)
      for (int w = 0; w < 8; ++w) d += s.red[w];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float dn = __shfl_down_sync(~0u, d, o);
      if (lane + o < 32) d += dn;
    }
    if (lane < p.n) {
      const int64_t at = (p.tok0 + lane) * a.Hv + p.h;
      static_cast<float*>(a.dg)[at] = d;
      static_cast<float*>(a.dbeta)[at] = s.dbeta[lane];
    }
  }
}

// dq and dk of a key head: the shares of its value heads added in order.
__global__ void __launch_bounds__(256) m3_delta_share_kernel(const __grid_constant__ DeltaArgs a) {
  grid_dep_wait();
  const int per = a.Hk * a.DK / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.B * a.T * per) return;
  const int64_t tok = i / per;
  const int c = (int)(i % per) * 4, hk = c / a.DK, k = c % a.DK;
  const float* src = blockIdx.y ? a.pdk : a.pdq;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int m = 0; m < a.share; ++m) {
    const float4 x = *reinterpret_cast<const float4*>(src + ((size_t)tok * a.Hv + hk * a.share + m) * a.DK + k);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  float* o = static_cast<float*>(blockIdx.y ? a.dk : a.dq) + tok * (blockIdx.y ? a.dks : a.dqs) + c;
  *reinterpret_cast<float4*>(o) = s;
}

cudaError_t launch_delta_bwd(const DeltaArgs& a, cudaStream_t st) {
  const struct { void (*kern)(DeltaArgs); size_t smem; unsigned x, y; } steps[] = {
      {m3_delta_bwd_prep_kernel, sizeof(PrepSmem), (unsigned)(a.B * a.Hv * a.nc), 1},
      {m3_delta_bwd_rev_kernel, sizeof(RevSmem), (unsigned)(a.B * a.Hv), DMAX / RV},
      {m3_delta_bwd_grad_kernel, sizeof(GradSmem), (unsigned)(a.B * a.Hv * a.nc), 1}};
  for (const auto& s : steps) {
    // (the attribute belongs to the current context, and setting it costs under a microsecond)
    cudaError_t e = cudaFuncSetAttribute(s.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s.smem);
    if (e == cudaSuccess) e = launch_k(s.kern, dim3(s.x, s.y), 256, s.smem, st, false, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
cudaError_t launch_delta_share(const DeltaArgs& a, cudaStream_t st) {
  const int64_t n = (int64_t)a.B * a.T * (a.Hk * a.DK / 4);
  return launch_k(m3_delta_share_kernel, dim3((unsigned)((n + 255) / 256), 2), 256, 0, st, true, a);
}

}  // namespace m3
