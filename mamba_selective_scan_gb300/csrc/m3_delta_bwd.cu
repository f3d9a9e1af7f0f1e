// m3_delta_bwd.cu -- backward of the gated delta rule in f32 arithmetic, and
// the sum over the value heads that share a key head.
#include "m3_delta.cuh"

namespace m3 {

namespace {
constexpr int C = 32;         // tokens per chunk (the checkpoint interval)
constexpr int LD = DMAX + 4;  // row length of the [C][128] arrays: float4 columns, rows 4 banks apart
constexpr int LS = C + 1;     // row length of the [C][C] arrays

struct DeltaBwdSmem {
  float K[C][LD], Q[C][LD], dO[C][LD];
  float U[C][LD], dR[C][LD];  // side by side: half of S0's rows fit in their place before they are made,
  float E[C][LD], dU[C][LD];  // and in that of these two when they are used up
  float dS[DMAX][LD];
  float A[C][LS], P[C][LS], Ti[C][LS], X[C][LS];
  float gam[C], beta[C], nq[C], nk[C], dgam[C], dbeta[C], eg[C], el[C];
  float red[8];
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
__device__ __forceinline__ void axpy4(float4& o, float s, float4 x) {
  o.x = fmaf(s, x.x, o.x); o.y = fmaf(s, x.y, o.y); o.z = fmaf(s, x.z, o.z); o.w = fmaf(s, x.w, o.w);
}
}  // namespace

// One block of 8 warps per (batch row, value head) walks the chunks last to
// first with the state's adjoint dS in shared memory.  With the chunk's
// start state S0 from the checkpoint (read through the caches), gam, D as in
// m3_delta.cuh, k and q normalised, P = scale D o QK^T:
//
//   forward again   E = V - e^gam (K S0), T = (I + A)^-1, U = T (beta E)
//   dU = P^T dO + (e^{gam_C - gam} K) dS,   dR = T^T dU,   dV = beta dR
//   dA = -(dR U^T) below the diagonal,      dP = dO U^T on and below it
//   dQ = scale e^gam dO S0^T + (scale dP o D) K
//   dK = e^{gam_C - gam} U dS^T - beta e^gam dR S0^T
//        + (scale dP o D)^T Q + (dA beta D) K + (dA beta D)^T K
//   dS0 = e^{gam_C} dS + scale (e^gam Q)^T dO - (beta e^gam K)^T dR
//
// and each exponent gam_i that a term carries takes that term's share; dg is
// their sum from the end of the chunk.  Every warp owns four rows of a chunk
// (and 16 rows of dS); a lane four columns, side by side where the sum runs
// over rows, 32 apart where it runs along a row.
template <typename T>
__global__ void __launch_bounds__(256) m3_delta_bwd_kernel(const __grid_constant__ DeltaArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  DeltaBwdSmem& s = *reinterpret_cast<DeltaBwdSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x, b = bh / a.Hv, h = bh % a.Hv, hk = h / a.share;
  const int r0 = warp * 4, c0 = lane * 4;

  for (int i = tid; i < DMAX * DMAX; i += 256) {
    const int k = i / DMAX, v = i % DMAX;
    s.dS[k][v] = a.ds_out && k < a.DK && v < a.DV ? a.ds_out[((size_t)bh * a.DK + k) * a.DV + v] : 0.0f;
  }

  for (int ch = a.nc - 1; ch >= 0; --ch) {
    const int t0 = ch * C, n = min(C, a.T - t0);
    const int64_t tok0 = (int64_t)b * a.T + t0;
    __syncthreads();
    for (int i = tid; i < C * DMAX; i += 256) {
      const int r = i / DMAX, c = i % DMAX;
      const int64_t tk = tok0 + r;
      const bool okk = r < n && c < a.DK, okv = r < n && c < a.DV;
      s.K[r][c] = okk ? Act<T>::ld(static_cast<const T*>(a.k) + tk * a.ks + (int64_t)hk * a.DK + c) : 0.0f;
      s.Q[r][c] = okk ? Act<T>::ld(static_cast<const T*>(a.q) + tk * a.qs + (int64_t)hk * a.DK + c) : 0.0f;
      s.E[r][c] = okv ? Act<T>::ld(static_cast<const T*>(a.v) + tk * a.vs + (int64_t)h * a.DV + c) : 0.0f;
      s.dO[r][c] = okv ? Act<T>::ld(static_cast<const T*>(a.d_o) + (tk * a.Hv + h) * a.DV + c) : 0.0f;
    }
    if (warp == 0) {
      const bool ok = lane < n;
      float g = ok ? clamp_g(Act<T>::ld(static_cast<const T*>(a.g) + (tok0 + lane) * a.Hv + h)) : 0.0f;
      s.beta[lane] = ok ? Act<T>::ld(static_cast<const T*>(a.beta) + (tok0 + lane) * a.Hv + h) : 0.0f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float up = __shfl_up_sync(~0u, g, o);
        if (lane >= o) g += up;
      }
      s.gam[lane] = g;
      s.eg[lane] = expf(g);
      s.el[lane] = expf(__shfl_sync(~0u, g, 31) - g);
      s.dgam[lane] = 0.0f;
      s.dbeta[lane] = 0.0f;
    }
    __syncthreads();
    const float* S0 = a.ckpt_in + ((size_t)bh * a.nc + ch) * a.DK * a.DV;
    // normalise the rows of K and Q
#pragma unroll
    for (int r = r0; r < r0 + 4; ++r) {
      float4& k4 = *reinterpret_cast<float4*>(&s.K[r][c0]);
      float4& q4 = *reinterpret_cast<float4*>(&s.Q[r][c0]);
      float nk = 1.0f, nq = 1.0f;
      if (a.l2) {
        nk = rsqrtf(wsum(dot4(k4, k4, 0.0f)) + DELTA_L2_EPS);
        nq = rsqrtf(wsum(dot4(q4, q4, 0.0f)) + DELTA_L2_EPS);
        k4.x *= nk; k4.y *= nk; k4.z *= nk; k4.w *= nk;
        q4.x *= nq; q4.y *= nq; q4.z *= nq; q4.w *= nq;
      }
      if (lane == 0) {
        s.nk[r] = nk;
        s.nq[r] = nq;
      }
    }
    __syncthreads();
    auto half_of_S0 = [&](float (*to)[LD], int half) {  // 64 rows
      for (int i = tid; i < 64 * (DMAX / 4); i += 256) {
        const int k = i >> 5, v = (i & 31) * 4, kk = half * 64 + k;
        *reinterpret_cast<float4*>(&to[k][v]) =
            kk < a.DK && v < a.DV ? __ldg(reinterpret_cast<const float4*>(S0 + (size_t)kk * a.DV + v)) : make_float4(0, 0, 0, 0);
      }
    };
    // A, P (row i of a warp, column j = lane), and E -= e^gam (K S0)
    float kk[4] = {0, 0, 0, 0};  // k_i.k_j
    {
      float qk[4] = {0, 0, 0, 0};
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
        const float D = lane <= r ? expf(s.gam[r] - s.gam[lane]) : 0.0f;
        s.P[r][lane] = a.scale * D * qk[i];
        s.A[r][lane] = lane < r ? s.beta[r] * D * kk[i] : 0.0f;
      }
      float4 acc[4] = {};
      float (*S0h)[LD] = s.U;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        half_of_S0(S0h, half);
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < 64; ++k) {
          const float4 sv = f4(&S0h[k][c0]);
#pragma unroll
          for (int i = 0; i < 4; ++i) axpy4(acc[i], s.K[r0 + i][half * 64 + k], sv);
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) axpy4(*reinterpret_cast<float4*>(&s.E[r0 + i][c0]), -s.eg[r0 + i], acc[i]);
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
      }
    }
    __syncthreads();
    // U = T (beta E);  dU = P^T dO + (e^{gam_C - gam} K) dS
    {
      float4 u[4] = {}, d[4] = {};
      for (int j = 0; j < C; ++j) {
        const float4 e = f4(&s.E[j][c0]), o = f4(&s.dO[j][c0]);
        const float bj = s.beta[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          axpy4(u[i], s.Ti[r0 + i][j] * bj, e);
          axpy4(d[i], s.P[j][r0 + i], o);
        }
      }
      float4 w[4] = {};
      for (int k = 0; k < DMAX; ++k) {
        const float4 x = f4(&s.dS[k][c0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) axpy4(w[i], s.K[r0 + i][k], x);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        axpy4(d[i], s.el[r0 + i], w[i]);
        *reinterpret_cast<float4*>(&s.U[r0 + i][c0]) = u[i];
        *reinterpret_cast<float4*>(&s.dU[r0 + i][c0]) = d[i];
      }
    }
    __syncthreads();
    // dR = T^T dU;  dV = beta dR;  dbeta and the exponent of e^gam (K S0)
    {
      float4 d[4] = {};
      for (int j = 0; j < C; ++j) {
        const float4 x = f4(&s.dU[j][c0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) axpy4(d[i], s.Ti[j][r0 + i], x);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + i;
        *reinterpret_cast<float4*>(&s.dR[r][c0]) = d[i];
        const float db = wsum(dot4(d[i], f4(&s.E[r][c0]), 0.0f));
        if (lane == 0) s.dbeta[r] += db;
        if (r < n && c0 < a.DV) {
          T* o = static_cast<T*>(a.dv) + (tok0 + r) * a.dvs + (int64_t)h * a.DV + c0;
          const float bt = s.beta[r];
          Act<T>::st(o, bt * d[i].x); Act<T>::st(o + 1, bt * d[i].y);
          Act<T>::st(o + 2, bt * d[i].z); Act<T>::st(o + 3, bt * d[i].w);
        }
      }
    }
    __syncthreads();
    // dA and dP (row i of a warp, column j = lane); A and P become
    // dA beta D and scale dP D
    {
      float da[4] = {0, 0, 0, 0}, dp[4] = {0, 0, 0, 0};
      for (int c = 0; c < DMAX; c += 4) {
        const float4 uj = f4(&s.U[lane][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          da[i] = dot4(f4(&s.dR[r0 + i][c]), uj, da[i]);
          dp[i] = dot4(f4(&s.dO[r0 + i][c]), uj, dp[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + i;
        const float D = lane <= r ? expf(s.gam[r] - s.gam[lane]) : 0.0f;
        const float xa = lane < r ? -da[i] : 0.0f, xp = lane <= r ? dp[i] : 0.0f;
        const float ma = xa * s.A[r][lane], mp = xp * s.P[r][lane];
        // A carries beta_r: its derivative is taken with A / beta_r = D k_r.k_j
        const float db = wsum(xa * D * kk[i]);
        const float row = wsum(ma + mp);
        if (lane == 0) {
          s.dbeta[r] += db;
          s.dgam[r] += row;
        }
        s.X[r][lane] = ma + mp;
        s.A[r][lane] = xa * s.beta[r] * D;
        s.P[r][lane] = xp * a.scale * D;
      }
    }
    __syncthreads();
    if (warp == 0) {
      float col = 0.0f;
      for (int i = lane; i < C; ++i) col += s.X[i][lane];
      s.dgam[lane] -= col;
    }
    __syncthreads();
    // dQ, dK (rows of a warp; columns lane + 32 m), the rest of dgam
    float dqr[4][4], dkr[4][4];
    float wtot = 0.0f;
    {
      float os[4][4] = {}, us[4][4] = {}, rs[4][4] = {};
      float (*S0h)[LD] = s.E;  // 64 rows of S0 at a time
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        half_of_S0(S0h, half);
        __syncthreads();
        for (int v = 0; v < a.DV; v += 4) {
          float4 sv[2], dv[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            sv[m] = f4(&S0h[lane + 32 * m][v]);
            dv[m] = f4(&s.dS[half * 64 + lane + 32 * m][v]);
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
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + i;
        float dq_ = 0.0f, dk_ = 0.0f, dw_ = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int k = lane + 32 * m;
          dqr[i][m] = a.scale * s.eg[r] * os[i][m];
          const float x = -s.beta[r] * s.eg[r] * rs[i][m], w = s.el[r] * us[i][m];
          dkr[i][m] = x + w;
          dq_ = fmaf(dqr[i][m], s.Q[r][k], dq_);
          dk_ = fmaf(x, s.K[r][k], dk_);
          dw_ = fmaf(w, s.K[r][k], dw_);
        }
        const float own = wsum(dq_ + dk_), w = wsum(dw_);
        wtot += w;
        if (lane == 0) s.dgam[r] += own - w;
      }
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
      if (r < n) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int k = lane + 32 * m;
          if (k < a.DK) {
            const float q = s.nq[r] * (dqr[i][m] - s.Q[r][k] * pq), kx = s.nk[r] * (dkr[i][m] - s.K[r][k] * pk);
            if (a.share == 1) {
              Act<T>::st(static_cast<T*>(a.dq) + (tok0 + r) * a.dqs + (int64_t)h * a.DK + k, q);
              Act<T>::st(static_cast<T*>(a.dk) + (tok0 + r) * a.dks + (int64_t)h * a.DK + k, kx);
            } else {
              const size_t at = ((size_t)(tok0 + r) * a.Hv + h) * a.DK + k;
              a.pdq[at] = q;
              a.pdk[at] = kx;
            }
          }
        }
      }
    }
    // dS0 (the reads of dS above are behind the barrier), and <dS, S0>
    __syncthreads();
    float inner = 0.0f;
    {
      const float ec = s.eg[C - 1];
      const int k0 = warp * 16;
      float4 d[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 x = f4(&s.dS[k0 + i][c0]);
        if (k0 + i < a.DK && c0 < a.DV)
          inner = dot4(x, __ldg(reinterpret_cast<const float4*>(S0 + (size_t)(k0 + i) * a.DV + c0)), inner);
        d[i] = make_float4(ec * x.x, ec * x.y, ec * x.z, ec * x.w);
      }
      inner *= ec;
      for (int j = 0; j < C; ++j) {
        const float4 o = f4(&s.dO[j][c0]), r = f4(&s.dR[j][c0]);
        const float fq = a.scale * s.eg[j], fk = -s.beta[j] * s.eg[j];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          axpy4(d[i], fq * s.Q[j][k0 + i], o);
          axpy4(d[i], fk * s.K[j][k0 + i], r);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) *reinterpret_cast<float4*>(&s.dS[k0 + i][c0]) = d[i];
    }
    inner = wsum(inner);
    if (lane == 0) s.red[warp] = inner + wtot;
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
      if (lane < n) {
        const int64_t at = (tok0 + lane) * a.Hv + h;
        Act<T>::st(static_cast<T*>(a.dg) + at, d);
        Act<T>::st(static_cast<T*>(a.dbeta) + at, s.dbeta[lane]);
      }
    }
  }
  __syncthreads();
  if (a.ds_in)
    for (int i = tid; i < a.DK * a.DV; i += 256)
      a.ds_in[(size_t)bh * a.DK * a.DV + i] = s.dS[i / a.DV][i % a.DV];
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
  // per call: the attribute belongs to the current context, and setting it costs under a microsecond
  cudaError_t e = cudaFuncSetAttribute(m3_delta_bwd_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(DeltaBwdSmem));
  if (e != cudaSuccess) return e;
  return launch_k(m3_delta_bwd_kernel<float>, dim3((unsigned)(a.B * a.Hv)), 256, sizeof(DeltaBwdSmem), st, false, a);
}
cudaError_t launch_delta_share(const DeltaArgs& a, cudaStream_t st) {
  const int64_t n = (int64_t)a.B * a.T * (a.Hk * a.DK / 4);
  return launch_k(m3_delta_share_kernel, dim3((unsigned)((n + 255) / 256), 2), 256, 0, st, true, a);
}

}  // namespace m3
