// m3_delta_rec.cu -- the gated delta rule token by token: decoding, and
// sequences of f32 activations.
#include "m3_delta.cuh"

namespace m3 {

// One block of 256 threads holds TV columns of one head's state in registers:
// a thread has the four columns 4 vi .. 4 vi + 3 of the rows kr, kr + RPP, ...
// so a warp reads and writes whole 128-byte lines of the state.  The two sums
// over rows (S'^T k and S^T q) are butterflies inside a warp and one
// shared-memory pass over the eight warps.  All arithmetic is f32.
//
// NT tokens at a time are brought into shared memory (the next ones are in
// flight meanwhile) and their rows of q and k normalised there, so that a
// token costs two barriers and no trip to memory.  NT = 1 is decoding: a
// single step is bound by the state's way in and out of HBM (2 x 64 KB per
// head of 128 x 128); TV = 128 moves the most per block, TV = 32 gives four
// times the blocks when there are few heads.
template <typename T, int TV, int NT>
__global__ void __launch_bounds__(256, 2) m3_delta_rec_kernel(const __grid_constant__ DeltaArgs a) {
  constexpr int LPR = TV / 4;        // lanes per row
  constexpr int RPP = 256 / LPR;     // rows per pass
  constexpr int NI = DMAX / RPP;     // passes (rows per thread)
  constexpr int KQL = 2 * NT * DMAX / 256, VL = (NT * TV + 255) / 256;  // values a thread brings in
  __shared__ __align__(16) float kq[2][NT][DMAX];  // k, q
  __shared__ __align__(16) float vs[NT][TV];
  __shared__ __align__(16) float ps[8][TV], os[8][TV];
  __shared__ float dec[NT], bt[NT], nrm[2][NT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (a.DV + TV - 1) / TV;
  const int bh = blockIdx.x / tiles, v0 = (blockIdx.x % tiles) * TV;
  const int b = bh / a.Hv, h = bh % a.Hv, hk = h / a.share;
  const int vi = tid % LPR, kr = tid / LPR;
  const int vcol = v0 + vi * 4;
  const bool vok = vcol < a.DV;
  const size_t sbase = (size_t)bh * a.DK * a.DV + vcol;

  float4 S[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = kr + i * RPP;
    S[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.s_in && vok && k < a.DK) S[i] = *reinterpret_cast<const float4*>(a.s_in + sbase + (size_t)k * a.DV);
  }

  const int64_t tok0 = (int64_t)b * a.T;
  const int c = tid & (DMAX - 1), which = tid >> 7;  // this thread brings column c of k (0) or q (1)
  const T* xp = static_cast<const T*>(which ? a.q : a.k) + tok0 * (which ? a.qs : a.ks) + (int64_t)hk * a.DK + c;
  const int64_t xs = which ? a.qs : a.ks;
  const T* vp = static_cast<const T*>(a.v) + tok0 * a.vs + (int64_t)h * a.DV + v0;
  const T* gp = static_cast<const T*>(a.g) + tok0 * a.Hv + h;
  const T* bp = static_cast<const T*>(a.beta) + tok0 * a.Hv + h;
  T* op = static_cast<T*>(a.o) + (tok0 * a.Hv + h) * a.DV + v0 + tid;

  float x[KQL], v[VL], g = 0.0f;
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < KQL; ++i) x[i] = t0 + i < a.T && c < a.DK ? Act<T>::ld(xp + (t0 + i) * xs) : 0.0f;
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int j = tid + i * 256, t = t0 + j / TV, d = j % TV;
      v[i] = j < NT * TV && t < a.T && v0 + d < a.DV ? Act<T>::ld(vp + (int64_t)t * a.vs + d) : 0.0f;
    }
    const int t = t0 + (tid >> 1);
    if (tid < 2 * NT && t < a.T) g = Act<T>::ld((tid & 1 ? bp : gp) + (int64_t)t * a.Hv);
  };
  fetch(0);
  for (int t0 = 0; t0 < a.T; t0 += NT) {
    if (t0 > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < KQL; ++i) kq[which][i][c] = x[i];
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int j = tid + i * 256;
      if (j < NT * TV) vs[j / TV][j % TV] = v[i];
    }
    if (tid < 2 * NT) (tid & 1 ? bt : dec)[tid >> 1] = tid & 1 ? g : expf(clamp_g(g));
    __syncthreads();
    if (t0 + NT < a.T) fetch(t0 + NT);
    if (a.l2) {
#pragma unroll
      for (int r = warp; r < 2 * NT; r += 8) {
        const float4 e = *reinterpret_cast<const float4*>(&kq[r & 1][r >> 1][lane * 4]);
        float ss = fmaf(e.x, e.x, fmaf(e.y, e.y, fmaf(e.z, e.z, e.w * e.w)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        if (lane == 0) nrm[r & 1][r >> 1] = rsqrtf(ss + DELTA_L2_EPS);
      }
      __syncthreads();
    }
    const int n = min(NT, a.T - t0);
    for (int j = 0; j < n; ++j) {
      const int t = t0 + j;
      if (a.ckpt && t % a.chunk == 0) {
        float* ck = a.ckpt + ((size_t)bh * a.nc + t / a.chunk) * a.DK * a.DV + vcol;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int k = kr + i * RPP;
          if (vok && k < a.DK) *reinterpret_cast<float4*>(ck + (size_t)k * a.DV) = S[i];
        }
      }
      const float nk = a.l2 ? nrm[0][j] : 1.0f, nq = a.l2 ? a.scale * nrm[1][j] : a.scale;
      const float de = dec[j], be = bt[j];
      float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float kk[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        kk[i] = kq[0][j][kr + i * RPP] * nk;
        S[i].x *= de; S[i].y *= de; S[i].z *= de; S[i].w *= de;
        p.x = fmaf(S[i].x, kk[i], p.x); p.y = fmaf(S[i].y, kk[i], p.y);
        p.z = fmaf(S[i].z, kk[i], p.z); p.w = fmaf(S[i].w, kk[i], p.w);
      }
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        p.x += __shfl_xor_sync(~0u, p.x, o); p.y += __shfl_xor_sync(~0u, p.y, o);
        p.z += __shfl_xor_sync(~0u, p.z, o); p.w += __shfl_xor_sync(~0u, p.w, o);
      }
      if (lane < LPR) *reinterpret_cast<float4*>(&ps[warp][vi * 4]) = p;
      __syncthreads();
      p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float4 r = *reinterpret_cast<const float4*>(&ps[w][vi * 4]);
        p.x += r.x; p.y += r.y; p.z += r.z; p.w += r.w;
      }
      const float4 vc = *reinterpret_cast<const float4*>(&vs[j][vi * 4]);
      const float4 u = make_float4(be * (vc.x - p.x), be * (vc.y - p.y), be * (vc.z - p.z), be * (vc.w - p.w));
      float4 o4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const float qv = kq[1][j][kr + i * RPP];
        S[i].x = fmaf(kk[i], u.x, S[i].x); S[i].y = fmaf(kk[i], u.y, S[i].y);
        S[i].z = fmaf(kk[i], u.z, S[i].z); S[i].w = fmaf(kk[i], u.w, S[i].w);
        o4.x = fmaf(S[i].x, qv, o4.x); o4.y = fmaf(S[i].y, qv, o4.y);
        o4.z = fmaf(S[i].z, qv, o4.z); o4.w = fmaf(S[i].w, qv, o4.w);
      }
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        o4.x += __shfl_xor_sync(~0u, o4.x, o); o4.y += __shfl_xor_sync(~0u, o4.y, o);
        o4.z += __shfl_xor_sync(~0u, o4.z, o); o4.w += __shfl_xor_sync(~0u, o4.w, o);
      }
      if (lane < LPR) *reinterpret_cast<float4*>(&os[warp][vi * 4]) = o4;
      __syncthreads();
      if (tid < TV && v0 + tid < a.DV) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += os[w][tid];
        Act<T>::st(op, s * nq);
      }
      op += (size_t)a.Hv * a.DV;
    }
  }
  if (a.s_out) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = kr + i * RPP;
      if (vok && k < a.DK) *reinterpret_cast<float4*>(a.s_out + sbase + (size_t)k * a.DV) = S[i];
    }
  }
}

// One token: wide blocks once there are two per SM.  Sequences: narrow blocks
// (a token's arithmetic and its butterflies are shared by four times as many
// SMs) unless there are eight heads per SM to choose from.
template <typename T>
cudaError_t launch_delta_rec(const DeltaArgs& a, cudaStream_t st, int sms) {
  const int64_t heads = (int64_t)a.B * a.Hv;
  const bool wide = heads >= (a.T == 1 ? 2 : 8) * (int64_t)sms;
  const int tv = wide ? 128 : 32;
  const dim3 grid((unsigned)(heads * ((a.DV + tv - 1) / tv)));
  if (a.T == 1) {
    if (wide) m3_delta_rec_kernel<T, 128, 1><<<grid, 256, 0, st>>>(a);
    else m3_delta_rec_kernel<T, 32, 1><<<grid, 256, 0, st>>>(a);
  } else {
    if (wide) m3_delta_rec_kernel<T, 128, 16><<<grid, 256, 0, st>>>(a);
    else m3_delta_rec_kernel<T, 32, 16><<<grid, 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}
template cudaError_t launch_delta_rec<float>(const DeltaArgs&, cudaStream_t, int);
template cudaError_t launch_delta_rec<__nv_bfloat16>(const DeltaArgs&, cudaStream_t, int);

}  // namespace m3
