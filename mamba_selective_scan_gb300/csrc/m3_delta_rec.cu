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
// A single step is bound by the state's way in and out of HBM (2 x 64 KB per
// head of 128 x 128, against 64 KB of multiply-adds); TV = 128 moves the most
// per block, TV = 32 gives four times the blocks when there are few heads.
template <typename T, int TV>
__global__ void __launch_bounds__(256) m3_delta_rec_kernel(const __grid_constant__ DeltaArgs a) {
  constexpr int LPR = TV / 4;        // lanes per row
  constexpr int RPP = 256 / LPR;     // rows per pass
  constexpr int NI = DMAX / RPP;     // passes (rows per thread)
  __shared__ __align__(16) float kq[2][DMAX];
  __shared__ __align__(16) float ps[8][TV], os[8][TV];
  __shared__ float red[8];
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
  const int c = tid & (DMAX - 1);
  const T* xp = tid < DMAX ? static_cast<const T*>(a.k) + tok0 * a.ks + (int64_t)hk * a.DK + c
                           : static_cast<const T*>(a.q) + tok0 * a.qs + (int64_t)hk * a.DK + c;
  const int64_t xs = tid < DMAX ? a.ks : a.qs;
  const T* vp = static_cast<const T*>(a.v) + tok0 * a.vs + (int64_t)h * a.DV + vcol;
  const T* gp = static_cast<const T*>(a.g) + tok0 * a.Hv + h;
  const T* bp = static_cast<const T*>(a.beta) + tok0 * a.Hv + h;
  T* op = static_cast<T*>(a.o) + (tok0 * a.Hv + h) * a.DV + v0 + tid;

  float x = c < a.DK ? Act<T>::ld(xp) : 0.0f;
  float g = Act<T>::ld(gp), beta = Act<T>::ld(bp);
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = vok ? Act<T>::ld(vp + j) : 0.0f;

  for (int t = 0; t < a.T; ++t) {
    if (a.ckpt && t % a.chunk == 0) {
      float* ck = a.ckpt + ((size_t)bh * a.nc + t / a.chunk) * a.DK * a.DV + vcol;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int k = kr + i * RPP;
        if (vok && k < a.DK) *reinterpret_cast<float4*>(ck + (size_t)k * a.DV) = S[i];
      }
    }
    kq[tid >> 7][c] = x;
    if (a.l2) {
      float ss = x * x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
      if (lane == 0) red[warp] = ss;
    }
    __syncthreads();
    float nk = 1.0f, nq = a.scale;
    if (a.l2) {
      nk = rsqrtf((red[0] + red[1]) + (red[2] + red[3]) + DELTA_L2_EPS);
      nq *= rsqrtf((red[4] + red[5]) + (red[6] + red[7]) + DELTA_L2_EPS);
    }
    const float dec = expf(clamp_g(g)), bt = beta;
    float vc[4] = {v[0], v[1], v[2], v[3]};
    if (t + 1 < a.T) {  // the next token's values, while this one is worked on
      xp += xs; vp += a.vs; gp += a.Hv; bp += a.Hv;
      x = c < a.DK ? Act<T>::ld(xp) : 0.0f;
      g = Act<T>::ld(gp);
      beta = Act<T>::ld(bp);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = vok ? Act<T>::ld(vp + j) : 0.0f;
    }
    float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float kk[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      kk[i] = kq[0][kr + i * RPP] * nk;
      S[i].x *= dec; S[i].y *= dec; S[i].z *= dec; S[i].w *= dec;
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
    const float4 u = make_float4(bt * (vc[0] - p.x), bt * (vc[1] - p.y), bt * (vc[2] - p.z), bt * (vc[3] - p.w));
    float4 o4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const float qv = kq[1][kr + i * RPP];
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
  if (a.s_out) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = kr + i * RPP;
      if (vok && k < a.DK) *reinterpret_cast<float4*>(a.s_out + sbase + (size_t)k * a.DV) = S[i];
    }
  }
}

template <typename T>
cudaError_t launch_delta_rec(const DeltaArgs& a, cudaStream_t st, int sms) {
  const int64_t heads = (int64_t)a.B * a.Hv;
  if (heads >= 2 * sms)
    m3_delta_rec_kernel<T, 128><<<dim3((unsigned)(heads * ((a.DV + 127) / 128))), 256, 0, st>>>(a);
  else
    m3_delta_rec_kernel<T, 32><<<dim3((unsigned)(heads * ((a.DV + 31) / 32))), 256, 0, st>>>(a);
  return cudaGetLastError();
}
template cudaError_t launch_delta_rec<float>(const DeltaArgs&, cudaStream_t, int);
template cudaError_t launch_delta_rec<__nv_bfloat16>(const DeltaArgs&, cudaStream_t, int);

}  // namespace m3
