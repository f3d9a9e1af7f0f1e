// m3_delta_rec.cu -- the gated delta rule token by token: decoding, and
// sequences of f32 activations.
#include "m3_delta.cuh"

namespace m3 {

// One token.  A block of 256 threads holds TV columns of one head's state in
// registers: a thread has the four columns 4 vi .. 4 vi + 3 of the rows kr,
// kr + RPP, ... so a warp reads and writes whole 128-byte lines of the state.
// The two sums over rows (S'^T k and S^T q) are butterflies inside a warp and
// one shared-memory pass over the eight warps.  All arithmetic is f32.
//
// Bound by the state's way in and out of HBM (2 x 64 KB per head of 128 x
// 128): 64 sequences x 40 heads take 52 us, 97 % of the measured copy
// bandwidth.  TV = 128 moves the most per block, TV = 32 gives four times the
// blocks when there are few heads (16 heads: 4 us, latency).
template <typename T, int TV>
__global__ void __launch_bounds__(256, 2) m3_delta_step_kernel(const __grid_constant__ DeltaArgs a) {
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
  const int c = tid & (DMAX - 1);
  const T* xp = tid < DMAX ? static_cast<const T*>(a.k) + b * a.ks + (int64_t)hk * a.DK + c
                           : static_cast<const T*>(a.q) + b * a.qs + (int64_t)hk * a.DK + c;
  const T* vp = static_cast<const T*>(a.v) + b * a.vs + (int64_t)h * a.DV + vcol;
  const float x = c < a.DK ? Act<T>::ld(xp) : 0.0f;
  const float dec = expf(clamp_g(Act<T>::ld(static_cast<const T*>(a.g) + bh))), bt = Act<T>::ld(static_cast<const T*>(a.beta) + bh);
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = vok ? Act<T>::ld(vp + j) : 0.0f;
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
  float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const float kk = kq[0][kr + i * RPP] * nk;
    S[i].x *= dec; S[i].y *= dec; S[i].z *= dec; S[i].w *= dec;
    p.x = fmaf(S[i].x, kk, p.x); p.y = fmaf(S[i].y, kk, p.y);
    p.z = fmaf(S[i].z, kk, p.z); p.w = fmaf(S[i].w, kk, p.w);
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
  const float4 u = make_float4(bt * (v[0] - p.x), bt * (v[1] - p.y), bt * (v[2] - p.z), bt * (v[3] - p.w));
  float4 o4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = kr + i * RPP;
    const float kk = kq[0][k] * nk, qv = kq[1][k];
    S[i].x = fmaf(kk, u.x, S[i].x); S[i].y = fmaf(kk, u.y, S[i].y);
    S[i].z = fmaf(kk, u.z, S[i].z); S[i].w = fmaf(kk, u.w, S[i].w);
    o4.x = fmaf(S[i].x, qv, o4.x); o4.y = fmaf(S[i].y, qv, o4.y);
    o4.z = fmaf(S[i].z, qv, o4.z); o4.w = fmaf(S[i].w, qv, o4.w);
    if (a.s_out && vok && k < a.DK) *reinterpret_cast<float4*>(a.s_out + sbase + (size_t)k * a.DV) = S[i];
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
    Act<T>::st(static_cast<T*>(a.o) + (size_t)bh * a.DV + v0 + tid, s * nq);
  }
}

// A sequence: 32 columns of one head's state per block, eight lanes to a
// column (a lane has rows 4 s .. 4 s + 3 of every 32), so that both sums over
// rows are three shuffles inside a warp and no barrier stands between
// tokens: a token is about 300 cycles of latency.  16 tokens at a time are
// brought into shared memory, the next 16 in flight meanwhile; outputs leave
// from there in whole rows.  Bound by that latency: 0.37 us a token (8 x 128 x
// 4 heads f32, 128 blocks, checkpoints written: 47 us).
template <typename T>
__global__ void __launch_bounds__(256) m3_delta_seq_kernel(const __grid_constant__ DeltaArgs a) {
  constexpr int NT = 16, TV = 32;
  __shared__ __align__(16) float kq[2][NT][DMAX];  // k, q
  __shared__ float vs[NT][TV], os[NT][TV];
  __shared__ float dec[NT], bt[NT], nrm[2][NT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (a.DV + TV - 1) / TV;
  const int bh = blockIdx.x / tiles, v0 = (blockIdx.x % tiles) * TV;
  const int b = bh / a.Hv, h = bh % a.Hv, hk = h / a.share;
  const int s = lane & 7, col = warp * 4 + (lane >> 3);
  const bool vok = v0 + col < a.DV;
  const size_t sbase = (size_t)bh * a.DK * a.DV + v0 + col;

  float S[16];  // rows 32 (i / 4) + 4 s + i % 4
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int k = (i >> 2) * 32 + s * 4 + (i & 3);
    S[i] = a.s_in && vok && k < a.DK ? a.s_in[sbase + (size_t)k * a.DV] : 0.0f;
  }
  const int64_t tok0 = (int64_t)b * a.T;
  const int c = tid & (DMAX - 1), which = tid >> 7;  // this thread brings column c of k (0) or q (1)
  const T* xp = static_cast<const T*>(which ? a.q : a.k) + tok0 * (which ? a.qs : a.ks) + (int64_t)hk * a.DK + c;
  const int64_t xs = which ? a.qs : a.ks;
  const T* vp = static_cast<const T*>(a.v) + tok0 * a.vs + (int64_t)h * a.DV + v0;
  const T* gp = static_cast<const T*>(tid & 1 ? a.beta : a.g) + tok0 * a.Hv + h;
  T* op = static_cast<T*>(a.o) + (tok0 * a.Hv + h) * a.DV + v0;

  float x[NT], v[2], g = 0.0f;
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < NT; ++i) x[i] = t0 + i < a.T && c < a.DK ? Act<T>::ld(xp + (t0 + i) * xs) : 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + warp + i * 8;
      v[i] = t < a.T && v0 + lane < a.DV ? Act<T>::ld(vp + (int64_t)t * a.vs + lane) : 0.0f;
    }
    const int t = t0 + (tid >> 1);
    if (tid < 2 * NT && t < a.T) g = Act<T>::ld(gp + (int64_t)t * a.Hv);
  };
  fetch(0);
  for (int t0 = 0; t0 < a.T; t0 += NT) {
#pragma unroll
    for (int i = 0; i < NT; ++i) kq[which][i][c] = x[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) vs[warp + i * 8][lane] = v[i];
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
    if (a.ckpt && t0 % a.chunk == 0) {  // (a chunk is a whole number of NT)
      float* ck = a.ckpt + ((size_t)bh * a.nc + t0 / a.chunk) * a.DK * a.DV + v0 + col;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = (i >> 2) * 32 + s * 4 + (i & 3);
        if (vok && k < a.DK) ck[(size_t)k * a.DV] = S[i];
      }
    }
    const int n = min(NT, a.T - t0);
#pragma unroll 2
    for (int j = 0; j < n; ++j) {
      const float nk = a.l2 ? nrm[0][j] : 1.0f, nq = a.l2 ? a.scale * nrm[1][j] : a.scale;
      const float de = dec[j];
      float4 kk[4], p = make_float4(0.0f, 0.0f, 0.0f, 0.0f), o = p;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kk[i] = *reinterpret_cast<const float4*>(&kq[0][j][i * 32 + s * 4]);
        S[4 * i] *= de; S[4 * i + 1] *= de; S[4 * i + 2] *= de; S[4 * i + 3] *= de;
        p.x = fmaf(S[4 * i], kk[i].x, p.x); p.y = fmaf(S[4 * i + 1], kk[i].y, p.y);
        p.z = fmaf(S[4 * i + 2], kk[i].z, p.z); p.w = fmaf(S[4 * i + 3], kk[i].w, p.w);
      }
      float ps = (p.x + p.y) + (p.z + p.w);
#pragma unroll
      for (int m = 1; m < 8; m <<= 1) ps += __shfl_xor_sync(~0u, ps, m);
      const float u = bt[j] * fmaf(-nk, ps, vs[j][col]) * nk;  // beta (v - S'^T k), times k's factor
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(&kq[1][j][i * 32 + s * 4]);
        S[4 * i] = fmaf(kk[i].x, u, S[4 * i]); S[4 * i + 1] = fmaf(kk[i].y, u, S[4 * i + 1]);
        S[4 * i + 2] = fmaf(kk[i].z, u, S[4 * i + 2]); S[4 * i + 3] = fmaf(kk[i].w, u, S[4 * i + 3]);
        o.x = fmaf(S[4 * i], q.x, o.x); o.y = fmaf(S[4 * i + 1], q.y, o.y);
        o.z = fmaf(S[4 * i + 2], q.z, o.z); o.w = fmaf(S[4 * i + 3], q.w, o.w);
      }
      float so = (o.x + o.y) + (o.z + o.w);
#pragma unroll
      for (int m = 1; m < 8; m <<= 1) so += __shfl_xor_sync(~0u, so, m);
      if (s == 0) os[j][col] = so * nq;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = warp + i * 8;
      if (j < n && v0 + lane < a.DV) Act<T>::st(op + (int64_t)(t0 + j) * a.Hv * a.DV + lane, os[j][lane]);
    }
  }
  if (a.s_out) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = (i >> 2) * 32 + s * 4 + (i & 3);
      if (vok && k < a.DK) a.s_out[sbase + (size_t)k * a.DV] = S[i];
    }
  }
}

// One token (that needs no checkpoint): wide blocks once there are two per
// SM.
template <typename T>
cudaError_t launch_delta_rec(const DeltaArgs& a, cudaStream_t st, int sms) {
  const int64_t heads = (int64_t)a.B * a.Hv;
  const bool step = a.T == 1 && !a.ckpt;
  const int tv = step && heads >= 2 * (int64_t)sms ? 128 : 32;
  const dim3 grid((unsigned)(heads * ((a.DV + tv - 1) / tv)));
  if (!step) m3_delta_seq_kernel<T><<<grid, 256, 0, st>>>(a);
  else if (tv == 128) m3_delta_step_kernel<T, 128><<<grid, 256, 0, st>>>(a);
  else m3_delta_step_kernel<T, 32><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}
template cudaError_t launch_delta_rec<float>(const DeltaArgs&, cudaStream_t, int);
template cudaError_t launch_delta_rec<__nv_bfloat16>(const DeltaArgs&, cudaStream_t, int);

}  // namespace m3
