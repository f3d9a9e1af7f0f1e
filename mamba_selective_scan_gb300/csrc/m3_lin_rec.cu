// m3_lin_rec.cu -- linear attention with a decay for each head, token by
// token: decoding, and sequences of f32 activations.
#include <type_traits>

#include "m3_lin.cuh"

namespace m3 {

// One token.  A block of 256 threads holds TV columns of one head's state in
// registers: a thread has four columns of the rows kr, kr + RPP, ..., so a
// warp reads and writes whole 128-byte lines.  The sum over rows (S^T q) is a
// butterfly inside a warp and one shared-memory pass over the eight warps.
// All arithmetic is f32.  Bound by the state's way in and out of HBM (2 x 64
// KB per head of 128 x 128): 64 x 40 heads take 49.5 us, the 338 MB at the rate
// of a plain copy.  Whole heads per block where they fill the SMs; with fewer,
// blocks of 32 columns, four times as many (one row of 16 heads: 4 us, in the
// call's shadow either way).
template <typename T, int TV>
__global__ void __launch_bounds__(256, 2) m3_lin_step_kernel(const __grid_constant__ LinArgs a) {
  constexpr int LPR = TV / 4;           // lanes per row
  constexpr int RPP = 256 / LPR;        // rows per pass
  constexpr int NI = LIN_DMAX / RPP;    // rows per thread
  __shared__ __align__(16) float kq[2][LIN_DMAX];
  __shared__ __align__(16) float os[8][TV];
  const LinPass& p = a.p[0];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (p.DV + TV - 1) / TV;
  const int bh = blockIdx.x / tiles, v0 = (blockIdx.x % tiles) * TV;
  const int b = bh / a.Hv, h = bh % a.Hv;
  const int vi = tid % LPR, kr = tid / LPR, vcol = v0 + vi * 4;
  const bool vok = vcol < p.DV;
  const size_t sbase = (size_t)bh * p.DK * p.DV + vcol;

  float4 S[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = kr + i * RPP;
    S[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (p.s_in && vok && k < p.DK) S[i] = *reinterpret_cast<const float4*>(p.s_in + sbase + (size_t)k * p.DV);
  }
  const int c = tid & (LIN_DMAX - 1);
  const T* xp = tid < LIN_DMAX ? static_cast<const T*>(p.k) + b * p.ks + (int64_t)(h / p.kh) * p.DK + c
                               : static_cast<const T*>(p.q) + b * p.qs + (int64_t)(h / p.qh) * p.DK + c;
  kq[tid >> 7][c] = c < p.DK ? Act<T>::ld(xp) : 0.0f;
  const T* vp = static_cast<const T*>(p.v) + b * p.vs + (int64_t)(h / p.vh) * p.DV + vcol;
  float v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = vok ? Act<T>::ld(vp + j) : 0.0f;
  const LinDecay lam = lin_decay(a.ld[h], 1);
  __syncthreads();
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = kr + i * RPP;
    const float kk = kq[0][k], q = kq[1][k];
    S[i].x = fmaf(lam.near, S[i].x, fmaf(lam.off, S[i].x, kk * v[0]));
    S[i].y = fmaf(lam.near, S[i].y, fmaf(lam.off, S[i].y, kk * v[1]));
    S[i].z = fmaf(lam.near, S[i].z, fmaf(lam.off, S[i].z, kk * v[2]));
    S[i].w = fmaf(lam.near, S[i].w, fmaf(lam.off, S[i].w, kk * v[3]));
    o.x = fmaf(S[i].x, q, o.x); o.y = fmaf(S[i].y, q, o.y);
    o.z = fmaf(S[i].z, q, o.z); o.w = fmaf(S[i].w, q, o.w);
    if (p.s_out && vok && k < p.DK) *reinterpret_cast<float4*>(p.s_out + sbase + (size_t)k * p.DV) = S[i];
  }
#pragma unroll
  for (int m = LPR; m < 32; m <<= 1) {
    o.x += __shfl_xor_sync(~0u, o.x, m); o.y += __shfl_xor_sync(~0u, o.y, m);
    o.z += __shfl_xor_sync(~0u, o.z, m); o.w += __shfl_xor_sync(~0u, o.w, m);
  }
  if (lane < LPR) *reinterpret_cast<float4*>(&os[warp][vi * 4]) = o;
  __syncthreads();
  if (tid < TV && v0 + tid < p.DV) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += os[w][tid];
    Act<T>::st(static_cast<T*>(p.out) + (size_t)b * p.os + (size_t)h * p.DV + v0 + tid, s * a.scale);
  }
}

// Four values into shared memory as f32: zeros where there are none
__device__ __forceinline__ void copy4(float* dst, const float* src, bool live) {
  cp_async16(dst, src, live);
}
__device__ __forceinline__ void copy4(float* dst, const __nv_bfloat16* src, bool live) {
  const uint2 x = live ? *reinterpret_cast<const uint2*>(src) : make_uint2(0, 0);
  *reinterpret_cast<float4*>(dst) = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u),
                                                __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xFFFF0000u));
}

// A sequence: 32 columns of one head's state per block of four warps, eight
// lanes to two neighbouring columns (a lane has rows 4 s .. 4 s + 3 of every
// 32).  16 tokens at a time are brought into shared memory, the next 16 in
// flight meanwhile.  Within those 16 the state that they start from stays as it
// is and what they add grows beside it from zero,
//
//   o_i = scale (lam^{i+1} S0^T q_i + L_i^T q_i),  L_i = lam L_{i-1} + k_i v_i^T
//
// which costs what updating the state itself would, and rounds the state once
// in 16 tokens: with a state that hardly fades, roundings that all fall the
// same way added up to 3e-5 over 16384 tokens.  The outputs of eight tokens
// are summed over the lanes at once (seven shuffles instead of 24).
//
// With every SM at work shared memory is the bound: a lane reads its 16 rows'
// k and q of every token, 128 bytes, 32 wavefronts a warp whatever the lanes
// share.  A second column per lane halves that, a fourth needs more registers
// than latency can spare (training passes, f32, heads of 128 x 128: 8 x 128 x 4
// heads 78 us, 8 x 512 x 16 heads 849; before the last step 82 and 881, with one
// column 99 and 1143, with four 125 and 1037, in blocks of eight warps 101 and
// 891).
//
// blockIdx.z: time segments, from the chaining's start states.  AGG: only the
// states, each segment's end from a zero start.
constexpr int SEQ_THREADS = 128, SEQ_COLS = 2;
template <typename T, bool AGG>
__global__ void __launch_bounds__(SEQ_THREADS, 3) m3_lin_seq_kernel(const __grid_constant__ LinArgs a) {
  constexpr int NT = 16, COLS = SEQ_COLS, THREADS = SEQ_THREADS, TV = THREADS / 8 * COLS, KQ = AGG ? 1 : 2;
  __shared__ __align__(16) float kq[2][KQ][NT][LIN_DMAX];  // k, q; of two tiles
  __shared__ __align__(16) float vs[2][NT][TV];
  __shared__ float os[NT][TV + 1];
  __shared__ float pw[NT];  // the start state's weight in each token's output
  const LinPass& p = a.p[blockIdx.y];
  constexpr int MAX_TILES = LIN_DMAX / TV;
  const int tid = threadIdx.x, lane = tid & 31;
  const int bh = blockIdx.x / MAX_TILES, v0 = (blockIdx.x % MAX_TILES) * TV;
  if (v0 >= p.DV) return;
  const int b = bh / a.Hv, h = bh % a.Hv;
  const int s = lane & 7, col = (tid >> 3) * COLS;
  // this segment's tokens, in the pass's order
  const int seg = blockIdx.z, seg_tok = a.seg_chunks * LIN_C, odd = p.rev ? a.nc * LIN_C - a.T : 0;
  const int first = seg ? seg * seg_tok - odd : 0, last = seg + 1 < a.segs ? (seg + 1) * seg_tok - odd : a.T;
  const size_t slot = ((size_t)(bh * a.np + blockIdx.y) * a.segs + seg) * LIN_DMAX * LIN_DMAX + v0 + col;  // row k: + k LIN_DMAX
  const size_t sbase = (size_t)bh * p.DK * p.DV;
  auto where = [&](int k, int c) { return p.st ? sbase + (size_t)(v0 + col + c) * p.DK + k : sbase + (size_t)k * p.DV + v0 + col + c; };
  auto row = [&](int i) { return (i >> 2) * 32 + s * 4 + (i & 3); };

  const float ld = lin_ld(a.ld[h]);
  const float fv = p.rev ? a.scale : 1.0f, fo = p.rev ? 1.0f : a.scale;
  if (tid < NT) pw[tid] = expf(ld * (float)(p.rev ? tid : tid + 1));
  const float2 lam = f2b(expf(ld));
  const int64_t tok0 = (int64_t)b * a.T;
  const T* kp = static_cast<const T*>(p.k) + tok0 * p.ks + (int64_t)(h / p.kh) * p.DK;
  const T* qp = static_cast<const T*>(p.q) + tok0 * p.qs + (int64_t)(h / p.qh) * p.DK;
  const T* vp = static_cast<const T*>(p.v) + tok0 * p.vs + (int64_t)(h / p.vh) * p.DV + v0;
  const size_t ob = (size_t)tok0 * p.os + (size_t)h * p.DV + v0;
  auto time = [&](int i) { return (int64_t)(p.rev ? a.T - 1 - i : i); };  // of the pass's i-th token

  // four values a thread on their way into a tile, zeros past the ends
  auto fetch = [&](int buf, int t0) {
#pragma unroll
    for (int j = 0; j < KQ * NT * 32 / THREADS; ++j) {
      const int e = tid + j * THREADS, which = e / (NT * 32), i = e / 32 % NT, c = e % 32 * 4;
      const bool live = t0 + i < last && c < p.DK;
      copy4(&kq[buf][which][i][c], live ? (which ? qp + time(t0 + i) * p.qs : kp + time(t0 + i) * p.ks) + c : kp, live);
    }
#pragma unroll
    for (int j = 0; j < (NT * TV / 4 + THREADS - 1) / THREADS; ++j) {
      const int e = tid + j * THREADS, i = e / (TV / 4), c = e % (TV / 4) * 4;
      const bool live = t0 + i < last && v0 + c < p.DV;
      if (i < NT) copy4(&vs[buf][i][c], live ? vp + time(t0 + i) * p.vs + c : vp, live);
    }
    cp_async_commit();
  };
  fetch(0, first);
  float2 S[COLS][8], L[COLS][8];  // rows row(2 i), row(2 i + 1)
  grid_dep_wait();
#pragma unroll
  for (int c = 0; c < COLS; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = row(i);
      float x = 0.0f;
      if (!AGG && v0 + col + c < p.DV && k < p.DK) {
        if (a.segs > 1) x = a.seg_start[slot + (size_t)k * LIN_DMAX + c];
        else if (p.s_in) x = p.s_in[where(k, c)];
      }
      (i & 1 ? S[c][i >> 1].y : S[c][i >> 1].x) = x;
    }
  int buf = 0;
  for (int t0 = first; t0 < last; t0 += NT, buf ^= 1) {
    cp_async_wait<0>();
    __syncthreads();
    if (t0 + NT < last) fetch(buf ^ 1, t0 + NT);
    const int n = min(NT, last - t0);
#pragma unroll
    for (int c = 0; c < COLS; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) L[c][i] = f2b(0.0f);
    auto tile = [&](auto whole) {  // (whole tiles without a condition for each token: 4 % faster)
#pragma unroll
      for (int g = 0; g < NT; g += 8) {
        float o[COLS][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float2 old[COLS], sum[COLS];
#pragma unroll
          for (int c = 0; c < COLS; ++c) old[c] = sum[c] = f2b(0.0f);
          if (whole.value || g + j < n) {
            float2 vv[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) vv[c] = f2b(vs[buf][g + j][col + c] * fv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 kk = *reinterpret_cast<const float4*>(&kq[buf][0][g + j][i * 32 + s * 4]);
              float4 q;
              if (!AGG) q = *reinterpret_cast<const float4*>(&kq[buf][KQ - 1][g + j][i * 32 + s * 4]);
              const float2 q0 = make_float2(q.x, q.y), q1 = make_float2(q.z, q.w);
#pragma unroll
              for (int c = 0; c < COLS; ++c) {
                L[c][2 * i] = __ffma2_rn(lam, L[c][2 * i], __fmul2_rn(make_float2(kk.x, kk.y), vv[c]));
                L[c][2 * i + 1] = __ffma2_rn(lam, L[c][2 * i + 1], __fmul2_rn(make_float2(kk.z, kk.w), vv[c]));
                if (AGG) continue;
                sum[c] = __ffma2_rn(L[c][2 * i], q0, sum[c]);
                old[c] = __ffma2_rn(S[c][2 * i], q0, old[c]);
                sum[c] = __ffma2_rn(L[c][2 * i + 1], q1, sum[c]);
                old[c] = __ffma2_rn(S[c][2 * i + 1], q1, old[c]);
              }
            }
#pragma unroll
            for (int c = 0; c < COLS; ++c) sum[c] = __ffma2_rn(f2b(pw[g + j]), old[c], sum[c]);
          }
#pragma unroll
          for (int c = 0; c < COLS; ++c) o[c][j] = sum[c].x + sum[c].y;
        }
        // lane s ends with the sum of token g + s
#pragma unroll
        for (int c = 0; c < (AGG ? 0 : COLS); ++c) {
#pragma unroll
          for (int m = 4; m > 0; m >>= 1) {
            const bool up = s & m;
#pragma unroll
            for (int j = 0; j < m; ++j) {
              const float give = up ? o[c][j] : o[c][j + m], keep = up ? o[c][j + m] : o[c][j];
              o[c][j] = keep + __shfl_xor_sync(~0u, give, m);
            }
          }
          os[g + s][col + c] = o[c][0] * fo;
        }
      }
    };
    if (n == NT) tile(std::true_type{});
    else tile(std::false_type{});
    const LinDecay d = lin_decay(ld, n);
    const float2 fl = p.rev ? lam : f2b(1.0f);
#pragma unroll
    for (int c = 0; c < COLS; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        S[c][i] = __ffma2_rn(f2b(d.near), S[c][i], __ffma2_rn(f2b(d.off), S[c][i], __fmul2_rn(fl, L[c][i])));
    if (AGG) continue;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT * TV / THREADS; ++j) {
      const int e = tid + j * THREADS, i = e / TV, c = e % TV;
      if (i < n && v0 + c < p.DV) {
        const size_t at = ob + (size_t)time(t0 + i) * p.os + c;
        if (p.out_f32) static_cast<float*>(p.out)[at] = os[i][c];
        else Act<T>::st(static_cast<T*>(p.out) + at, os[i][c]);
      }
    }
  }
  if (AGG) {
#pragma unroll
    for (int c = 0; c < COLS; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) a.seg_end[slot + (size_t)row(i) * LIN_DMAX + c] = i & 1 ? S[c][i >> 1].y : S[c][i >> 1].x;
  } else if (p.s_out && last == a.T) {
#pragma unroll
    for (int c = 0; c < COLS; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (v0 + col + c < p.DV && row(i) < p.DK) p.s_out[where(row(i), c)] = i & 1 ? S[c][i >> 1].y : S[c][i >> 1].x;
  }
}

template <typename T>
cudaError_t launch_lin_seq(const LinArgs& a, cudaStream_t st) {
  const unsigned x = (unsigned)((int64_t)a.B * a.Hv * (LIN_DMAX / (SEQ_THREADS / 8 * SEQ_COLS)));
  cudaError_t e = cudaSuccess;
  if constexpr (sizeof(T) == 4) {  // (bf16 has segments on the tensor cores alone)
    if (a.segs > 1) {  // (the last segment's end is nobody's start)
      e = launch_k(m3_lin_seq_kernel<T, true>, dim3(x, a.np, a.segs - 1), SEQ_THREADS, 0, st, false, a);
      if (e == cudaSuccess) e = launch_lin_seg(a, st);
    }
  }
  return e == cudaSuccess ? launch_k(m3_lin_seq_kernel<T, false>, dim3(x, a.np, a.segs), SEQ_THREADS, 0, st, a.segs > 1, a) : e;
}

// One token of one pass (decoding): wide blocks once there are two per SM
template <typename T>
cudaError_t launch_lin_rec(LinArgs a, cudaStream_t st, int sms) {
  const int64_t heads = (int64_t)a.B * a.Hv;
  if (a.T == 1 && a.np == 1 && !a.p[0].rev) {
    const int tv = heads >= 2 * (int64_t)sms ? 128 : 32;
    const dim3 grid((unsigned)(heads * ((a.p[0].DV + tv - 1) / tv)));
    if (tv == 128) m3_lin_step_kernel<T, 128><<<grid, 256, 0, st>>>(a);
    else m3_lin_step_kernel<T, 32><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
  }
  if (a.segs < 1) {  // no plan of segments: one
    a.segs = 1;
    a.nc = a.seg_chunks = (a.T + LIN_C - 1) / LIN_C;
  }
  return launch_lin_seq<T>(a, st);
}
template cudaError_t launch_lin_rec<float>(LinArgs, cudaStream_t, int);
template cudaError_t launch_lin_rec<__nv_bfloat16>(LinArgs, cudaStream_t, int);

// dq and dk of shared key heads: the value heads' shares added in their order
// (f32, the same bits on every call), rounded once.  Four columns per thread.
template <typename T>
__global__ void __launch_bounds__(256) m3_lin_share_kernel(const __grid_constant__ LinShare a) {
  grid_dep_wait();
  const int per = a.Hk * a.D / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens * per) return;
  const int64_t tok = a.tokens * per < ((int64_t)1 << 32) ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per;
  const int c = (int)(i % per) * 4, hk = c / a.D, k = c % a.D;
  const int which = blockIdx.y;
  const float* src = a.part[which] + ((size_t)tok * a.Hk * a.share + (size_t)hk * a.share) * a.D + k;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int m = 0; m < a.share; ++m) {
    const float4 x = *reinterpret_cast<const float4*>(src + (size_t)m * a.D);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  T* o = static_cast<T*>(a.out[which]) + tok * a.os[which] + c;  // (16-byte tokens and heads of 8)
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(o) = s;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}
template <typename T> cudaError_t launch_lin_share(const LinShare& a, cudaStream_t st) {
  const int64_t n = a.tokens * (a.Hk * a.D / 4);
  return launch_k(m3_lin_share_kernel<T>, dim3((unsigned)((n + 255) / 256), 2), 256, 0, st, true, a);
}
template cudaError_t launch_lin_share<float>(const LinShare&, cudaStream_t);
template cudaError_t launch_lin_share<__nv_bfloat16>(const LinShare&, cudaStream_t);

}  // namespace m3
