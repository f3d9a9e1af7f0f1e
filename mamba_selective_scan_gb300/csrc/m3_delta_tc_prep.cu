// m3_delta_tc_prep.cu -- what a chunk of the gated delta rule needs besides
// the state: T, P and the per-token factors, for every chunk at once.
#include "m3_delta_tc.cuh"

namespace m3 {

// nonzero once a kernel here gave up waiting
__device__ unsigned int g_delta_prep_status;

cudaError_t take_delta_prep_status(unsigned* out) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_delta_prep_status, sizeof(v));
  if (e == cudaSuccess && v) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_delta_prep_status, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}

namespace {

constexpr int TP_THREADS = 256;
struct TcWork {  // scratch
  float M[32][36];
  float gam[TC], ss[2][2 * TC], beta[TC], nk[TC], nq[TC];
  float tot;
};


// shared memory: the K/Q tiles; once their product is there, A and P with the
// factors take their place, and T at last A's (four blocks per SM)
constexpr int A_BYTES = TC * (TC + 4) * 4;
static_assert(A_BYTES % 1024 == 0 && A_BYTES >= 2 * TILE, "P's tiles follow A");
constexpr int PV = A_BYTES;
constexpr int PV_BYTES = (int)sizeof(TcPrep) - 2 * TILE;
constexpr int WORK = (PV + PV_BYTES + 1023) / 1024 * 1024;
static_assert(WORK >= 4 * TILE, "the K/Q tiles");
constexpr size_t SMEM_BYTES = WORK + sizeof(TcWork) + 1024;

// D (16 x 8) += A (16 x K) B (K x 8) by one warp, f32 in shared memory, each
// operand as two bf16 terms (three products; these blocks are far too small
// for a tcgen05 product and its way through tensor memory)
__device__ __forceinline__ void warp_mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <int K>
__device__ __forceinline__ void warp_mma_split(float (&d)[4], const float* A, int lda, const float* B, int ldb, int lane) {
  const int g = lane >> 2, t = (lane & 3) * 2;
#pragma unroll
  for (int k = 0; k < K; k += 16) {
    uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 x = *reinterpret_cast<const float2*>(A + (g + (q & 1) * 8) * lda + k + t + (q >> 1) * 8);
      split2(x.x, x.y, ah[q], al[q]);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float* p = B + (k + t + q * 8) * ldb + g;
      split2(p[0], p[ldb], bh[q], bl[q]);
    }
    warp_mma(d, ah, bh);
    warp_mma(d, al, bh);
    warp_mma(d, ah, bl);
  }
}
__device__ __forceinline__ void warp_mma_store(const float (&d)[4], float* o, int ld, int lane, float sign) {
  const int g = lane >> 2, t = (lane & 3) * 2;
  *reinterpret_cast<float2*>(o + g * ld + t) = make_float2(sign * d[0], sign * d[1]);
  *reinterpret_cast<float2*>(o + (g + 8) * ld + t) = make_float2(sign * d[2], sign * d[3]);
}

}  // namespace

// A chunk's T = (I + A)^-1 and P = scale D o (Q K^T), by 256 threads, one
// block per (chunk, head), four blocks per SM.
//
// K over Q times K^T is one 128 x 64 MMA; a thread then has half a row of
// K K^T (rows 0-63) or of Q K^T (64-127).  I + A is inverted by blocks: the
// eight 8 x 8 diagonal blocks by forward substitution (a column per thread),
// then 8 -> 16 -> 32 -> 64 with [[P, 0], [-R C P, R]], the last two steps as
// warp products of two bf16 terms.  T and P are stored as two bf16 terms, 17
// bits of mantissa, so that what they multiply keeps f32-grade sums.
//
// The chain kernels that follow (the forward's and the reverse pass's, each
// twice more over time segments) go through a head's chunks one after the
// other and are bound by that chain; this work has no order, so it is done
// here once, with full SMs, and read back (34 KB per chunk and head).
template <bool L2>
__global__ void __launch_bounds__(TP_THREADS, 4)
m3_delta_tc_prep_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap mk) {
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full, mbk;
  __shared__ uint32_t slot;
  float (&A)[TC][TC + 4] = *reinterpret_cast<float (*)[TC][TC + 4]>(base);
  unsigned char *t_hi = base, *t_lo = base + TILE, *p_hi = base + PV, *p_lo = base + PV + TILE;
  TcVec& vec = *reinterpret_cast<TcVec*>(base + PV + 2 * TILE);
  TcWork& w = *reinterpret_cast<TcWork*>(base + WORK);
  const int pt = threadIdx.x, lane = pt & 31, wp = __shfl_sync(~0u, pt >> 5, 0);
  const int bh = blockIdx.x / a.nc, c = blockIdx.x % a.nc, b = bh / a.Hv, h = bh % a.Hv, hk = h / a.share;
  const uint32_t kq = smem_u32(base);
  const float scale = a.scale;
  TcWait wait;
  if (pt == 0) {
    mbar_init(&full, 1);
    mbar_init(&mbk, 1);
    mbar_init_fence();
  }
  if (wp == 0) tmem_alloc(&slot, 64);
  // this thread's token's gates (threads 0-63; 0 past the sequence)
  float g = 0.0f, beta = 0.0f;
  if (pt < TC && c * TC + pt < a.T) {
    const int64_t at = ((int64_t)b * a.T + c * TC + pt) * a.Hv + h;
    g = __bfloat162float(static_cast<const __nv_bfloat16*>(a.g)[at]);
    beta = __bfloat162float(static_cast<const __nv_bfloat16*>(a.beta)[at]);
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t acc = __shfl_sync(~0u, slot, 0);
  grid_dep_trigger();  // the chain's blocks may come up (they need this block's tensor memory only once it is given back)
  if (wp == 0 && elect_one()) {
    mbar_expect_tx(&full, 4 * TILE);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      tma_tile(kq + blk * 2 * TILE, &mk, blk * 64, hk, c * TC, b, &full);
      tma_tile(kq + blk * 2 * TILE + TILE, &mq, blk * 64, hk, c * TC, b, &full);
    }
    wait(&full, 0);
    if (wait.ok) tc_mma_kq(kq, acc, &mbk);
  }
  __syncwarp();
  wait(&full, 0);
  const int row = (wp & 3) * 32 + lane, ch = wp >> 2;  // row of K over Q, half of its columns
  if (L2) {  // sums of squares, half a row per thread
    float2 s0 = f2b(0.0f), s1 = f2b(0.0f);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint4 x;
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                   : "r"(kq + ch * (2 * TILE) + sw(row, u)));
      const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 e = make_float2(__uint_as_float(q[j] << 16), __uint_as_float(q[j] & 0xFFFF0000u));
        (j & 1 ? s1 : s0) = __ffma2_rn(e, e, j & 1 ? s1 : s0);
      }
    }
    w.ss[ch][row] = (s0.x + s0.y) + (s1.x + s1.y);
  }
  float gam = clamp_g(g) * LOG2E;  // exponents in powers of two
  if (wp < 2) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float up = __shfl_up_sync(~0u, gam, o);
      if (lane >= o) gam += up;
    }
    if (pt == 31) w.tot = gam;
    w.beta[pt] = beta;
  }
  __syncthreads();
  if (wp < 2) {
    if (wp == 1) gam += w.tot;
    w.gam[pt] = gam;
    w.nk[pt] = L2 ? rsqrtf(w.ss[0][pt] + w.ss[1][pt] + DELTA_L2_EPS) : 1.0f;
    w.nq[pt] = L2 ? rsqrtf(w.ss[0][TC + pt] + w.ss[1][TC + pt] + DELTA_L2_EPS) : 1.0f;
  }
  __syncthreads();
  wait(&mbk, 0);  // (and every thread has read its rows of K and Q)
  tmem_fence_after_sync();
  if (wp < 2) {
    const float gc = w.gam[TC - 1], eg = ex2(gam);
    vec.beta[pt] = beta;
    vec.bfx[pt] = beta * eg * w.nk[pt];
    vec.fu[pt] = ex2(gc - gam) * w.nk[pt];
    vec.fq[pt] = scale * eg * w.nq[pt];
    if (pt == 0) vec.ec = ex2(gc);
  }
  {
    const int i = row & (TC - 1);
    const bool isA = (wp & 3) < 2;
    const float gi = w.gam[i];
    const float f = isA ? w.beta[i] * w.nk[i] : scale * w.nq[i];
    const int last = isA ? i - 1 : i;  // last column that counts
    const bool any = ch == 0 || (wp & 1);   // rows 0-31 have nothing in the second half,
    const bool all = ch == 0 && (wp & 1);   // rows 32-63 everything in the first
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c0 = ch * 32 + q * 16;
      float2 v[8];
      if (any) {
        tc_ld16(acc + ((uint32_t)((wp & 3) * 32) << 16) + c0, v);
        const Vec16 gj{&w.gam[c0]}, nj{&w.nk[c0]};
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const float2 d = __ffma2_rn(gj[m], f2b(-1.0f), f2b(gi));
          v[m] = __fmul2_rn(__fmul2_rn(__fmul2_rn(nj[m], f2b(f)), ex2x2(d)), v[m]);
        }
        if (!all) {
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            if (c0 + 2 * m > last) v[m].x = 0.0f;
            if (c0 + 2 * m + 1 > last) v[m].y = 0.0f;
          }
        }
      } else {
#pragma unroll
        for (int m = 0; m < 8; ++m) v[m] = f2b(0.0f);
      }
      if (isA) {
#pragma unroll
        for (int m = 0; m < 8; m += 2)
          *reinterpret_cast<float4*>(&A[i][c0 + 2 * m]) = make_float4(v[m].x, v[m].y, v[m + 1].x, v[m + 1].y);
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint4 h, l;
          split2(v[4 * u], h.x, l.x);
          split2(v[4 * u + 1], h.y, l.y);
          split2(v[4 * u + 2], h.z, l.z);
          split2(v[4 * u + 3], h.w, l.w);
          const uint32_t at = sw(i, (c0 >> 3) + u);
          *reinterpret_cast<uint4*>(p_hi + at) = h;
          *reinterpret_cast<uint4*>(p_lo + at) = l;
        }
      }
    }
  }
  __syncthreads();
  if (wp < 4) {  // a 16 x 16 diagonal block per warp
    const int d = wp * 16;
    if (lane < 16) {  // its two 8 x 8 blocks, a column per thread
      const int e = d + (lane & 8), c = lane & 7;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float s0 = i == c ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
        for (int l = 0; l < i; ++l) (l & 1 ? s1 : s0) = fmaf(-A[e + i][e + l], x[l], l & 1 ? s1 : s0);
        x[i] = s0 + s1;
      }
      __syncwarp(0xFFFF);
#pragma unroll
      for (int i = 0; i < 8; ++i) A[e + i][e + c] = x[i];
    }
    __syncwarp();
    {  // 8 -> 16: two columns of a row per thread
      const int r = lane >> 2, c = (lane & 3) * 2;
      float2 m = f2b(0.0f);
#pragma unroll
      for (int l = 0; l < 8; ++l)
        m = __ffma2_rn(f2b(A[d + 8 + r][d + l]), *reinterpret_cast<const float2*>(&A[d + l][d + c]), m);
      float* M = &w.M[wp * 8][0];
      *reinterpret_cast<float2*>(M + r * 36 + c) = m;
      __syncwarp();
      m = f2b(0.0f);
#pragma unroll
      for (int l = 0; l < 8; ++l)
        m = __ffma2_rn(f2b(-A[d + 8 + r][d + 8 + l]), *reinterpret_cast<const float2*>(M + l * 36 + c), m);
      *reinterpret_cast<float2*>(&A[d + 8 + r][d + c]) = m;
    }
    // 16 -> 32: a pair of warps, a 16 x 8 tile each
    bar_sync(1 + (wp >> 1), 64);
    {
      const int e = (wp >> 1) * 32, c = (wp & 1) * 8;
      float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      warp_mma_split<16>(m, &A[e + 16][e], TC + 4, &A[e][e + c], TC + 4, lane);
      float* M = &w.M[e >> 1][c];  // (a tile's columns are its own warp's)
      warp_mma_store(m, M, 36, lane, 1.0f);
      bar_sync(1 + (wp >> 1), 64);  // both warps have read C
      m[0] = m[1] = m[2] = m[3] = 0.0f;
      warp_mma_split<16>(m, &A[e + 16][e + 16], TC + 4, M, 36, lane);
      warp_mma_store(m, &A[e + 16][e + c], TC + 4, lane, -1.0f);
    }
  }
  __syncthreads();
  {  // 32 -> 64: eight tiles of 16 x 8
    const int r = (wp & 1) * 16, c = (wp >> 1) * 8;
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    warp_mma_split<32>(m, &A[32 + r][0], TC + 4, &A[0][c], TC + 4, lane);
    warp_mma_store(m, &w.M[r][c], 36, lane, 1.0f);
    __syncthreads();
    m[0] = m[1] = m[2] = m[3] = 0.0f;
    warp_mma_split<32>(m, &A[32 + r][32], TC + 4, &w.M[0][c], 36, lane);
    warp_mma_store(m, &A[32 + r][c], TC + 4, lane, -1.0f);
  }
  __syncthreads();
  {  // T as hi and lo in place of A: a quarter row per thread
    const int r = pt >> 2, u0 = (pt & 3) * 2;
    float4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const float4*>(&A[r][u0 * 8 + u * 4]);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint4 h, l;
      split2(x[2 * u].x, x[2 * u].y, h.x, l.x);
      split2(x[2 * u].z, x[2 * u].w, h.y, l.y);
      split2(x[2 * u + 1].x, x[2 * u + 1].y, h.z, l.z);
      split2(x[2 * u + 1].z, x[2 * u + 1].w, h.w, l.w);
      const uint32_t at = sw(r, u0 + u);
      *reinterpret_cast<uint4*>(t_hi + at) = h;
      *reinterpret_cast<uint4*>(t_lo + at) = l;
    }
  }
  fence_proxy_async();
  __syncthreads();
  if (pt == 0) {
    if (wait.ok) {
      unsigned char* dst = a.tp + (size_t)blockIdx.x * a.tp_stride;
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                   ::"l"(dst), "r"(kq), "r"(2 * TILE) : "memory");
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                   ::"l"(dst + 2 * TILE), "r"(kq + PV), "r"(PV_BYTES) : "memory");
      bulk_commit();
      bulk_wait_read();
    }
  }
  if (!wait.ok) report_timeout(&g_delta_prep_status, a.status);
  if (wp == 0) tmem_dealloc(acc, 64);
}

cudaError_t launch_delta_tc_prep(const DeltaArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk;
  if (!delta_tile_map(&mq, a.q, a.DK, a.Hk, a.T, a.B, a.qs) || !delta_tile_map(&mk, a.k, a.DK, a.Hk, a.T, a.B, a.ks))
    return cudaErrorInvalidValue;
  auto kern = a.l2 ? m3_delta_tc_prep_kernel<true> : m3_delta_tc_prep_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3((unsigned)(a.B * a.Hv * a.nc)), TP_THREADS, SMEM_BYTES, st, false, a, mq, mk);
}

}  // namespace m3
