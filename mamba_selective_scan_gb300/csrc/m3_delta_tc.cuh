// m3_delta_tc.cuh -- shared by the tensor-core kernels of the gated delta
// rule (bf16 activations, chunks of 64 tokens): tcgen05 helpers, the stage
// layout in shared memory and the warpgroup that makes T and P.
#pragma once

#include "m3_delta.cuh"

namespace m3 {

constexpr int TC = 64;                    // tokens per chunk
constexpr int TILE = TC * 128;            // bytes of a [64 rows][64 bf16] tile (128-byte rows, swizzled)
constexpr float FINITE_MAX = 3.0e38f;

// ---- tcgen05 ----
// Shared-memory operand tiles have 128-byte rows in the 128-byte swizzle:
// the 16-byte unit u of row r sits at unit u ^ (r & 7).  The same bytes serve
// as a K-major operand (rows = M or N, the row's 64 elements = K) and as an
// MN-major one (row = K, its elements = M or N).
// K-major: 8 rows (1024 bytes) repeat every sbo; a step of 16 in K is 32 bytes.
// MN-major: 8 rows repeat every sbo, blocks of 64 elements every lbo; a step
// of 16 in K is 16 rows.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 |
         (uint64_t)((sbo >> 4) & 0x3FFF) << 32 | 1ull << 46 | 2ull << 61;
}
// bf16 x bf16 -> f32, M x N, operands K-major unless set
__host__ __device__ constexpr uint32_t tc_idesc(int M, int N, bool a_mn, bool b_mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}
// D (tensor memory) = A (tensor memory) B (shared memory), added to D when acc
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
// the mbarrier gets one arrival when every MMA this thread issued so far is done
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// 32 columns of the calling thread's tensor-memory lane, as f32 or raw words
__device__ __forceinline__ void tc_ld32(uint32_t t, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(t) : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t t, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(t), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// x = hi + lo + at most 2^-18 |x|: two bf16 terms, packed for neighbours a, b
// (a in the low half)
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  const float2 f = __bfloat1622float2(h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - f.x, b - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
// byte offset of the 16-byte unit u of row r in a swizzled tile
__device__ __forceinline__ uint32_t sw(uint32_t r, uint32_t u) { return r * 128 + ((u ^ (r & 7)) << 4); }

// ---- shared memory ----
// A stage holds one chunk's inputs as tiles [64 tokens][64 columns].  K and Q
// alternate (K of columns 0-63, Q of 0-63, K of 64-127, Q of 64-127), so that
// K over Q is one operand of 128 rows whose column halves are 2 tiles apart.
struct TcVec {
  float beta[TC];  // beta
  float bfx[TC];   // beta e^gam nk
  float fu[TC];    // e^{gam_C - gam} nk
  float fq[TC];    // scale e^gam nq
  float ec;        // e^{gam_C}
  float pad[3];
};
struct TcTP {  // one chunk's T and P, each as bf16 hi and lo [64][64]
  unsigned char t_hi[TILE], t_lo[TILE], p_hi[TILE], p_lo[TILE];
};
struct TcWork {  // scratch of the warpgroup that makes T and P
  float A[TC][TC + 4];
  float M[32][36];
  float gam[TC], n[2 * TC], beta[TC];
  float tot;
};

// What a kernel's roles share about giving up: a role that ran out of
// patience at a wait goes on without waiting (and without issuing copies or
// MMAs), passing every barrier, so that no other role is left behind.
struct TcWait {
  bool ok = true;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait(bar, parity);
  }
};

// A chunk's T = (I + A)^-1 and P = scale D o (Q K^T), by 128 threads.
//
// K over Q times K^T is one 128 x 64 MMA; a thread then has a row of K K^T
// (threads 0-63) or of Q K^T (64-127).  I + A is inverted by blocks: the four
// 16 x 16 diagonal blocks by forward substitution (a column per thread), then
// 16 -> 32 -> 64 with [[P, 0], [-R C P, R]].  All of it f32; T and P are
// stored as two bf16 terms, 17 bits of mantissa, so that what they multiply
// keeps f32-grade sums.
//   kq: the stage's K/Q tiles;  acc: 64 tensor-memory columns (all lanes)
//   g, beta: this thread's token's (threads 0-63; 0 past the sequence)
//   empty: completes (parity ep) when tp and vec may be overwritten
template <bool L2>
__device__ __forceinline__ void tc_make_tp(uint32_t kq, uint32_t acc, TcTP& tp, TcVec& vec, TcWork& w, float g,
                                           float beta, float scale, int pt, uint64_t* mbk, uint32_t kpar,
                                           uint64_t* empty, uint32_t epar, bool wait_empty, TcWait& wait) {
  constexpr int BAR = 2;
  const int lane = pt & 31, wp = pt >> 5;
  if (pt == 0 && wait.ok) {
    tmem_fence_after_sync();
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint32_t at = kq + (ks >> 2) * (2 * TILE) + (ks & 3) * 32;
      const uint64_t d = tc_desc(at, 16, 1024);
      tc_mma_ss(acc, d, d, tc_idesc(128, 64, false, false), ks > 0);
    }
    tc_commit(mbk);
  }
  __syncwarp();
  // norms: thread r < 64 has row r of K, r >= 64 row r - 64 of Q
  float nrm = 1.0f;
  if (L2) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(kq + blk * (2 * TILE) + sw(pt, u)));
        const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = __uint_as_float(q[j] << 16), hi = __uint_as_float(q[j] & 0xFFFF0000u);
          s0 = fmaf(lo, lo, s0);
          s1 = fmaf(hi, hi, s1);
        }
      }
    nrm = rsqrtf(s0 + s1 + DELTA_L2_EPS);
  }
  w.n[pt] = nrm;
  float gam = clamp_g(g);
  if (wp < 2) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float up = __shfl_up_sync(~0u, gam, o);
      if (lane >= o) gam += up;
    }
    if (pt == 31) w.tot = gam;
    w.beta[pt] = beta;
  }
  bar_sync(BAR, 128);
  if (wp < 2) {
    if (wp == 1) gam += w.tot;
    w.gam[pt] = gam;
  }
  bar_sync(BAR, 128);
  if (wait_empty) wait(empty, epar);
  if (wp < 2) {
    const float gc = w.gam[TC - 1], eg = expf(gam);
    vec.beta[pt] = beta;
    vec.bfx[pt] = beta * eg * nrm;
    vec.fu[pt] = expf(gc - gam) * nrm;
    vec.fq[pt] = scale * eg * w.n[TC + pt];
    if (pt == 0) vec.ec = expf(gc);
  }
  wait(mbk, kpar);
  tmem_fence_after_sync();
  {
    const int i = pt & (TC - 1);
    const bool isA = wp < 2;
    const float gi = w.gam[i];
    const float f = isA ? w.beta[i] * nrm : scale * nrm;
    float v[32];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      // columns past this warp's last row are zero (rows 0-31: half 1)
      const bool any = half == 0 || (wp & 1);
      if (any) tc_ld32(acc + ((uint32_t)(wp * 32) << 16) + half * 32, v);
#pragma unroll
      for (int c = 0; c < 32; c += 4) {
        const int j = half * 32 + c;
        const float4 gj = *reinterpret_cast<const float4*>(&w.gam[j]);
        const float4 nj = *reinterpret_cast<const float4*>(&w.n[j]);
        const float gv[4] = {gj.x, gj.y, gj.z, gj.w}, nv[4] = {nj.x, nj.y, nj.z, nj.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const bool in = any && (isA ? j + m < i : j + m <= i);
          v[c + m] = in ? f * nv[m] * expf(gi - gv[m]) * v[c + m] : 0.0f;
        }
      }
      if (isA) {
#pragma unroll
        for (int c = 0; c < 32; c += 4)
          *reinterpret_cast<float4*>(&w.A[i][half * 32 + c]) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint4 h, l;
          split2(v[8 * u], v[8 * u + 1], h.x, l.x);
          split2(v[8 * u + 2], v[8 * u + 3], h.y, l.y);
          split2(v[8 * u + 4], v[8 * u + 5], h.z, l.z);
          split2(v[8 * u + 6], v[8 * u + 7], h.w, l.w);
          const uint32_t at = sw(i, half * 4 + u);
          *reinterpret_cast<uint4*>(tp.p_hi + at) = h;
          *reinterpret_cast<uint4*>(tp.p_lo + at) = l;
        }
      }
    }
  }
  tmem_fence_before_sync();  // the accumulator is read: the next chunk's MMA may overwrite it
  bar_sync(BAR, 128);
  if (pt < TC) {  // diagonal blocks
    const int d = (pt >> 4) * 16, c = pt & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[4] = {i == c ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int l = 0; l < i; l += 4) {
        const float4 a = *reinterpret_cast<const float4*>(&w.A[d + i][d + l]);
        s[0] = fmaf(-a.x, x[l], s[0]);
        if (l + 1 < i) s[1] = fmaf(-a.y, x[l + 1], s[1]);
        if (l + 2 < i) s[2] = fmaf(-a.z, x[l + 2], s[2]);
        if (l + 3 < i) s[3] = fmaf(-a.w, x[l + 3], s[3]);
      }
      x[i] = (s[0] + s[1]) + (s[2] + s[3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) w.A[d + i][d + c] = x[i];
  }
  bar_sync(BAR, 128);
  {  // 16 -> 32: two blocks of 64 threads, four columns of a row each
    const int d = (pt >> 6) * 32, r = (pt >> 2) & 15, c = (pt & 3) * 4;
    float4 m = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int l = 0; l < 16; ++l) {
      const float a = w.A[d + 16 + r][d + l];
      const float4 t = *reinterpret_cast<const float4*>(&w.A[d + l][d + c]);
      m.x = fmaf(a, t.x, m.x); m.y = fmaf(a, t.y, m.y); m.z = fmaf(a, t.z, m.z); m.w = fmaf(a, t.w, m.w);
    }
    float* M = &w.M[(pt >> 6) * 16][0];
    *reinterpret_cast<float4*>(M + r * 36 + c) = m;
    bar_sync(BAR, 128);
    m = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int l = 0; l < 16; ++l) {
      const float a = -w.A[d + 16 + r][d + 16 + l];
      const float4 t = *reinterpret_cast<const float4*>(M + l * 36 + c);
      m.x = fmaf(a, t.x, m.x); m.y = fmaf(a, t.y, m.y); m.z = fmaf(a, t.z, m.z); m.w = fmaf(a, t.w, m.w);
    }
    *reinterpret_cast<float4*>(&w.A[d + 16 + r][d + c]) = m;
  }
  bar_sync(BAR, 128);
  {  // 32 -> 64: eight columns of a row per thread
    const int r = pt >> 2, c = (pt & 3) * 8;
    float m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 8
    for (int l = 0; l < 32; ++l) {
      const float a = w.A[32 + r][l];
      const float4 t = *reinterpret_cast<const float4*>(&w.A[l][c]), q = *reinterpret_cast<const float4*>(&w.A[l][c + 4]);
      m[0] = fmaf(a, t.x, m[0]); m[1] = fmaf(a, t.y, m[1]); m[2] = fmaf(a, t.z, m[2]); m[3] = fmaf(a, t.w, m[3]);
      m[4] = fmaf(a, q.x, m[4]); m[5] = fmaf(a, q.y, m[5]); m[6] = fmaf(a, q.z, m[6]); m[7] = fmaf(a, q.w, m[7]);
    }
    *reinterpret_cast<float4*>(&w.M[r][c]) = make_float4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<float4*>(&w.M[r][c + 4]) = make_float4(m[4], m[5], m[6], m[7]);
    bar_sync(BAR, 128);
#pragma unroll
    for (int e = 0; e < 8; ++e) m[e] = 0.0f;
#pragma unroll 8
    for (int l = 0; l < 32; ++l) {
      const float a = -w.A[32 + r][32 + l];
      const float4 t = *reinterpret_cast<const float4*>(&w.M[l][c]), q = *reinterpret_cast<const float4*>(&w.M[l][c + 4]);
      m[0] = fmaf(a, t.x, m[0]); m[1] = fmaf(a, t.y, m[1]); m[2] = fmaf(a, t.z, m[2]); m[3] = fmaf(a, t.w, m[3]);
      m[4] = fmaf(a, q.x, m[4]); m[5] = fmaf(a, q.y, m[5]); m[6] = fmaf(a, q.z, m[6]); m[7] = fmaf(a, q.w, m[7]);
    }
    *reinterpret_cast<float4*>(&w.A[32 + r][c]) = make_float4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<float4*>(&w.A[32 + r][c + 4]) = make_float4(m[4], m[5], m[6], m[7]);
  }
  bar_sync(BAR, 128);
  {  // T as hi and lo: half a row per thread
    const int r = pt >> 1, u0 = (pt & 1) * 4;
#pragma unroll
    for (int u = u0; u < u0 + 4; ++u) {
      const float4 a = *reinterpret_cast<const float4*>(&w.A[r][u * 8]), b = *reinterpret_cast<const float4*>(&w.A[r][u * 8 + 4]);
      uint4 h, l;
      split2(a.x, a.y, h.x, l.x);
      split2(a.z, a.w, h.y, l.y);
      split2(b.x, b.y, h.z, l.z);
      split2(b.z, b.w, h.w, l.w);
      const uint32_t at = sw(r, u);
      *reinterpret_cast<uint4*>(tp.t_hi + at) = h;
      *reinterpret_cast<uint4*>(tp.t_lo + at) = l;
    }
  }
  fence_proxy_async();
  bar_sync(BAR, 128);
}

// One chunk's tiles of a [B, T, H, D] tensor as [64 tokens][64 columns],
// 128-byte swizzle; columns past D and tokens past T arrive as zeros.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int col, int head, int tok, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(tok), "r"(b), "r"(smem_u32(bar)) : "memory");
}

}  // namespace m3
