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
// one lane of a converged warp, the same one every time (lane 0 on a full warp)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// 16 columns of the calling thread's tensor-memory lane
__device__ __forceinline__ void tc_ld16(uint32_t t, float2 (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y), "=f"(v[2].x), "=f"(v[2].y), "=f"(v[3].x),
        "=f"(v[3].y), "=f"(v[4].x), "=f"(v[4].y), "=f"(v[5].x), "=f"(v[5].y), "=f"(v[6].x), "=f"(v[6].y),
        "=f"(v[7].x), "=f"(v[7].y)
      : "r"(t) : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t t, float (&v)[16]) {
  float2 x[8];
  tc_ld16(t, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[2 * j] = x[j].x;
    v[2 * j + 1] = x[j].y;
  }
}
__device__ __forceinline__ void tc_st8(uint32_t t, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(t), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// x = hi + lo + at most 2^-18 |x|: two bf16 terms of a pair (x in the low
// half)
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const float2 r = __ffma2_rn(make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)), f2b(-1.0f), x);
  const __nv_bfloat162 l = __floats2bfloat162_rn(r.x, r.y);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) { split2(make_float2(a, b), hi, lo); }
// values 2 j and 2 j + 1 of 16 consecutive shared-memory floats, as pairs
struct Vec16 {
  const float* p;
  __device__ __forceinline__ float2 operator[](int j) const { return *reinterpret_cast<const float2*>(p + 2 * j); }
};
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
struct TcWork {  // scratch of the warps that make T and P
  float A[TC][TC + 4];
  float M[32][36];
  float gam[TC], ss[2][2 * TC], beta[TC], nk[TC], nq[TC];
  float tot;
};
constexpr int TP_THREADS = 256;

// mbar_wait of m3_common.cuh for the short waits of these kernels' chains:
// a try may sleep up to 20 us, and the clock is looked at every 64th only.
__device__ __forceinline__ bool mbar_wait_fast(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(a), "r"(parity) : "memory");
    if (done) return true;
    if ((i & 63) == 63) {
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > 1000000000ull) return false;
    }
  }
}

// What a kernel's roles share about giving up: a role that ran out of
// patience at a wait goes on without waiting (and without issuing copies or
// MMAs), passing every barrier, so that no other role is left behind.
struct TcWait {
  bool ok = true;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait_fast(bar, parity);
  }
};

// K over Q times K^T into 64 columns (one thread)
__device__ __forceinline__ void tc_mma_kq(uint32_t kq, uint32_t acc, uint64_t* mbk) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint64_t d = tc_desc(kq + (ks >> 2) * (2 * TILE) + (ks & 3) * 32, 16, 1024);
    tc_mma_ss(acc, d, d, tc_idesc(128, 64, false, false), ks > 0);
  }
  tc_commit(mbk);
}
__device__ __forceinline__ float exp_neg(float d) { return ex2(d * LOG2E); }
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

// Which (head, chunk) a block works on at each step.  Either one run of
// chunks of one head (a time segment), or, when there are more heads than
// SMs, an equal share of all chunks of all heads: block s of G has the range
// [s, s + 1) / G of the heads' chunks laid end to end.  It starts with the
// first chunks of the head that the next block ends, hands that head's state
// on, goes through its whole heads, and ends with the last chunks of the
// head that the block before began.  A share is at least a head long, so the
// part handed on is never longer than what its receiver does before it.
struct TcStep {
  int bh, c;          // head (batch row x value head), chunk
  bool first, last;   // of a run
  bool take, give;    // the run starts from, or ends in, a state handed over
};
struct TcWalk {
  int nc, n, len_a, whole, h0, c0, ha, ca;
  bool stream;
  __device__ __forceinline__ TcWalk(const DeltaArgs& a, int seg) {
    nc = a.nc;
    stream = a.stream;
    if (stream) {
      const int64_t total = (int64_t)a.B * a.Hv * nc;
      const int64_t r0 = total * blockIdx.x / gridDim.x, r1 = total * (blockIdx.x + 1) / gridDim.x;
      const int hs = (int)(r0 / nc);
      c0 = (int)(r0 % nc);
      ha = (int)(r1 / nc);
      len_a = (int)(r1 % nc);
      ca = 0;
      h0 = c0 ? hs : hs - 1;  // whole heads are h0 + 1 ...
      whole = ha - h0 - 1;
      n = (int)(r1 - r0);
    } else {
      ha = blockIdx.x;
      ca = seg * a.seg_chunks;
      len_a = n = min(nc, ca + a.seg_chunks) - ca;
      h0 = c0 = whole = 0;
    }
  }
  __device__ __forceinline__ TcStep at(int i) const {
    TcStep r;
    if (i < len_a) {
      r.bh = ha;
      r.c = ca + i;
      r.first = i == 0;
      r.last = i == len_a - 1;
      r.take = false;
      r.give = stream;
    } else if (i < len_a + whole * nc) {
      const int m = i - len_a, w = m / nc;
      r.bh = h0 + 1 + w;
      r.c = m - w * nc;
      r.first = r.c == 0;
      r.last = r.c == nc - 1;
      r.take = r.give = false;
    } else {
      r.bh = h0;
      r.c = c0 + i - len_a - whole * nc;
      r.first = r.c == c0;
      r.last = r.c == nc - 1;
      r.take = true;
      r.give = false;
    }
    return r;
  }
};
// The flag of a state handed over: set behind its writes, waited for (at
// most ten seconds; see TcWalk for why it is hardly ever waited for at all).
__device__ __forceinline__ void flag_set(unsigned* f) {
  asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(f) : "memory");
}
__device__ __forceinline__ bool flag_wait(const unsigned* f) {
  uint64_t t0 = 0;
  for (;;) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(f) : "memory");
    if (v) return true;
    const uint64_t now = global_ns();
    if (t0 == 0) t0 = now;
    else if (now - t0 > 10000000000ull) return false;
    __nanosleep(200);
  }
}

// A chunk's T = (I + A)^-1 and P = scale D o (Q K^T), by 256 threads.
//
// K over Q times K^T is one 128 x 64 MMA; a thread then has half a row of
// K K^T (rows 0-63) or of Q K^T (64-127).  I + A is inverted by blocks: the
// eight 8 x 8 diagonal blocks by forward substitution (a column per thread),
// then 8 -> 16 -> 32 -> 64 with [[P, 0], [-R C P, R]], the last two steps as
// warp products of two bf16 terms.  T and P are stored as two bf16 terms, 17
// bits of mantissa, so that what they multiply keeps f32-grade sums.
//   kq: the stage's K/Q tiles;  acc: 64 tensor-memory columns (all lanes)
//   mbk: tc_mma_kq's commit (parity kpar)
//   g, beta: this thread's token's (threads 0-63; 0 past the sequence)
//   empty: completes (parity epar) when tp and vec may be overwritten
template <bool L2>
__device__ __forceinline__ void tc_make_tp(uint32_t kq, uint32_t acc, TcTP& tp, TcVec& vec, TcWork& w, float g,
                                           float beta, float scale, int pt, uint64_t* mbk, uint32_t kpar,
                                           uint64_t* k_free, uint64_t* empty, uint32_t epar, bool wait_empty, TcWait& wait) {
  constexpr int BAR = 2;
  const int lane = pt & 31, wp = __shfl_sync(~0u, pt >> 5, 0);
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
  bar_sync(BAR, TP_THREADS);
  if (wp < 2) {
    if (wp == 1) gam += w.tot;
    w.gam[pt] = gam;
    w.nk[pt] = L2 ? rsqrtf(w.ss[0][pt] + w.ss[1][pt] + DELTA_L2_EPS) : 1.0f;
    w.nq[pt] = L2 ? rsqrtf(w.ss[0][TC + pt] + w.ss[1][TC + pt] + DELTA_L2_EPS) : 1.0f;
  }
  bar_sync(BAR, TP_THREADS);
  if (wait_empty) wait(empty, epar);
  if (wp < 2) {
    const float gc = w.gam[TC - 1], eg = ex2(gam);
    vec.beta[pt] = beta;
    vec.bfx[pt] = beta * eg * w.nk[pt];
    vec.fu[pt] = ex2(gc - gam) * w.nk[pt];
    vec.fq[pt] = scale * eg * w.nq[pt];
    if (pt == 0) vec.ec = ex2(gc);
  }
  wait(mbk, kpar);
  tmem_fence_after_sync();
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
          *reinterpret_cast<float4*>(&w.A[i][c0 + 2 * m]) = make_float4(v[m].x, v[m].y, v[m + 1].x, v[m + 1].y);
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint4 h, l;
          split2(v[4 * u], h.x, l.x);
          split2(v[4 * u + 1], h.y, l.y);
          split2(v[4 * u + 2], h.z, l.z);
          split2(v[4 * u + 3], h.w, l.w);
          const uint32_t at = sw(i, (c0 >> 3) + u);
          *reinterpret_cast<uint4*>(tp.p_hi + at) = h;
          *reinterpret_cast<uint4*>(tp.p_lo + at) = l;
        }
      }
    }
  }
  tmem_fence_before_sync();
  bar_sync(BAR, TP_THREADS);
  if (pt == 0) mbar_arrive(k_free);  // the accumulator is read: the next chunk's MMA may overwrite it
  if (wp < 4) {  // a 16 x 16 diagonal block per warp
    const int d = wp * 16;
    if (lane < 16) {  // its two 8 x 8 blocks, a column per thread
      const int e = d + (lane & 8), c = lane & 7;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float s0 = i == c ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
        for (int l = 0; l < i; ++l) (l & 1 ? s1 : s0) = fmaf(-w.A[e + i][e + l], x[l], l & 1 ? s1 : s0);
        x[i] = s0 + s1;
      }
      __syncwarp(0xFFFF);
#pragma unroll
      for (int i = 0; i < 8; ++i) w.A[e + i][e + c] = x[i];
    }
    __syncwarp();
    {  // 8 -> 16: two columns of a row per thread
      const int r = lane >> 2, c = (lane & 3) * 2;
      float2 m = f2b(0.0f);
#pragma unroll
      for (int l = 0; l < 8; ++l)
        m = __ffma2_rn(f2b(w.A[d + 8 + r][d + l]), *reinterpret_cast<const float2*>(&w.A[d + l][d + c]), m);
      float* M = &w.M[wp * 8][0];
      *reinterpret_cast<float2*>(M + r * 36 + c) = m;
      __syncwarp();
      m = f2b(0.0f);
#pragma unroll
      for (int l = 0; l < 8; ++l)
        m = __ffma2_rn(f2b(-w.A[d + 8 + r][d + 8 + l]), *reinterpret_cast<const float2*>(M + l * 36 + c), m);
      *reinterpret_cast<float2*>(&w.A[d + 8 + r][d + c]) = m;
    }
    // 16 -> 32: a pair of warps, a 16 x 8 tile each
    bar_sync(4 + (wp >> 1), 64);
    {
      const int e = (wp >> 1) * 32, c = (wp & 1) * 8;
      float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      warp_mma_split<16>(m, &w.A[e + 16][e], TC + 4, &w.A[e][e + c], TC + 4, lane);
      float* M = &w.M[e >> 1][c];  // (a tile's columns are its own warp's)
      warp_mma_store(m, M, 36, lane, 1.0f);
      bar_sync(4 + (wp >> 1), 64);  // both warps have read C
      m[0] = m[1] = m[2] = m[3] = 0.0f;
      warp_mma_split<16>(m, &w.A[e + 16][e + 16], TC + 4, M, 36, lane);
      warp_mma_store(m, &w.A[e + 16][e + c], TC + 4, lane, -1.0f);
    }
  }
  bar_sync(BAR, TP_THREADS);
  {  // 32 -> 64: eight tiles of 16 x 8
    const int r = (wp & 1) * 16, c = (wp >> 1) * 8;
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    warp_mma_split<32>(m, &w.A[32 + r][0], TC + 4, &w.A[0][c], TC + 4, lane);
    warp_mma_store(m, &w.M[r][c], 36, lane, 1.0f);
    bar_sync(BAR, TP_THREADS);
    m[0] = m[1] = m[2] = m[3] = 0.0f;
    warp_mma_split<32>(m, &w.A[32 + r][32], TC + 4, &w.M[0][c], 36, lane);
    warp_mma_store(m, &w.A[32 + r][c], TC + 4, lane, -1.0f);
  }
  bar_sync(BAR, TP_THREADS);
  {  // T as hi and lo: a quarter row per thread
    const int r = pt >> 2, u0 = (pt & 3) * 2;
#pragma unroll
    for (int u = u0; u < u0 + 2; ++u) {
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
  bar_sync(BAR, TP_THREADS);
}

// One chunk's tiles of a [B, T, H, D] tensor as [64 tokens][64 columns],
// 128-byte swizzle; columns past D and tokens past T arrive as zeros.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int col, int head, int tok, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(tok), "r"(b), "r"(smem_u32(bar)) : "memory");
}

// The same tile back (only columns below D and tokens below T are written)
__device__ __forceinline__ void tma_tile_store(const CUtensorMap* map, uint32_t src, int col, int head, int tok, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(col), "r"(head), "r"(tok), "r"(b) : "memory");
}

// The chain kernels' grid: a block per (head, segment), or one per SM in
// equal shares.  Those wait for a state that the block before hands over, so
// they are launched cooperatively (all of them resident at once).
template <typename... Args, typename... Vals>
cudaError_t launch_delta_blocks(void (*kern)(Args...), const DeltaArgs& a, int threads, size_t smem, cudaStream_t st, Vals... maps) {
  cudaLaunchConfig_t cfg{};
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  cfg.gridDim = a.stream ? dim3((unsigned)sms) : dim3((unsigned)(a.B * a.Hv), (unsigned)a.segs);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.stream ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, maps...);
}

}  // namespace m3
