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
  float D[4][16][20];  // the diagonal blocks of I + A, then of T
  float M[4][8][12];
  float beta[TC], nk[TC], nq[TC];
  uint4 lost;  // bits: tokens with a k (x: 0-31, y: 32-63) or a gate (z: even, w: odd) that is not finite
};

struct TcGates {  // behind the factors, where the tiles' alignment leaves room
  float gam[TC], lo[TC];  // the gates' sum (lo in powers of e)
  float nj[TC];           // nk (1 - lo)
};

// shared memory: T (A at first), P, the factors, the gates; the K/Q tiles
constexpr int KQ = ((int)sizeof(TcPrep) + 1023) / 1024 * 1024;
static_assert(sizeof(TcPrep) + sizeof(TcGates) <= KQ && sizeof(TcPrep) % 16 == 0, "the gates' place");
constexpr int WORK = KQ + 4 * TILE;
constexpr size_t SMEM_BYTES = WORK + sizeof(TcWork) + 1024;
constexpr int PREP_PER_SM = 3;
static_assert(PREP_PER_SM * (SMEM_BYTES + 1024 + 256) <= 233472, "shared memory of an SM");

// The products of the inversion are far too small for a tcgen05 product and
// its way through tensor memory: D (16 x 8) += A (16 x 16) B (16 x 8) by one
// warp, both operands as two bf16 terms (lo x lo is below f32's rounding).
struct Terms {  // an operand's registers: hi and lo
  uint32_t h[4], l[4];
};
__device__ __forceinline__ void warp_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void warp_mma3(float (&d)[4], const Terms& a, uint32_t bh0, uint32_t bh1, uint32_t bl0, uint32_t bl1) {
  warp_mma(d, a.h, bh0, bh1);
  warp_mma(d, a.l, bh0, bh1);
  warp_mma(d, a.h, bl0, bl1);
}
template <bool TRANS> __device__ __forceinline__ void ldmatrix4(uint32_t (&x)[4], uint32_t at) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
// the 16 x 16 block at (row, col) of the tiles hi at `t`, lo behind it, as the
// A operand, or as the B operand (registers 0, 1: its first eight columns)
__device__ __forceinline__ void block_a(Terms& x, uint32_t t, int row, int col, int lane) {
  const uint32_t at = t + sw(row + (lane & 15), (col >> 3) + (lane >> 4));
  ldmatrix4<false>(x.h, at);
  ldmatrix4<false>(x.l, at + TILE);
}
__device__ __forceinline__ void block_b(Terms& x, uint32_t t, int row, int col, int lane) {
  const uint32_t at = t + sw(row + (lane & 15), (col >> 3) + (lane >> 4));
  ldmatrix4<true>(x.h, at);
  ldmatrix4<true>(x.l, at + TILE);
}
// two products' sums side by side (16 x 16) as the next one's A operand
__device__ __forceinline__ void sums_a(Terms& x, const float (&m0)[4], const float (&m1)[4]) {
  split2(m0[0], m0[1], x.h[0], x.l[0]);
  split2(m0[2], m0[3], x.h[1], x.l[1]);
  split2(m1[0], m1[1], x.h[2], x.l[2]);
  split2(m1[2], m1[3], x.h[3], x.l[3]);
}
// -d to the 16 x 8 block at (row, col) of the tiles
__device__ __forceinline__ void block_store(unsigned char* t, const float (&d)[4], int row, int col, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h, l;
    split2(-d[2 * i], -d[2 * i + 1], h, l);
    const uint32_t at = sw(row + i * 8 + (lane >> 2), col >> 3) + (lane & 3) * 4;
    *reinterpret_cast<uint32_t*>(t + at) = h;
    *reinterpret_cast<uint32_t*>(t + TILE + at) = l;
  }
}

}  // namespace

// A chunk's T = (I + A)^-1 and P = scale D o (Q K^T), by blocks of 256
// threads, three per SM, one (chunk, head) after the other.  Half the warps
// invert; the others meanwhile do what the next item needs of its inputs.
//
// K over Q times K^T is one 128 x 64 MMA; a thread then has half a row of
// K K^T (rows 0-63) or of Q K^T (64-127).  I + A is inverted by blocks: the
// eight 8 x 8 diagonal blocks by forward substitution (a column per thread)
// and 8 -> 16 in f32, then 16 -> 32 -> 64 with [[P, 0], [-(R C) P, R]] as warp
// products of two bf16 terms, whose operands are read from the tiles that T
// is stored in; the sums R C stay in registers as the next product's operand.
// T and P are stored as two bf16 terms, 17 bits of mantissa, so that what
// they multiply keeps f32-grade sums.
//
// From the first token on whose k, g or beta is not finite, T's rows are the
// identity's (so that nothing of them meets the zeros in the rows above), P's
// rows and beta are NaN: the forward's outputs and the state are NaN from that
// token on and untouched before it, the adjoint is NaN.
//
// The chain kernels that follow (the forward's and the reverse pass's, with
// time segments each twice) go through a head's chunks one after the other and
// are bound by that chain; this work has no order, so it is done here once,
// with full SMs, and read back (34 KB per chunk and head).
//
// Bound by HBM for many chunks (32 KB in, 34 KB out per item), between events
// with L2 flushed before: 16384 items take 192 us, 5.7 TB/s; 4 x 4096 x 40 heads
// (K and Q of 20 heads) 123 us; 8 x 2048 x 12 heads 45 us.  10, 6 and 2 us of
// it are the gates' second term and the search for values that are not finite.
// With I + A's blocks in f32, split at every use, and a block per item it was
// bound by shared memory and barriers, and took a third longer.
template <bool L2>
__global__ void __launch_bounds__(TP_THREADS, PREP_PER_SM)
m3_delta_tc_prep_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap mk) {
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full, mbk;
  __shared__ uint32_t slot;
  TcVec& vec = *reinterpret_cast<TcVec*>(base + 4 * TILE);
  TcWork& w = *reinterpret_cast<TcWork*>(base + WORK);
  TcGates& gt = *reinterpret_cast<TcGates*>(base + sizeof(TcPrep));
  const int pt = threadIdx.x, lane = pt & 31, wp = __shfl_sync(~0u, pt >> 5, 0);
  const uint32_t sb = smem_u32(base), kq = sb + KQ;
  const uint32_t items = (uint32_t)(a.B * a.Hv * a.nc), nc = (uint32_t)a.nc, hv = (uint32_t)a.Hv;  // (below 2^31)
  const bool io = pt == TP_THREADS - 32;  // this thread copies (its warp has the least to do)
  const float scale = a.scale;
  uint32_t acc = 0;
  TcWait wait;
  if (io) {
    mbar_init(&full, 1);
    mbar_init(&mbk, 1);
    mbar_init_fence();
  }
  // a chunk's K and Q (one thread)
  int n_kq = 0;  // loads issued
  auto load_kq = [&](uint32_t it) {
    ++n_kq;
    const uint32_t bh = it / nc, bb = bh / hv;
    const int c = (int)(it - bh * nc), b = (int)bb, hk = (int)((bh - bb * hv) / (uint32_t)a.share);
    mbar_expect_tx(&full, 4 * TILE);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      tma_tile(kq + blk * 2 * TILE, &mk, blk * 64, hk, c * TC, b, &full);
      tma_tile(kq + blk * 2 * TILE + TILE, &mq, blk * 64, hk, c * TC, b, &full);
    }
  };
  // what needs only an item's inputs, by warps 4-7 under the inversion of the
  // item before: the product of K over Q with K^T, the gates (two tokens per
  // lane of warp 4; 0 past the sequence), the rows' norms (a row of K over Q
  // per thread) and, once K and Q are read, the next item's copies
  __nv_bfloat16 g_in[2], beta_in[2];
  auto load_gates = [&](uint32_t it) {
    const uint32_t bh = it / nc, b = bh / hv, h = bh - b * hv;
    const int t = (int)(it - bh * nc) * TC + lane * 2;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      g_in[j] = beta_in[j] = __float2bfloat16_rn(0.0f);
      if (t + j < a.T) {
        const int64_t at = ((int64_t)b * a.T + t + j) * hv + h;
        g_in[j] = static_cast<const __nv_bfloat16*>(a.g)[at];
        beta_in[j] = static_cast<const __nv_bfloat16*>(a.beta)[at];
      }
    }
  };
  auto inputs = [&](uint32_t it, uint32_t par) {
    wait(&full, par);
    if (wp == 7) {
      tmem_fence_after_sync();
      if (elect_one() && wait.ok) tc_mma_kq(kq, acc, &mbk);
      __syncwarp();
    }
    if (wp == 4) {
      const float g0 = clamp_g(__bfloat162float(g_in[0])) * LOG2E;  // exponents in powers of two
      const float g1 = clamp_g(__bfloat162float(g_in[1])) * LOG2E;
      const float b0 = __bfloat162float(beta_in[0]), b1 = __bfloat162float(beta_in[1]);
      w.lost.z = __ballot_sync(~0u, !(fmaf(g0, 0.0f, b0 * 0.0f) == 0.0f));
      w.lost.w = __ballot_sync(~0u, !(fmaf(g1, 0.0f, b1 * 0.0f) == 0.0f));
      const GateSum sum = gate_scan(gate_add({g0, 0.0f}, {g1, 0.0f}), lane);
      GateSum even = {__shfl_up_sync(~0u, sum.h, 1), __shfl_up_sync(~0u, sum.l, 1)};
      if (lane == 0) even = {0.0f, 0.0f};
      even = gate_add(even, {g0, 0.0f});
      *reinterpret_cast<float2*>(&gt.gam[lane * 2]) = make_float2(even.h, sum.h);
      *reinterpret_cast<float2*>(&gt.lo[lane * 2]) = make_float2(even.l * LN2, sum.l * LN2);
      *reinterpret_cast<float2*>(&w.beta[lane * 2]) = make_float2(b0, b1);
      if (it + gridDim.x < items) load_gates(it + gridDim.x);
    }
    const int r = pt - 128;  // row of K over Q
    float nrm = 1.0f;
    if (L2 || wp < 6) {
      auto row16 = [&](int u) {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(kq + (u >> 3) * (2 * TILE) + sw(r, u & 7)));
        return x;
      };
      float2 s0 = f2b(0.0f), s1 = f2b(0.0f);
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const uint4 x = row16(u);
        const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 e = make_float2(__uint_as_float(q[j] << 16), __uint_as_float(q[j] & 0xFFFF0000u));
          (j & 1 ? s1 : s0) = __ffma2_rn(e, e, j & 1 ? s1 : s0);
        }
      }
      const float sum = (s0.x + s0.y) + (s1.x + s1.y);
      if (L2) nrm = rsqrtf(sum + DELTA_L2_EPS);
      if (wp < 6) {
        bool lost = false;
        if (!(sum <= FINITE_MAX)) {  // (finite values whose squares overflow are none of these)
          for (int u = 0; u < 16; ++u) {
            const uint4 x = row16(u);
            const uint32_t q[4] = {x.x, x.y, x.z, x.w};
            for (int j = 0; j < 4; ++j) lost |= (q[j] & 0x7F80u) == 0x7F80u || (q[j] & 0x7F800000u) == 0x7F800000u;
          }
        }
        (wp == 4 ? w.lost.x : w.lost.y) = __ballot_sync(~0u, lost);
      }
    }
    (r < TC ? w.nk : w.nq)[r & (TC - 1)] = nrm;
    bar_sync(3, 128);  // K and Q are read
    if (wp < 6) gt.nj[r] = nrm * (1.0f - gt.lo[r]);
    if (io && it + gridDim.x < items) {
      wait(&mbk, par);
      if (wait.ok) load_kq(it + gridDim.x);
    }
    __syncwarp();
  };
  if (io) load_kq(blockIdx.x);
  if (wp == 4) load_gates(blockIdx.x);
  if (wp == 0) tmem_alloc(&slot, 64);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  acc = __shfl_sync(~0u, slot, 0);
  grid_dep_trigger();  // the chain's blocks may come up (they need this block's tensor memory only once it is given back)
  if (wp >= 4) inputs(blockIdx.x, 0);
  uint32_t par = 0;
  for (uint32_t it = blockIdx.x; it < items; it += gridDim.x, par ^= 1) {
    if (io) bulk_wait_read();  // the item before has left P's place
    __syncthreads();
    wait(&mbk, par);
    tmem_fence_after_sync();
    const int row = (wp & 3) * 32 + lane, ch = wp >> 2;  // row of K over Q, half of its columns
    int lost = TC;  // first token whose k, g or beta is not finite
    if (const uint4 at = w.lost; at.x | at.y | at.z | at.w) {
      if (at.x | at.y) lost = at.x ? __ffs(at.x) - 1 : __ffs(at.y) + 31;
      if (at.z) lost = min(lost, 2 * __ffs(at.z) - 2);
      if (at.w) lost = min(lost, 2 * __ffs(at.w) - 1);
    }
    if (wp == 4 || wp == 6) {  // (without work in the next step)
      const int t = (wp - 4) * 16 + lane;
      const float gc = gt.gam[TC - 1], gam = gt.gam[t], lc = gt.lo[TC - 1], lo = gt.lo[t];
      const float eg = ex2(gam) * (1.0f + lo), beta = t < lost ? w.beta[t] : NAN;
      vec.beta[t] = beta;
      vec.bfx[t] = beta * eg * w.nk[t];
      vec.fu[t] = ex2(gc - gam) * (1.0f + (lc - lo)) * w.nk[t];
      vec.fq[t] = scale * eg * w.nq[t];
      if (t == 0) vec.ec = ex2(gc) * (1.0f + lc);
    }
    {
      const int i = row & (TC - 1);
      const bool isA = (wp & 3) < 2;
      const float gi = gt.gam[i];
      const float f = (isA ? w.beta[i] * w.nk[i] : scale * w.nq[i]) * (1.0f + gt.lo[i]);
      const int last = isA ? i - 1 : i;  // last column that counts
      const bool any = ch == 0 || (wp & 1);   // rows 0-31 have nothing in the second half,
      const bool all = ch == 0 && (wp & 1);   // rows 32-63 everything in the first
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c0 = ch * 32 + q * 16;
        float2 v[8];
        if (any) {
          tc_ld16(acc + ((uint32_t)((wp & 3) * 32) << 16) + c0, v);
          const Reg16 gj{&gt.gam[c0]}, nj{&gt.nj[c0]};
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
        if (i >= lost) {
#pragma unroll
          for (int m = 0; m < 8; ++m) v[m] = f2b(isA ? 0.0f : NAN);
        }
        unsigned char* t = base + (isA ? 0 : 2 * TILE);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint4 h, l;
          split2(v[4 * u], h.x, l.x);
          split2(v[4 * u + 1], h.y, l.y);
          split2(v[4 * u + 2], h.z, l.z);
          split2(v[4 * u + 3], h.w, l.w);
          const uint32_t at = sw(i, (c0 >> 3) + u);
          *reinterpret_cast<uint4*>(t + at) = h;
          *reinterpret_cast<uint4*>(t + TILE + at) = l;
        }
        if (isA && c0 == (i & 48)) {
          float* d = w.D[i >> 4][i & 15];
#pragma unroll
          for (int m = 0; m < 8; m += 2) *reinterpret_cast<float4*>(d + 2 * m) = make_float4(v[m].x, v[m].y, v[m + 1].x, v[m + 1].y);
        }
      }
    }
    tmem_fence_before_sync();
    fence_proxy_async();
    __syncthreads();
    unsigned char* dst = a.tp + (size_t)it * a.tp_stride;
    if (io && wait.ok) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                   ::"l"(dst + 2 * TILE), "r"(sb + 2 * TILE), "r"((int)sizeof(TcPrep) - 2 * TILE) : "memory");
      bulk_commit();
    }
    if (wp >= 4 && it + gridDim.x < items) inputs(it + gridDim.x, par ^ 1);
    if (wp < 4) {
      // a 16 x 16 diagonal block per warp, f32
      float (&D)[16][20] = w.D[wp];
      if (lane < 16) {  // its two 8 x 8 blocks, a column per thread
        const int e = lane & 8, c = lane & 7;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float s0 = i == c ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
          for (int l = 0; l < i; ++l) (l & 1 ? s1 : s0) = fmaf(-D[e + i][e + l], x[l], l & 1 ? s1 : s0);
          x[i] = s0 + s1;
        }
        __syncwarp(0xFFFF);
#pragma unroll
        for (int i = 0; i < 8; ++i) D[e + i][e + c] = x[i];
      }
      __syncwarp();
      {  // 8 -> 16: two columns of a row per thread
        const int r = lane >> 2, c = (lane & 3) * 2;
        float2 m = f2b(0.0f);
#pragma unroll
        for (int l = 0; l < 8; ++l) m = __ffma2_rn(f2b(D[8 + r][l]), *reinterpret_cast<const float2*>(&D[l][c]), m);
        *reinterpret_cast<float2*>(&w.M[wp][r][c]) = m;
        __syncwarp();
        m = f2b(0.0f);
#pragma unroll
        for (int l = 0; l < 8; ++l)
          m = __ffma2_rn(f2b(-D[8 + r][8 + l]), *reinterpret_cast<const float2*>(&w.M[wp][l][c]), m);
        *reinterpret_cast<float2*>(&D[8 + r][c]) = m;
        __syncwarp();
      }
      {  // to the tiles: half a row per thread
        const float4 x = *reinterpret_cast<const float4*>(&D[lane >> 1][(lane & 1) * 8]);
        const float4 y = *reinterpret_cast<const float4*>(&D[lane >> 1][(lane & 1) * 8 + 4]);
        uint4 h, l;
        split2(x.x, x.y, h.x, l.x);
        split2(x.z, x.w, h.y, l.y);
        split2(y.x, y.y, h.z, l.z);
        split2(y.z, y.w, h.w, l.w);
        const uint32_t at = sw(wp * 16 + (lane >> 1), wp * 2 + (lane & 1));
        *reinterpret_cast<uint4*>(base + at) = h;
        *reinterpret_cast<uint4*>(base + TILE + at) = l;
      }
      {  // 16 -> 32 by a pair of warps, eight columns each
        const int e = (wp >> 1) * 32, c = wp & 1;
        bar_sync(1 + (wp >> 1), 64);
        Terms x, y;
        float m[2][4] = {}, o[4] = {};
        block_a(x, sb, e + 16, e + 16, lane);
        block_b(y, sb, e + 16, e, lane);
#pragma unroll
        for (int n = 0; n < 2; ++n) warp_mma3(m[n], x, y.h[2 * n], y.h[2 * n + 1], y.l[2 * n], y.l[2 * n + 1]);
        sums_a(x, m[0], m[1]);
        block_b(y, sb, e, e, lane);
        warp_mma3(o, x, c ? y.h[2] : y.h[0], c ? y.h[3] : y.h[1], c ? y.l[2] : y.l[0], c ? y.l[3] : y.l[1]);
        bar_sync(1 + (wp >> 1), 64);  // both warps have read C
        block_store(base, o, e + 16, e + c * 8, lane);
      }
      {  // 32 -> 64 by four warps, 16 x 16 each; what is zero by their triangles is left out
        const int r = wp & 1, c = wp >> 1;
        bar_sync(4, 128);
        Terms x, y;
        float m[4][4] = {}, o[2][4] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (k > r) break;
          block_a(x, sb, 32 + r * 16, 32 + k * 16, lane);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (j < c) continue;
            block_b(y, sb, 32 + k * 16, j * 16, lane);
#pragma unroll
            for (int n = 0; n < 2; ++n) warp_mma3(m[2 * j + n], x, y.h[2 * n], y.h[2 * n + 1], y.l[2 * n], y.l[2 * n + 1]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (k < c) continue;
          sums_a(x, m[2 * k], m[2 * k + 1]);
          block_b(y, sb, k * 16, c * 16, lane);
#pragma unroll
          for (int n = 0; n < 2; ++n) warp_mma3(o[n], x, y.h[2 * n], y.h[2 * n + 1], y.l[2 * n], y.l[2 * n + 1]);
        }
        bar_sync(4, 128);  // all have read C
#pragma unroll
        for (int n = 0; n < 2; ++n) block_store(base, o[n], 32 + r * 16, c * 16 + n * 8, lane);
      }
    }
    __syncthreads();
    // T leaves through registers, so that its place is free by the next barrier
    for (int at = pt * 16; at < 2 * TILE; at += TP_THREADS * 16)
      *reinterpret_cast<uint4*>(dst + at) = *reinterpret_cast<const uint4*>(base + at);
  }
  if (io) {
    bulk_wait_read();
    // after a wait ran out, copies still in flight land first (bounded)
    if (!wait.ok) mbar_wait(&full, (n_kq - 1) & 1);
  }
  if (!wait.ok) report_timeout(&g_delta_prep_status, a.status);
  if (wp == 0) {
    __syncwarp();
    tmem_dealloc(acc, 64);
  }
}

cudaError_t launch_delta_tc_prep(const DeltaArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk;
  if (!delta_tile_map(&mq, a.q, a.DK, a.Hk, a.T, a.B, a.qs) || !delta_tile_map(&mk, a.k, a.DK, a.Hk, a.T, a.B, a.ks))
    return cudaErrorInvalidValue;
  auto kern = a.l2 ? m3_delta_tc_prep_kernel<true> : m3_delta_tc_prep_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e != cudaSuccess) return e;
  int sms = 0;
  e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)a.B * a.Hv * a.nc, blocks = (int64_t)PREP_PER_SM * sms;
  return launch_k(kern, dim3((unsigned)(items < blocks ? items : blocks)), TP_THREADS, SMEM_BYTES, st, false, a, mq, mk);
}

}  // namespace m3
