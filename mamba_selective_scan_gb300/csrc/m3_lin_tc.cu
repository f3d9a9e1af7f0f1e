// m3_lin_tc.cu -- linear attention with a decay for each head on the tensor
// cores: bf16 activations, chunks of 64 tokens, f32 states.
#include <initializer_list>

#include "m3_delta_tc.cuh"
#include "m3_lin.cuh"

namespace m3 {

// nonzero once a kernel here gave up waiting
__device__ unsigned int g_lin_status;

cudaError_t take_lin_status(unsigned* out) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_lin_status, sizeof(v));
  if (e == cudaSuccess && v) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_lin_status, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}

namespace {

static_assert(LIN_C == TC && LIN_DMAX == 128, "the tiles of m3_delta_tc.cuh");

struct LinMaps {  // of each pass: queries, keys, values, outputs
  CUtensorMap m[3][4];
};

// Where a step works: item (pass, batch row, value head) and chunk.  The
// loading warp finds it, the others read it.
struct LinInfo {
  int pass, b, h, item;
  int w;        // chunk in the pass's order
  int tok, n;   // its first token, and its tokens
  int flags;
};
enum { F_REV = 1, F_TAKE = 2, F_GIVE = 4, F_FIRST = 8, F_LAST = 16 };

// A step's factors (lam the head's decay, n the chunk's tokens)
struct LinVec {
  float fk[TC];      // of a token's share in the next state
  float fo[TC];      // of the start state in a token's output
  float pz[2 * TC];  // at 64 + i - j: of token j's share in token i's output
  float near, off;   // lam^n
  float pad[2];
};

constexpr int GROUP = 256;             // threads on the state, and as many on the outputs
constexpr int GW = GROUP / 32;
constexpr int THREADS = 2 * GROUP + 128;  // and a warp each for the MMAs, the loads, the stores
constexpr int STAGES = 3;
constexpr int STAGE = 6 * TILE;        // K, Q (columns 0-63), K, Q (64-127), V, V
constexpr int PT = STAGES * STAGE;     // P
constexpr int OUT = PT + TILE;         // a chunk's outputs, for the tile store
constexpr int SMALL = OUT + 2 * TILE;

struct Smem {  // at SMALL
  LinVec vec[4];
  unsigned bad[4][128];  // per row: (step + 1) << 7 | 127 - (first token whose value is not finite)
  unsigned any_bad[4];   // step + 1
  LinInfo info[8];       // (a step's stores come up to two steps later)
  uint64_t full[STAGES], empty[STAGES];
  uint64_t mbp, mbx, mbq, mbo, o_free;
  uint64_t rdy_v, rdy_x, rdy_s, rdy_q, rdy_p, rdy_o;  // one arrival per warp of a group
  uint32_t tmem;
};
constexpr size_t SMEM_BYTES = SMALL + sizeof(Smem) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of one block");

// tensor-memory columns
constexpr uint32_t T_S = 0;     // S, bf16
constexpr uint32_t T_X = 64;    // V'^T K
constexpr uint32_t T_Q = 192;   // S Q^T
constexpr uint32_t T_O = 256;   // V^T P^T
constexpr uint32_t T_V = 320;   // V' in three terms of 32 columns
constexpr uint32_t T_P = 416;   // Q K^T: row i in lane 32 (i / 16) + i % 16

// Waits of a kernel's roles, few instructions each (their loops have to stay
// in the instruction cache): a try may sleep up to a microsecond, and 2^22
// tries end the wait.  A role that ran out of patience goes on without waiting
// (and without issuing copies or MMAs), passing every barrier, so that no
// other role is left behind.
struct LinWait {
  bool ok = true;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    uint32_t done = ok ? 0u : 1u;
#pragma unroll 1
    for (uint32_t i = 0; !done; ++i) {
      asm volatile(
          "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done) : "r"(a), "r"(parity) : "memory");
      if (!done && i == 1u << 22) {
        ok = false;
        done = 1;
      }
    }
  }
};

struct LinCursor : LinInfo {
  int left, step;  // chunks left in the run, this one too
  __device__ __forceinline__ LinCursor() : left(0), step(-1) {}
  __device__ __forceinline__ void next(const LinArgs& a, const TcWalk& walk) {
    ++step;
    if (--left > 0) {
      ++w;
      flags &= ~F_FIRST;
    } else {
      const TcStep t = walk.at(step);
      item = t.bh;
      const int bh = item / a.np;
      pass = item - bh * a.np;
      b = bh / a.Hv;
      h = bh - b * a.Hv;
      w = t.c;
      left = step < walk.len_a ? walk.len_a : walk.nc - t.c;
      flags = (a.p[pass].rev ? F_REV : 0) | (t.take ? F_TAKE : 0) | (t.give ? F_GIVE : 0) | F_FIRST;
    }
    if (left == 1) flags |= F_LAST;
    tok = (flags & F_REV ? a.nc - 1 - w : w) * TC;
    n = min(TC, a.T - tok);
  }
};

// One warp: a step's factors
__device__ __forceinline__ void lin_factors(const LinArgs& a, const LinInfo& t, LinVec& v, int lane) {
  const bool rev = t.flags & F_REV;
  const float raw = a.ld[t.h], ld = lin_ld(raw);
#pragma unroll 1
  for (int j = lane; j < TC; j += 32) {
    // in time: lam^{n-1-j} and scale lam^{j+1}; backwards: scale lam^{j+1} and lam^{n-1-j}
    const float w = a.scale * expf(ld * (float)j);
    const float up = a.scale * expf(ld * (float)(j + 1)), down = j < t.n ? expf(ld * (float)(t.n - 1 - j)) : 0.0f;
    v.fk[j] = rev ? up : down;
    v.fo[j] = rev ? down : up;
    v.pz[TC + j] = rev && j ? 0.0f : w;
    if (j) v.pz[TC - j] = rev ? w : 0.0f;
  }
  if (lane == 0) {
    const LinDecay d = lin_decay(raw, t.n);
    v.near = d.near;
    v.off = d.off;
  }
}

// Tensor memory in the layout of matrix fragments: 16 lanes x 8 columns per
// four registers; thread l has lane l / 4 (+ 8), columns 2 (l % 4), + 1
__device__ __forceinline__ void tc_ld_frag(uint32_t t, float2 (&v)[8]) {  // 16 lanes x 32 columns
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0].x), "=f"(v[0].y), "=f"(v[1].x), "=f"(v[1].y), "=f"(v[2].x), "=f"(v[2].y), "=f"(v[3].x), "=f"(v[3].y),
        "=f"(v[4].x), "=f"(v[4].y), "=f"(v[5].x), "=f"(v[5].y), "=f"(v[6].x), "=f"(v[6].y), "=f"(v[7].x), "=f"(v[7].y)
      : "r"(t) : "memory");
}
__device__ __forceinline__ void tc_wait_frag(float2 (&a)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(a[0].x), "+f"(a[0].y), "+f"(a[1].x), "+f"(a[1].y), "+f"(a[2].x), "+f"(a[2].y), "+f"(a[3].x), "+f"(a[3].y),
                 "+f"(a[4].x), "+f"(a[4].y), "+f"(a[5].x), "+f"(a[5].y), "+f"(a[6].x), "+f"(a[6].y), "+f"(a[7].x), "+f"(a[7].y)
               :: "memory");
}
// 16 lanes x 16 columns: thread l has lane l / 4 (registers 0, 2, ...; + 8:
// 1, 3, ...), column l % 4 of each four
__device__ __forceinline__ void tc_st_frag(uint32_t t, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"r"(t), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t (&x)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
template <bool TRANS> __device__ __forceinline__ void stmatrix4(uint32_t at, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
  if constexpr (TRANS)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x0), "r"(x1), "r"(x2), "r"(x3) : "memory");
  else
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x0), "r"(x1), "r"(x2), "r"(x3) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float2 x) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x = hi + mid + lo, each a pair of bf16: f32's 24 bits cut into three
__device__ __forceinline__ void split3(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const uint32_t a0 = __float_as_uint(x.x), a1 = __float_as_uint(x.y);
  hi = __byte_perm(a0, a1, 0x7632);
  const float2 r = __ffma2_rn(make_float2(__uint_as_float(a0 & 0xFFFF0000u), __uint_as_float(a1 & 0xFFFF0000u)), f2b(-1.0f), x);
  const uint32_t b0 = __float_as_uint(r.x), b1 = __float_as_uint(r.y);
  mid = __byte_perm(b0, b1, 0x7632);
  const float2 q = __ffma2_rn(make_float2(__uint_as_float(b0 & 0xFFFF0000u), __uint_as_float(b1 & 0xFFFF0000u)), f2b(-1.0f), r);
  lo = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x7632);
}

}  // namespace

// A block walks the chunks of TcWalk; an item is a (pass, batch row, value
// head).  The state is held transposed, S^T [values][keys], one row per
// tensor-memory lane, f32 in registers (half a row per thread), so that the
// products have the state's rows (M = 128) as A and token tiles as B:
//
//   X   = V'^T K            V' = fk V             (N = keys)
//   S^T = lam^n S^T + X
//   O^T = fo (S^T Q^T) + V^T P^T,  P = pz o Q K^T (N = 64 tokens)
//
// Nothing but S^T itself goes from chunk to chunk, and its update is a sum in
// registers: X needs no state, so the products of a chunk run under the
// register work of the ones around it.
//
// V' enters as three bf16 terms, its 24 bits cut in three, so states are f32
// sums of exact products.  S and P enter the outputs' products as one: each
// rounding is of the size of the outputs' own (1.7e-3 in the 2-norm; both come
// to 2.3e-3 at most, their shares of the output being 1 together).
//
// A value that is not finite would reach the outputs of earlier tokens of its
// chunk, in its own column, through the zeros of P: it is taken out of the V
// tile, and the outputs from its token on are made NaN.  Everything else that
// is not finite (in K, Q, V', S) reaches exactly the rows and columns that it
// reaches in the recurrence.
//
// Roles: warps 0-7 the state (V', S^T), warps 8-15 the outputs (P, O^T), warp
// 16 issues the MMAs, warp 17 the loads (and makes the factors), warp 18 the
// stores.
__global__ void __launch_bounds__(THREADS, 1)
m3_lin_tc_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ LinMaps maps) {
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Smem& s = *reinterpret_cast<Smem*>(base + SMALL);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // uniform for the compiler too
  const int seg = blockIdx.y;
  const TcWalk walk(a.stream, (int64_t)a.np * a.B * a.Hv, a.nc, blockIdx.x, gridDim.x, seg, a.seg_chunks);
  const uint32_t st0 = smem_u32(base);

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&s.full[i], 2);  // the copies, the factors
      mbar_init(&s.empty[i], 1);
    }
    for (uint64_t* r : {&s.mbp, &s.mbx, &s.mbq, &s.mbo, &s.o_free}) mbar_init(r, 1);
    for (uint64_t* r : {&s.rdy_v, &s.rdy_x, &s.rdy_s, &s.rdy_q, &s.rdy_p, &s.rdy_o}) mbar_init(r, GW);
    mbar_init_fence();
  }
  if (tid < 512) reinterpret_cast<unsigned*>(s.bad)[tid] = 0;
  if (tid < 4) s.any_bad[tid] = 0;
  if (warp == 0) tmem_alloc(&s.tmem, 512);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = __shfl_sync(~0u, s.tmem, 0);
  LinWait wait;
  auto ready = [&](uint64_t* bar) {  // this warp's tensor-memory accesses so far are done
    tmem_wait_st();
    tmem_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  const uint32_t quad = (uint32_t)(warp & 3), tq = tm + (quad << 21);  // this warp's 32 lanes

  // registers go to the warps that hold the state: 144 x 256 + 72 x 256 + 48 x
  // 128 is what the block was launched with, 96 x 640
  if (warp >= 2 * GW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 2 * GW + 2) {  // stores
      if (elect_one()) {
#pragma unroll 1
        for (int n = 0; n < walk.n; ++n) {
          wait(&s.rdy_o, n & 1);  // the outputs are in place
          const LinInfo& t = s.info[n & 7];
          const LinPass& p = a.p[t.pass];
          if (wait.ok && !p.out_f32) {
            const int h = p.oh == 1 ? t.h : t.h / p.oh;
            tma_tile_store(&maps.m[t.pass][3], st0 + OUT, 0, h, t.tok, t.b);
            if (p.DV > 64) tma_tile_store(&maps.m[t.pass][3], st0 + OUT + TILE, 64, h, t.tok, t.b);
            bulk_commit();
            bulk_wait_read();
          }
          mbar_arrive(&s.o_free);
        }
        bulk_wait_all();
      }
      __syncwarp();
    } else if (warp == 2 * GW + 1) {  // loads and factors
      grid_dep_wait();  // what the kernels before this one leave is there
      int issued = 0;
      LinCursor t;
#pragma unroll 1
      for (int n = 0; n < walk.n; ++n) {
        const int i = n % STAGES;
        t.next(a, walk);
        if (n >= STAGES) wait(&s.empty[i], (n / STAGES - 1) & 1);
        if (lane == 0) {
          if (wait.ok) {
            const LinPass& p = a.p[t.pass];
            const CUtensorMap* m = maps.m[t.pass];
            const uint32_t st = st0 + i * STAGE;
            const int hk = p.kh == 1 ? t.h : t.h / p.kh, hv = p.vh == 1 ? t.h : t.h / p.vh, hq = p.qh == 1 ? t.h : t.h / p.qh;
            uint64_t* bar = &s.full[i];
            mbar_expect_tx(bar, STAGE);
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
              tma_tile(st + blk * 2 * TILE, &m[1], blk * 64, hk, t.tok, t.b, bar);
              tma_tile(st + (4 + blk) * TILE, &m[2], blk * 64, hv, t.tok, t.b, bar);
              tma_tile(st + blk * 2 * TILE + TILE, &m[0], blk * 64, hq, t.tok, t.b, bar);
            }
          }
          s.info[n & 7] = t;
        }
        if (wait.ok) issued = n + 1;
        lin_factors(a, t, s.vec[n & 3], lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.full[i]);
      }
      // after a wait ran out, copies still in flight land before the block's
      // shared memory is given up (bounded)
      if (!wait.ok)
#pragma unroll 1
        for (int m = issued > STAGES ? issued - STAGES : 0; m < issued; ++m) mbar_wait(&s.full[m % STAGES], (m / STAGES) & 1);
    } else if (warp == 2 * GW) {  // MMAs
      if (elect_one()) {
        const uint64_t pd = tc_desc(st0 + PT, 16, 1024);
#pragma unroll 1
        for (int n = 0; n < walk.n; ++n) {
          const uint32_t st = st0 + (n % STAGES) * STAGE, par = n & 1;
          // (an address in a descriptor counts 16 bytes)
          const uint64_t kd = tc_desc(st, 16, 1024), qd = tc_desc(st + TILE, 16, 1024);  // K, Q by rows
          const uint64_t kn = tc_desc(st, 2 * TILE, 1024), vn = tc_desc(st + 4 * TILE, TILE, 1024);  // K, V by columns
          wait(&s.full[n % STAGES], (n / STAGES) & 1);
          if (n > 0) wait(&s.rdy_p, par ^ 1);      // the last chunk's P is read
          if (wait.ok) {                           // Q K^T
            tmem_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const int off = ((ks >> 2) * 2 * TILE + (ks & 3) * 32) >> 4;
              tc_mma_ss(tm + T_P, qd + off, kd + off, tc_idesc(64, 64, false, false), ks > 0);
            }
            tc_commit(&s.mbp);
          }
          wait(&s.rdy_v, par);                     // V' is in tensor memory
          if (n > 0) wait(&s.rdy_x, par ^ 1);      // the last X is read
          if (wait.ok) {
            tmem_fence_after_sync();
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc_mma_ts(tm + T_X, tm + T_V + p * 32 + ks * 8, kn + (ks * 2048 >> 4), tc_idesc(128, 128, false, true), p + ks > 0);
            tc_commit(&s.mbx);
          }
          wait(&s.rdy_s, par);                     // S is in tensor memory
          if (n > 0) wait(&s.rdy_q, par ^ 1);      // the last outputs are read
          if (wait.ok) {
            tmem_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma_ts(tm + T_Q, tm + T_S + ks * 8, qd + (((ks >> 2) * 2 * TILE + (ks & 3) * 32) >> 4), tc_idesc(128, 64, false, false), ks > 0);
            tc_commit(&s.mbq);
          }
          wait(&s.rdy_p, par);                     // P is in shared memory
          if (wait.ok) {
            tmem_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ss(tm + T_O, vn + (ks * 2048 >> 4), pd + (ks * 32 >> 4), tc_idesc(128, 64, true, false), ks > 0);
            tc_commit(&s.mbo);
            tc_commit(&s.empty[n % STAGES]);
          }
        }
      }
      __syncwarp();
    }
  } else if (warp < GW) {  // the state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int hf = warp >> 2, row = quad * 32 + lane;  // half of the keys, and of the tokens; the row: a value
    float2 S[32];  // S^T[row][64 hf + k]
    uint32_t hi[2][8], mid[2][8], lo[2][8];  // V': [half of the lanes][fragment]
    const uint32_t vl = st0 + 4 * TILE + (quad >> 1) * TILE;

    grid_dep_wait();  // the segments' states, too
#pragma unroll 1
    for (int n = 0; n <= walk.n; ++n) {
      if (n < walk.n) {
        // V' of this step: 32 values (this warp's lanes) of 32 tokens,
        // transposed on their way out of shared memory.  Made while the X
        // before it runs, written as soon as that is done with the columns.
        wait(&s.full[n % STAGES], (n / STAGES) & 1);
        const uint32_t vt = vl + (n % STAGES) * STAGE;
        const float* fk = &s.vec[n & 3].fk[hf * 32 + 2 * (lane & 3)];
        float2 chk = f2b(0.0f);
#pragma unroll
        for (int tp = 0; tp < 2; ++tp) {  // tokens 32 hf + 16 tp ..
          const float2 f0 = *reinterpret_cast<const float2*>(fk + tp * 16), f1 = *reinterpret_cast<const float2*>(fk + tp * 16 + 8);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // lanes 16 h ..
            uint32_t x[4];  // (values 0-7, tokens 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
            ldmatrix4t(x, vt + sw(hf * 32 + tp * 16 + (lane & 7) + ((lane >> 4) << 3), (quad & 1) * 4 + h * 2 + ((lane >> 3) & 1)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
              chk = __ffma2_rn(v, f2b(0.0f), chk);  // 0 unless a value is not finite
              split3(__fmul2_rn(v, i < 2 ? f0 : f1), hi[h][tp * 4 + i], mid[h][tp * 4 + i], lo[h][tp * 4 + i]);
            }
          }
        }
        if (__any_sync(~0u, !(chk.x + chk.y == 0.0f))) {
          const bool rev = s.info[n & 7].flags & F_REV;
#pragma unroll 1
          for (int tok = hf * 32; tok < hf * 32 + 32; ++tok) {
            const uint32_t el = vt + sw(tok, (row & 63) >> 3) + (row & 7) * 2;
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(el) : "memory");
            if ((v & 0x7F80) == 0x7F80) {
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(el), "h"((uint16_t)0) : "memory");
              atomicMax(&s.bad[n & 3][row], ((unsigned)(n + 1) & 0xFFFFFF) << 7 | (unsigned)(127 - (rev ? TC - 1 - tok : tok)));
              s.any_bad[n & 3] = (unsigned)(n + 1);
            }
          }
          fence_proxy_async();
        }
      }
      if (n > 0) {
        wait(&s.mbx, (n - 1) & 1);
        tmem_fence_after_sync();
      }
      if (n < walk.n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = tq + (h << 20) + T_V + hf * 16;
          tc_st_frag(at, hi[h]);
          tc_st_frag(at + 32, mid[h]);
          tc_st_frag(at + 64, lo[h]);
        }
        ready(&s.rdy_v);
      }
      if (n > 0) {  // S = lam^n S + X of the step before
        const float2 near = f2b(s.vec[(n - 1) & 3].near), off = f2b(s.vec[(n - 1) & 3].off);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float2 x[8];
          tc_ld16(tq + T_X + hf * 64 + q * 16, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) S[q * 8 + k] = __ffma2_rn(near, S[q * 8 + k], __ffma2_rn(off, S[q * 8 + k], x[k]));
        }
        ready(&s.rdy_x);
        const LinInfo t = s.info[(n - 1) & 7];
        if (t.flags & F_LAST) {  // where the run leaves its state
          const LinPass& p = a.p[t.pass];
          if (t.flags & F_GIVE) {
            float* dst = a.seg_start + ((size_t)t.item * LIN_DMAX + hf * 64) * LIN_DMAX + row;
#pragma unroll
            for (int k = 0; k < 64; ++k) dst[k * LIN_DMAX] = k & 1 ? S[k >> 1].y : S[k >> 1].x;
            __threadfence();
            bar_sync(1, GROUP);
            if (tid == 0) flag_set(a.flags + t.item);
          } else if (p.s_out && t.w == a.nc - 1 && row < p.DV) {  // (never transposed)
            float* dst = p.s_out + (((size_t)t.b * a.Hv + t.h) * p.DK + hf * 64) * p.DV + row;
            const int live = p.DK - hf * 64;  // (a multiple of 8)
#pragma unroll
            for (int k = 0; k < 64; k += 8)
              if (k < live) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  *dst = j & 1 ? S[(k + j) >> 1].y : S[(k + j) >> 1].x;
                  dst += p.DV;
                }
              }
          }
        }
      }
      if (n == walk.n) break;
      {
        const LinInfo t = s.info[n & 7];
        if (t.flags & F_FIRST) {  // the state a run starts from
          const LinPass& p = a.p[t.pass];
          if (t.flags & F_TAKE && wait.ok) wait.ok = flag_wait(a.flags + t.item);
          if (t.w > 0 || a.segs > 1) {
            const float* src = a.seg_start + (((size_t)t.item * a.segs + seg) * LIN_DMAX + hf * 64) * LIN_DMAX + row;
#pragma unroll
            for (int k = 0; k < 64; ++k) (k & 1 ? S[k >> 1].y : S[k >> 1].x) = __ldcg(src + k * LIN_DMAX);
          } else {
            const int live = p.s_in && row < p.DV ? p.DK - hf * 64 : 0;
            const size_t head = ((size_t)t.b * a.Hv + t.h) * p.DK * p.DV;
            const float* src = p.s_in + head + (p.st ? (size_t)row * p.DK + hf * 64 : (size_t)hf * 64 * p.DV + row);
            const int step = p.st ? 1 : p.DV;
#pragma unroll
            for (int k = 0; k < 64; k += 8) {
#pragma unroll
              for (int j = 0; j < 8; ++j) (j & 1 ? S[(k + j) >> 1].y : S[(k + j) >> 1].x) = 0.0f;
              if (k < live) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  (j & 1 ? S[(k + j) >> 1].y : S[(k + j) >> 1].x) = __ldcg(src);
                  src += step;
                }
              }
            }
          }
        }
      }
      if (n > 0) {
        wait(&s.mbq, (n - 1) & 1);  // the last state is read
        tmem_fence_after_sync();
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {  // S into tensor memory
        uint32_t x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = pack2(S[8 * p + k]);
        tc_st8(tq + T_S + hf * 32 + p * 8, x);
      }
      ready(&s.rdy_s);
    }
  } else {  // the outputs
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int hf = (warp >> 2) & 1;  // half of the tokens (of P: of its columns)
    const int i0 = quad * 16, j0 = hf * 32;
#pragma unroll 1
    for (int n = 0; n <= walk.n; ++n) {
      // O of the step before: values 32 quad .. of tokens 32 hf ..
      float2 o[2][8];  // [half of the lanes][block of 8 tokens][row + 8]
      if (n > 0) {
        const int m = n - 1;
        float2 f[4];
        const float* fo = &s.vec[m & 3].fo[j0 + 2 * (lane & 3)];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) f[tb] = *reinterpret_cast<const float2*>(fo + tb * 8);
        wait(&s.mbq, m & 1);
        wait(&s.mbo, m & 1);
        tmem_fence_after_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 q[8];
          tc_ld_frag(tq + (h << 20) + T_Q + j0, q);
          tc_ld_frag(tq + (h << 20) + T_O + j0, o[h]);
          tc_wait_frag(q);
          tc_wait_frag(o[h]);
#pragma unroll
          for (int c = 0; c < 8; ++c) o[h][c] = __ffma2_rn(f[c >> 1], q[c], o[h][c]);
        }
        if (s.any_bad[m & 3] == (unsigned)n) {
          const bool rev = s.info[m & 7].flags & F_REV;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const unsigned b = s.bad[m & 3][quad * 32 + h * 16 + r * 8 + (lane >> 2)];
              const int first = (b >> 7) == ((unsigned)n & 0xFFFFFF) ? 127 - (int)(b & 127) : TC;  // in the pass's order
#pragma unroll
              for (int tb = 0; tb < 4; ++tb) {
                const int tok = j0 + tb * 8 + 2 * (lane & 3);
                if ((rev ? TC - 1 - tok : tok) >= first) o[h][tb * 2 + r].x = __int_as_float(0x7FFFFFFF);
                if ((rev ? TC - 2 - tok : tok + 1) >= first) o[h][tb * 2 + r].y = __int_as_float(0x7FFFFFFF);
              }
            }
        }
        ready(&s.rdy_q);
      }
      if (n < walk.n) {  // P: rows 16 quad .., columns 32 hf ..
        wait(&s.full[n % STAGES], (n / STAGES) & 1);
        const bool rev = s.info[n & 7].flags & F_REV;
        float2 x[8];  // [column block of 8][row + 8]
        wait(&s.mbp, n & 1);
        tmem_fence_after_sync();
        if (rev ? j0 + 31 >= i0 : j0 <= i0 + 15) {
          tc_ld_frag(tq + T_P + j0, x);
          tc_wait_frag(x);
          const int d = i0 + (lane >> 2) - j0 - 2 * (lane & 3);  // i - j of the first value
          const float* pz = &s.vec[n & 3].pz[TC + d];
          const int ds = rev ? -d : d, s1 = rev ? -1 : 1;        // tokens that j lies before i, in the pass's order
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int e = 8 * (c & 1) - 8 * (c >> 1);
            const float f0 = pz[e], f1 = pz[e - 1];
            x[c] = make_float2(ds >= -s1 * e ? x[c].x * f0 : 0.0f, ds >= s1 * (1 - e) ? x[c].y * f1 : 0.0f);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) x[c] = f2b(0.0f);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
          stmatrix4<false>(st0 + PT + sw(i0 + (lane & 15), hf * 4 + p * 2 + (lane >> 4)), pack2(x[4 * p]), pack2(x[4 * p + 1]),
                           pack2(x[4 * p + 2]), pack2(x[4 * p + 3]));
        fence_proxy_async();
        ready(&s.rdy_p);
      }
      if (n > 0) {
        if (n > 1) wait(&s.o_free, n & 1);
        const LinInfo& t = s.info[(n - 1) & 7];
        const LinPass& p = a.p[t.pass];
        if (p.out_f32) {  // straight to memory
          float* dst = static_cast<float*>(p.out) + ((int64_t)t.b * a.T + t.tok) * p.os + (int64_t)(t.h / p.oh) * p.DV;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int r = quad * 32 + h * 16 + (c & 1) * 8 + (lane >> 2), tok = j0 + (c >> 1) * 8 + 2 * (lane & 3);
              if (r < p.DV && tok < t.n) dst[tok * p.os + r] = o[h][c].x;
              if (r < p.DV && tok + 1 < t.n) dst[(tok + 1) * p.os + r] = o[h][c].y;
            }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int tp = 0; tp < 2; ++tp)
              stmatrix4<true>(st0 + OUT + (quad >> 1) * TILE + sw(j0 + tp * 16 + (lane & 7) + ((lane >> 4) << 3), (quad & 1) * 4 + h * 2 + ((lane >> 3) & 1)),
                              pack2(o[h][tp * 4]), pack2(o[h][tp * 4 + 1]), pack2(o[h][tp * 4 + 2]), pack2(o[h][tp * 4 + 3]));
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.rdy_o);
      }
    }
  }
  if (!wait.ok) report_timeout(&g_lin_status, a.status);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0) tmem_dealloc(tm, 512);
}

cudaError_t launch_lin_tc(const LinArgs& a, cudaStream_t st, int sms) {
  LinMaps maps{};
  for (int i = 0; i < a.np; ++i) {
    const LinPass& p = a.p[i];
    if (!delta_tile_map(&maps.m[i][0], p.q, p.DK, a.Hv / p.qh, a.T, a.B, p.qs) ||
        !delta_tile_map(&maps.m[i][1], p.k, p.DK, a.Hv / p.kh, a.T, a.B, p.ks) ||
        !delta_tile_map(&maps.m[i][2], p.v, p.DV, a.Hv / p.vh, a.T, a.B, p.vs))
      return cudaErrorInvalidValue;
    if (!p.out_f32 && !delta_tile_map(&maps.m[i][3], p.out, p.DV, a.Hv / p.oh, a.T, a.B, p.os)) return cudaErrorInvalidValue;
  }
  const int64_t items = (int64_t)a.np * a.B * a.Hv;
  cudaError_t e = cudaFuncSetAttribute(m3_lin_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e == cudaSuccess && a.stream) e = cudaMemsetAsync(a.flags, 0, (size_t)items * 4, st);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = a.stream ? dim3(delta_share_blocks(items, sms)) : dim3((unsigned)items, (unsigned)a.segs);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // shares: a block may wait for the state of the one before
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.stream ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, m3_lin_tc_kernel, a, maps);
}

}  // namespace m3
