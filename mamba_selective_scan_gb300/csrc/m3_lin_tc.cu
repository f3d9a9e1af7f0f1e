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
  uint4 fk[TC / 2];        // of two tokens' shares in the next state: three bf16 terms, the first negated
  float fo[TC];            // of the start state in a token's output
  // of token j's share in token i's output: pz[0][64 + j - i], and one place
  // earlier in pz[1], so that the two of a pair of j lie on 8 bytes for every i
  float pz[2][2 * TC + 4];
  float dec;         // lam^n
  float pad[3];
};

constexpr uint32_t TC_NEGATE_A = 1u << 13;  // in an MMA's instruction descriptor
constexpr int GROUP = 256;             // threads on the state, on V', on the outputs
constexpr int GW = GROUP / 32;
constexpr int THREADS = 3 * GROUP + 128;  // and a warp each for the MMAs, the loads, the stores
constexpr int STAGES = 3;
constexpr int STAGE = 6 * TILE;        // K, Q (columns 0-63), K, Q (64-127), V, V
constexpr int AGG_STAGES = 5;
constexpr int AGG_STAGE = 4 * TILE;    // K, K, V, V
constexpr int PT = STAGES * STAGE;     // P, and of short sequences its second term
constexpr int OUT = PT + 2 * TILE;     // a chunk's outputs, for the tile store
constexpr int SMALL = OUT + 4 * TILE;  // (f32: four tiles of 32 values)

struct Smem {  // at SMALL
  LinVec vec[8];
  unsigned bad[4][128];  // per row: (step + 1) << 7 | 127 - (first token whose value is not finite)
  unsigned any_bad[4];   // step + 1
  LinInfo info[8];       // (a step's stores come up to two steps later)
  uint64_t full[AGG_STAGES], empty[AGG_STAGES];
  // products done: X (AGG: by step, for two in flight), its first half of the
  // tokens, P, S Q^T, O
  uint64_t mbx[2], mbv, mbp, mbq, mbo, o_free;
  // ready for a step's products, one arrival per warp: V' is there and the X
  // before read; S is there and the outputs before are read; P; the outputs
  uint64_t rdy_x[2], rdy_s, rdy_p, rdy_o;
  uint32_t tmem;
};
constexpr size_t SMEM_BYTES = SMALL + sizeof(Smem) + 1024;
static_assert(SMEM_BYTES <= 232448 && AGG_STAGES * AGG_STAGE <= SMALL, "shared memory of one block");

// tensor-memory columns
constexpr uint32_t T_S = 0;     // S, bf16
constexpr uint32_t T_X = 64;    // V'^T K
constexpr uint32_t T_Q = 192;   // S Q^T
constexpr uint32_t T_O = 256;   // V^T P^T
constexpr uint32_t T_V = 320;   // V' in four terms of 32 columns
constexpr uint32_t T_P = 448;   // Q K^T: row i in lane 32 (i / 16) + i % 16
// and where only the states are wanted: two of each, by step
constexpr uint32_t A_X = 0, A_V = 256;

// Waits of a kernel's roles, few instructions each: a try may sleep up to a
// microsecond, and 2^22 tries end the wait.  A role that ran out of patience
// goes on without waiting (and without issuing copies or MMAs), passing every
// barrier, so that no other role is left behind.
struct LinWait {
  uint32_t tries = 1u << 22;  // 0 once a wait ran out
  __device__ __forceinline__ bool ok() const { return tries != 0; }
  __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 i;\n\t"
        "mov.b32 i, 0;\n"
        "LIN_WAIT_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "@p bra LIN_DONE_%=;\n\t"
        "add.u32 i, i, 1;\n\t"
        "setp.lt.u32 q, i, %0;\n\t"
        "@q bra LIN_WAIT_%=;\n\t"
        "mov.b32 %0, 0;\n"
        "LIN_DONE_%=:\n\t}"
        : "+r"(tries) : "r"(bar), "r"(parity) : "memory");
  }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) { (*this)(smem_u32(bar), parity); }
};
// The stage that a step's tiles are in, and its turn's parity
template <uint32_t N> struct LinStage {
  uint32_t i = 0, par = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      par ^= 1;
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
      pass = (int)(blockIdx.x % (unsigned)a.np);
      item = t.bh * a.np + pass;
      b = t.bh / a.Hv;
      h = t.bh - b * a.Hv;
      w = t.c;
      left = step < walk.len_a ? walk.len_a : walk.nc - t.c;
      flags = (a.p[pass].rev ? F_REV : 0) | (t.take ? F_TAKE : 0) | (t.give ? F_GIVE : 0) | F_FIRST;
    }
    if (left == 1) flags |= F_LAST;
    tok = (flags & F_REV ? a.nc - 1 - w : w) * TC;
    n = min(TC, a.T - tok);
  }
};

// One warp: a step's factors.  Those of tokens stay in their slot while the
// head and the chunk's length do; the state's decay is made anew.  Factors of
// as many tokens as the chunk does not have are 0: of a head that grows they
// may pass f32's range, and what they would multiply are zeros.
__device__ __forceinline__ void lin_factors(const LinArgs& a, const LinInfo& t, LinVec& v, int lane) {
  const bool rev = t.flags & F_REV;
  const float ld = lin_ld(a.ld[t.h]);
  float fk[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = 2 * lane + i;
    const bool there = j < t.n;
    // in time: lam^{n-1-j} and scale lam^{j+1}; backwards: scale lam^{j+1} and lam^{n-1-j}
    const float w = there ? a.scale * expf(ld * (float)j) : 0.0f;
    const float up = there ? a.scale * expf(ld * (float)(j + 1)) : 0.0f, down = there ? expf(ld * (float)(t.n - 1 - j)) : 0.0f;
    fk[i] = rev ? up : down;
    v.fo[j] = rev ? down : up;
    const float before = rev && j ? 0.0f : w, after = rev || !j ? w : 0.0f;
    v.pz[0][TC - j] = before;
    v.pz[1][TC - 1 - j] = before;
    v.pz[0][TC + j] = after;
    v.pz[1][TC - 1 + j] = after;
  }
  // f = f1 + f2 + f3 to f32's last bit
  uint32_t term[3];
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    const __nv_bfloat162 f = __floats2bfloat162_rn(fk[0], fk[1]);
    term[m] = *reinterpret_cast<const uint32_t*>(&f);
    fk[0] -= __low2float(f);
    fk[1] -= __high2float(f);
  }
  v.fk[lane] = make_uint4(term[0], term[1], term[2], term[0] ^ 0x80008000u);
}
// The decay of a chunk of n tokens, rounded to f32 now up and now down so that
// the product over a run's chunks stays within a rounding of the true one (`acc`
// carries what is owed, in last places)
__device__ __forceinline__ float lin_chunk_decay(float ld, int n, float& acc) {
  const LinDecay d = lin_decay(ld, n);
  if (d.near != 1.0f) return d.near;  // above a half: 1 + off
  const float near = 1.0f + d.off, ulp = near < 1.0f ? 0x1p-24f : 0x1p-23f;
  acc += (d.off - (near - 1.0f)) / ulp;
  const float up = acc > 0.5f ? 1.0f : acc < -0.5f ? -1.0f : 0.0f;
  acc -= up;
  return near + up * ulp;
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
__device__ __forceinline__ void tc_ld_rows(uint32_t t, float2 (&v)[8]) {  // 32 lanes x 16 columns
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
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
__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t*>(&x); }

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
// V' enters as four bf16 terms that hold its product with an f32 factor, so
// states are f32 sums of f32-grade products.  S and P enter the outputs'
// products as one term each: a rounding of the size of the outputs' own (1.7e-3
// of them in the 2-norm; all together come to 2.4e-3).  Of up to eight chunks,
// whose outputs are mostly P's, P enters as two terms (2 x 77 tokens: 1.8e-3
// instead of 2.3e-3, for no measurable time).
//
// A value that is not finite would reach the outputs of earlier tokens of its
// chunk, in its own column, through the zeros of P: it is taken out of the V
// tile, and the outputs from its token on are made NaN.  Everything else that
// is not finite (in K, Q, V', S) reaches exactly the rows and columns that it
// reaches in the recurrence.
//
// Roles: warps 0-7 the state, 8-15 V', 16-23 the outputs (P, O^T), warp 24
// issues the MMAs, 25 the loads (and makes the factors), 26 the stores.
//
// Bound: a chunk of a 128 x 128 head is 64 KB, 1.4 us at an SM's share of HBM's
// rate, and takes some 2350 cycles (1.15 us at 2.07 GHz), of which the tensor
// cores work 1670: 1024 on X, 256 on Q K^T (64 rows at half their rate), 256 on
// S Q^T, 128 on O.  The rest is P: its products wait for X to be read, and O for
// the outputs' warps, which read, weigh and write the chunk before first (2100
// cycles a chunk, the longest of the roles).  Measured: 8 x 2048 x 12 heads 49
// us; 4 x 4096 x 40 heads, forward 110 us (650 MB: 87 % of HBM's rate), the three
// backward passes side by side 284 us (1.56 GB, 81 %); 1 x 65536 x 16 heads in
// nine segments 266 us.  Seconds of such work meet the power limit: at 1.7 GHz a
// forward and backward of the former take 457, the latter 302.
//
// Tried: each role's code unrolled by tile (11000 instructions: bound by their
// fetches, 86 us for 8 x 2048 x 12 heads; rolled up it is a third of that); a second warp
// issuing MMAs, and prefetches of later chunks into L2 (no faster); P by four
// warps of its own (8 x 2048 x 12 heads 55 us, heads of 64 x 64 17 % slower), or by
// the warps of V' (55): every wait and arrival takes its share of the issue slots,
// so fewer and longer roles win; barriers polled without suspending (25 %
// slower).
//
// AGG: only the states, each time segment's end from a zero start (into
// seg_end); no queries, no outputs.  FINE: P in two terms.
template <bool AGG, bool FINE>
__global__ void __launch_bounds__(THREADS, 1)
m3_lin_tc_kernel(const __grid_constant__ LinArgs a, const __grid_constant__ LinMaps maps) {
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Smem& s = *reinterpret_cast<Smem*>(base + SMALL);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // uniform for the compiler too
  const int seg = blockIdx.y;
  // neighbouring blocks take the passes of one head: those of dk and dv go
  // through the same chunks at the same time, and share them in L2
  const unsigned np = (unsigned)a.np;
  const TcWalk walk(a.stream, (int64_t)a.B * a.Hv, a.nc, blockIdx.x / np, gridDim.x / np, seg, a.seg_chunks);
  const uint32_t st0 = smem_u32(base);
  // a block's pass, and how many tiles of 64 its keys and its values are: of
  // narrow heads the second ones are neither copied nor multiplied, and the
  // warps whose rows or columns lie there only keep step
  const int pass = (int)(blockIdx.x % np);
  const int DK = a.p[pass].DK, DV = a.p[pass].DV;
  const int nk = DK > 64 ? 2 : 1, nv = DV > 64 ? 2 : 1;
  constexpr int NST = AGG ? AGG_STAGES : STAGES, STB = AGG ? AGG_STAGE : STAGE;
  // X, V' and their barriers: one of each, or (AGG) two in turns
  auto two = [](int n) { return AGG ? n & 1 : 0; };
  auto two_par = [](int n) { return (uint32_t)(AGG ? n >> 1 : n) & 1u; };
  auto at_x = [&](int n) { return AGG ? A_X + (n & 1) * 128 : T_X; };
  auto at_v = [&](int n) { return AGG ? A_V + (n & 1) * 128 : T_V; };
  constexpr int BACK = AGG ? 2 : 1;  // steps after which X and V' are used again

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&s.full[i], 2);  // the copies, the factors
      mbar_init(&s.empty[i], 1);
    }
    for (uint64_t* r : {&s.mbx[0], &s.mbx[1], &s.mbv, &s.mbp, &s.mbq, &s.mbo, &s.o_free}) mbar_init(r, 1);
    for (uint64_t* r : {&s.rdy_x[0], &s.rdy_x[1], &s.rdy_s}) mbar_init(r, 2 * GW);
    for (uint64_t* r : {&s.rdy_p, &s.rdy_o}) mbar_init(r, GW);
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
  auto ready = [&](uint64_t* bar, bool wrote) {  // this warp's tensor-memory accesses so far are done
    if (wrote) tmem_wait_st();
    tmem_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  if (AGG) grid_dep_trigger();
  const uint32_t quad = (uint32_t)(warp & 3), tq = tm + (quad << 21);  // this warp's 32 lanes

  // registers go to the warps that hold the state: (RA + RB + RC) x 256 + RM x
  // 128 is what the block was launched with
  constexpr int LAUNCHED = 65536 / THREADS / 8 * 8, RA = 104, RB = 64, RC = 64, RM = 40;
  static_assert((RA + RB + RC) * GROUP + RM * 128 <= LAUNCHED * THREADS, "registers of the block");
  static_assert(RA >= LAUNCHED && RB <= LAUNCHED && RC <= LAUNCHED && RM <= LAUNCHED, "inc only raises, dec only lowers");
  if (warp >= 3 * GW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RM));
    if (warp == 3 * GW + 2) {  // stores
      if (!AGG && elect_one()) {
#pragma unroll 1
        for (int n = 0; n < walk.n; ++n) {
          wait(&s.rdy_o, n & 1);  // the outputs are in place
          const LinInfo& t = s.info[n & 7];
          const LinPass& p = a.p[t.pass];
          if (wait.ok()) {
            const int cols = p.out_f32 ? 32 : 64;
            for (int col = 0, at = OUT; col < p.DV; col += cols, at += TILE)
              tma_tile_store(&maps.m[t.pass][3], st0 + at, col, t.h, t.tok, t.b);
            bulk_commit();
            bulk_wait_read();
          }
          mbar_arrive(&s.o_free);
        }
        bulk_wait_all();
      }
      __syncwarp();
    } else if (warp == 3 * GW + 1) {  // loads and factors
      grid_dep_wait();  // what the kernels before this one leave is there
      int issued = 0, run = 0;  // run: steps since the factors changed
      float acc = 0.0f;
      LinCursor t;
      LinStage<NST> g;
#pragma unroll 1
      for (int n = 0; n < walk.n; ++n, g.next()) {
        const uint32_t i = g.i;
        t.next(a, walk);
        if (n >= NST) wait(&s.empty[i], g.par ^ 1);
        if (lane == 0) {
          if (wait.ok()) {
            const LinPass& p = a.p[t.pass];
            const CUtensorMap* m = maps.m[t.pass];
            const uint32_t st = st0 + i * STB;
            const int hk = p.kh == 1 ? t.h : t.h / p.kh, hv = p.vh == 1 ? t.h : t.h / p.vh, hq = p.qh == 1 ? t.h : t.h / p.qh;
            uint64_t* bar = &s.full[i];
            mbar_expect_tx(bar, (uint32_t)((AGG ? nk : 2 * nk) + nv) * TILE);
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
              if (blk < nk) tma_tile(st + blk * (AGG ? 1 : 2) * TILE, &m[1], blk * 64, hk, t.tok, t.b, bar);
              if (blk < nv) tma_tile(st + ((AGG ? 2 : 4) + blk) * TILE, &m[2], blk * 64, hv, t.tok, t.b, bar);
              if (!AGG && blk < nk) tma_tile(st + blk * 2 * TILE + TILE, &m[0], blk * 64, hq, t.tok, t.b, bar);
            }
          }
          s.info[n & 7] = t;
        }
        if (wait.ok()) issued = n + 1;
        LinVec& v = s.vec[n & 7];
        if (t.flags & F_FIRST) {
          run = 0;
          acc = 0.0f;
        }
        if (run < 8 || t.n < TC) {
          lin_factors(a, t, v, lane);
          run = t.n < TC ? -8 : run;  // (a short chunk's are made anew in every slot)
        }
        ++run;
        if (lane == 0) v.dec = lin_chunk_decay(a.ld[t.h], t.n, acc);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.full[i]);
      }
      // every product is done (and its arrivals are in) before the block ends
#pragma unroll 1
      for (int n = walk.n; n < walk.n + NST; ++n, g.next())
        if (n >= NST) wait(&s.empty[g.i], g.par ^ 1);
      // after a wait ran out, copies still in flight land before the block's
      // shared memory is given up (bounded)
      if (!wait.ok())
#pragma unroll 1
        for (int m = issued > NST ? issued - NST : 0; m < issued; ++m) mbar_wait(&s.full[m % NST], (m / NST) & 1);
    } else if (warp == 3 * GW) {  // MMAs
      if (elect_one()) {
        const uint64_t pd = tc_desc(st0 + PT, 16, 1024);
        LinStage<NST> g;
#pragma unroll 1
        for (int n = 0; n < walk.n; ++n, g.next()) {
          const uint32_t st = st0 + g.i * STB, par = n & 1;
          // (an address in a descriptor counts 16 bytes)
          const uint64_t kd = tc_desc(st, 16, 1024), qd = tc_desc(st + TILE, 16, 1024);  // K, Q by rows
          const uint64_t kn = tc_desc(st, (AGG ? 1 : 2) * TILE, 1024), vn = tc_desc(st + 4 * TILE, TILE, 1024);  // K, V by columns
          wait(&s.full[g.i], g.par);
          if (!AGG && wait.ok()) {  // Q K^T: the last P was read before its product
            tmem_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const int off = ((ks >> 2) * 2 * TILE + (ks & 3) * 32) >> 4;
              if (ks < 4 * nk) tc_mma_ss(tm + T_P, qd + off, kd + off, tc_idesc(64, 64, false, false), ks > 0);
            }
            tc_commit(&s.mbp);
          }
          wait(&s.rdy_x[two(n)], two_par(n));
          if (wait.ok()) {
            tmem_fence_after_sync();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              // half of the tokens after the other, and few changes of the kind of MMA
              const int half = i >> 3, p = (i & 2) | ((i >> 2 ^ i >> 3) & 1), ks = half * 2 | (i & 1);
              tc_mma_ts(tm + at_x(n), tm + at_v(n) + p * 32 + ks * 8, kn + (ks * 2048 >> 4),
                        (nk > 1 ? tc_idesc(128, 128, false, true) : tc_idesc(128, 64, false, true)) | (p & 1 ? 0u : TC_NEGATE_A), i > 0);
              if (!AGG && i == 7) tc_commit(&s.mbv);  // half of V' can be written again
            }
            tc_commit(&s.mbx[two(n)]);
            if (AGG) tc_commit(&s.empty[g.i]);
          }
          if (AGG) continue;
          wait(&s.rdy_s, par);
          if (wait.ok()) {
            tmem_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              if (ks < 4 * nk) tc_mma_ts(tm + T_Q, tm + T_S + ks * 8, qd + (((ks >> 2) * 2 * TILE + (ks & 3) * 32) >> 4), tc_idesc(128, 64, false, false), ks > 0);
            tc_commit(&s.mbq);
          }
          wait(&s.rdy_p, par);
          if (wait.ok()) {
            tmem_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ss(tm + T_O, vn + (ks * 2048 >> 4), pd + (ks * 32 >> 4), tc_idesc(128, 64, true, false), ks > 0);
            if (FINE) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc_mma_ss(tm + T_O, vn + (ks * 2048 >> 4), pd + ((TILE + ks * 32) >> 4), tc_idesc(128, 64, true, false), true);
            }
            tc_commit(&s.mbo);
            tc_commit(&s.empty[g.i]);
          }
        }
      }
      __syncwarp();
    }
  } else if (warp < GW) {  // the state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(RA));
    const int hf = warp >> 2, row = quad * 32 + lane;  // half of the keys; the row: a value
    const bool idle = hf >= nk || (int)quad * 32 >= DV;
    float2 S[32];  // S^T[row][64 hf + k]

    grid_dep_wait();  // the segments' states, too
    if (lane == 0)  // no X before the first
      for (int i = 0; i < BACK; ++i) mbar_arrive(&s.rdy_x[i]);
    int flags = F_LAST;  // of the step before
    LinStage<NST> g;
#pragma unroll 1
    for (int n = 0; n <= walk.n; ++n, g.next()) {
      if (n > 0) {  // S = lam^n S + X of the step before
        wait(&s.mbx[two(n - 1)], two_par(n - 1));
        tmem_fence_after_sync();
        // (the factors and the step's place are there: the products were issued behind them)
        const float2 dec = f2b(s.vec[(n - 1) & 7].dec);
        if (!idle) {
#pragma unroll
          for (int q = 0; q < 4; q += 2) {
            float2 x[8], y[8];
            tc_ld_rows(tq + at_x(n - 1) + hf * 64 + q * 16, x);
            tc_ld_rows(tq + at_x(n - 1) + hf * 64 + q * 16 + 16, y);
            tc_wait_frag(x);
            tc_wait_frag(y);
#pragma unroll
            for (int k = 0; k < 8; ++k) S[q * 8 + k] = __ffma2_rn(dec, S[q * 8 + k], x[k]);
#pragma unroll
            for (int k = 0; k < 8; ++k) S[q * 8 + 8 + k] = __ffma2_rn(dec, S[q * 8 + 8 + k], y[k]);
          }
        }
        ready(&s.rdy_x[two(n - 1)], false);
        flags = s.info[(n - 1) & 7].flags;
        if (flags & F_LAST) {  // where the run leaves its state
          const LinInfo t = s.info[(n - 1) & 7];
          const LinPass& p = a.p[t.pass];
          if (AGG) {
            float* dst = a.seg_end + (((size_t)t.item * a.segs + seg) * LIN_DMAX + hf * 64) * LIN_DMAX + row;
#pragma unroll
            for (int k = 0; k < 64; ++k) dst[k * LIN_DMAX] = k & 1 ? S[k >> 1].y : S[k >> 1].x;
          } else if (t.flags & F_GIVE) {
            float* dst = a.seg_start + ((size_t)blockIdx.x * LIN_DMAX + hf * 64) * LIN_DMAX + row;
#pragma unroll
            for (int k = 0; k < 64; ++k) dst[k * LIN_DMAX] = k & 1 ? S[k >> 1].y : S[k >> 1].x;
            __threadfence();
            bar_sync(1, GROUP);
            if (tid == 0) flag_set(a.flags + blockIdx.x);
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
        if (n == walk.n) break;
      }
      if (AGG) {
        if (n == 0) {
#pragma unroll
          for (int k = 0; k < 32; ++k) S[k] = f2b(0.0f);
        }
        continue;
      }
      if (flags & F_LAST) {  // the state a run starts from
        wait(&s.full[g.i], g.par);
        const LinInfo t = s.info[n & 7];
        const LinPass& p = a.p[t.pass];
        // (handed on by the share before, of the same pass)
        if (t.flags & F_TAKE && wait.ok()) wait.tries = flag_wait(a.flags + (blockIdx.x - np)) ? wait.tries : 0;
        if (t.w > 0 || a.segs > 1) {
          const size_t slot = t.flags & F_TAKE ? blockIdx.x - np : (size_t)t.item * a.segs + seg;
          const float* src = a.seg_start + (slot * LIN_DMAX + hf * 64) * LIN_DMAX + row;
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
      if (n > 0) {
        wait(&s.mbq, (n - 1) & 1);  // the last state is read
        tmem_fence_after_sync();
      }
      if (!idle) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // S into tensor memory
          uint32_t x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = pack2(S[8 * p + k]);
          tc_st8(tq + T_S + hf * 32 + p * 8, x);
        }
      }
      ready(&s.rdy_s, true);
    }
  } else if (warp < 2 * GW) {
    // V': 32 values (this warp's lanes) of 32 tokens, transposed on their way out of shared memory
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RC));
    const int hf = (warp >> 2) & 1, row = quad * 32 + lane;  // half of the tokens
    const bool idle = (int)quad * 32 >= DV;
    const uint32_t vl = st0 + (AGG ? 2 : 4) * TILE + (quad >> 1) * TILE;
    const uint32_t el = sw(hf * 32 + (lane & 7) + ((lane >> 4) << 3), (quad & 1) * 4 + ((lane >> 3) & 1));
    LinStage<NST> g;
#pragma unroll 1
    for (int n = 0; n < walk.n; ++n, g.next()) {
      // v f to f32's grade, as terms: hi = v f1 rounded (negated, for the rest's
      // sake: its MMAs negate their A), the rest v f1 - hi (exact, eight bits at
      // most), v f2 rounded (negated), and its rest with v f3.  Five packed bf16
      // instructions for two values, where three terms cut from the f32 product
      // take twelve.  (Three terms of this kind are 4 % faster, and 2e-6 off.)
      // Made while the X before runs; written as soon as that is done with the
      // columns.
      uint32_t x[2][8], y[4][8];  // [half of the lanes][fragment], [term][fragment]
      wait(&s.full[g.i], g.par);
      const uint32_t vt = vl + g.i * STB;
      const LinVec& vec = s.vec[n & 7];
      __nv_bfloat162 chk = as_bf2(0);
      if (!idle) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int tp = 0; tp < 2; ++tp) {  // tokens 32 hf + 16 tp ..
            // (values 0-7, tokens 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
            uint32_t (&z)[4] = reinterpret_cast<uint32_t(&)[4]>(x[h][tp * 4]);
            ldmatrix4t(z, vt + (el ^ (h * 32)) + tp * 2048);
#pragma unroll
            for (int i = 0; i < 4; i += 2) chk = __hfma2(as_bf2(z[i]), as_bf2(z[i + 1]), chk);  // finite only if all values are
          }
      }
      auto terms = [&](int h) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const uint4 f = vec.fk[hf * 16 + tb * 4 + (lane & 3)];
          const __nv_bfloat162 f1 = as_bf2(f.x), f2 = as_bf2(f.y), f3 = as_bf2(f.z), n1 = as_bf2(f.w);
          const __nv_bfloat162 n2 = as_bf2(f.y ^ 0x80008000u);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const __nv_bfloat162 v = as_bf2(x[h][tb * 2 + i]), hi = __hmul2_rn(v, n1), t = __hmul2_rn(v, n2);
            y[0][tb * 2 + i] = as_u32(hi);
            y[1][tb * 2 + i] = as_u32(__hfma2(v, f1, hi));
            y[2][tb * 2 + i] = as_u32(t);
            y[3][tb * 2 + i] = as_u32(__hfma2(v, f3, __hfma2(v, f2, t)));
          }
        }
      };
      if (!idle) terms(0);
      if (__any_sync(~0u, (as_u32(__hmul2(chk, as_bf2(0))) & 0x7FFF7FFFu) != 0)) {
        const bool rev = s.info[n & 7].flags & F_REV;
#pragma unroll 1
        for (int tok = hf * 32; tok < hf * 32 + 32; ++tok) {
          const uint32_t at = vt + sw(tok, (row & 63) >> 3) + (row & 7) * 2;
          uint16_t v;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
          if ((v & 0x7F80) == 0x7F80) {
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)0) : "memory");
            atomicMax(&s.bad[n & 3][row], ((unsigned)(n + 1) & 0xFFFFFF) << 7 | (unsigned)(127 - (rev ? TC - 1 - tok : tok)));
            s.any_bad[n & 3] = (unsigned)(n + 1);
          }
        }
        fence_proxy_async();
      }
      if (n >= BACK) {
        wait(AGG || hf ? &s.mbx[two(n)] : &s.mbv, two_par(n) ^ 1);
        tmem_fence_after_sync();
      }
      if (!idle) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h) terms(1);
#pragma unroll
          for (int m = 0; m < 4; ++m) tc_st_frag(tq + (h << 20) + at_v(n) + m * 32 + hf * 16, y[m]);
        }
      }
      ready(&s.rdy_x[two(n)], true);
    }
  } else {  // the outputs
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RB));
    const int hf = (warp >> 2) & 1;  // half of the tokens (of P: of its columns)
    const int i0 = quad * 16, j0 = hf * 32;
    const bool idle = (int)quad * 32 >= DV;  // (P's rows are tokens: no warp is idle there)
    const int pz_at = TC + j0 + 2 * (lane & 3) - i0 - (lane >> 2) - ((lane >> 2) & 1);  // (even)
    const bool out_f32 = a.p[pass].out_f32;
    // where this thread's first value goes: rows of 64 values (bf16), or of 32
    const uint32_t op = st0 + OUT + (out_f32 ? quad * TILE + sw(j0 + 2 * (lane & 3), lane >> 4) + ((lane >> 2) & 3) * 4
                                             : (quad >> 1) * TILE + sw(j0 + (lane & 7) + ((lane >> 4) << 3), (quad & 1) * 4 + ((lane >> 3) & 1)));
#pragma unroll 1
    for (int n = 0; n <= (AGG ? -1 : walk.n); ++n) {
      // O of the step before: values 32 quad .. of tokens 32 hf ..
      float2 o[2][8];  // [half of the lanes][block of 8 tokens][row + 8]
      if (n > 0) {
        const int m = n - 1;
        float2 f[4];
        const float* fo = &s.vec[m & 7].fo[j0 + 2 * (lane & 3)];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) f[tb] = *reinterpret_cast<const float2*>(fo + tb * 8);
        wait(&s.mbo, m & 1);  // (and S Q^T, which was issued before)
        tmem_fence_after_sync();
        if (!idle) {
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
        }
        if (!idle && s.any_bad[m & 3] == (unsigned)n) {
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
      }
      ready(&s.rdy_s, false);
      if (n < walk.n) {  // P: rows 16 quad .., columns 32 hf ..
        float2 x[8];  // [column block of 8][row + 8]
        wait(&s.mbp, n & 1);  // (and with it the factors, which the products were issued behind)
        const bool rev = s.info[n & 7].flags & F_REV;
        tmem_fence_after_sync();
        if (rev ? j0 + 31 >= i0 : j0 <= i0 + 15) {
          tc_ld_frag(tq + T_P + j0, x);
          const float* pz = s.vec[n & 7].pz[(lane >> 2) & 1] + pz_at;
          tc_wait_frag(x);
          float2 chk = f2b(0.0f);
#pragma unroll
          for (int c = 0; c < 8; c += 2) chk = __ffma2_rn(x[c], x[c + 1], chk);  // finite only if all are
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            x[c] = __fmul2_rn(x[c], *reinterpret_cast<const float2*>(pz + 8 * (c >> 1) - 8 * (c & 1)));
          }
          if ((chk.x + chk.y) * 0.0f != 0.0f) {  // what is not finite among pairs that do not count
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int d = i0 + (lane >> 2) + 8 * (c & 1) - j0 - 2 * (lane & 3) - 8 * (c >> 1);  // i - j
              if (rev ? d > 0 : d < 0) x[c].x = 0.0f;
              if (rev ? d > 1 : d < 1) x[c].y = 0.0f;
            }
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) x[c] = f2b(0.0f);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t at = st0 + PT + sw(i0 + (lane & 15), hf * 4 + p * 2 + (lane >> 4));
          stmatrix4<false>(at, pack2(x[4 * p]), pack2(x[4 * p + 1]), pack2(x[4 * p + 2]), pack2(x[4 * p + 3]));
          if (FINE) {
            uint32_t hi, lo[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) split2(x[4 * p + c], hi, lo[c]);
            stmatrix4<false>(at + TILE, lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async();
        ready(&s.rdy_p, false);
      }
      if (n > 0) {
        if (n > 1) wait(&s.o_free, n & 1);
        if (idle) {
        } else if (out_f32) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              // value 16 h + 8 (c & 1) + lane / 4 of this warp's tile, tokens j0 + 8 (c >> 1) + 2 (lane & 3), + 1
              const uint32_t at = (op ^ ((4 * h + 2 * (c & 1)) << 4)) + (c >> 1) * 1024;
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(o[h][c].x) : "memory");
              asm volatile("st.shared.f32 [%0], %1;" ::"r"((at ^ 16u) + 128u), "f"(o[h][c].y) : "memory");
            }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int tp = 0; tp < 2; ++tp)
              stmatrix4<true>((op ^ (h * 32)) + tp * 2048, pack2(o[h][tp * 4]), pack2(o[h][tp * 4 + 1]), pack2(o[h][tp * 4 + 2]), pack2(o[h][tp * 4 + 3]));
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.rdy_o);
      }
    }
  }
  if (!wait.ok()) report_timeout(&g_lin_status, a.status);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0) tmem_dealloc(tm, 512);
}

// The segments' start states: each is the one before, decayed over its
// segment's tokens, and that segment's end from zero.  A float4 per thread.
__global__ void __launch_bounds__(256) m3_lin_seg_kernel(const __grid_constant__ LinArgs a) {
  grid_dep_trigger();
  const int item = blockIdx.x, pass = item % a.np, bh = item / a.np;
  const LinPass& p = a.p[pass];
  const int at = (blockIdx.y * 256 + threadIdx.x) * 4, k = at / LIN_DMAX, v = at % LIN_DMAX;
  const size_t slot = LIN_DMAX * LIN_DMAX;
  const float* end = a.seg_end + (size_t)item * a.segs * slot + at;
  float* start = a.seg_start + (size_t)item * a.segs * slot + at;
  const float ld = a.ld[bh % a.Hv];
  const int whole = a.seg_chunks * TC, odd = a.nc * TC - a.T;  // (backwards, the short chunk comes first)
  const LinDecay d0 = lin_decay(ld, p.rev ? whole - odd : whole), d1 = lin_decay(ld, whole);
  grid_dep_wait();
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.s_in && k < p.DK) {
    const float* src = p.s_in + (size_t)bh * p.DK * p.DV;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v + i < p.DV) x[i] = src[p.st ? (size_t)(v + i) * p.DK + k : (size_t)k * p.DV + v + i];
  }
  *reinterpret_cast<float4*>(start) = make_float4(x[0], x[1], x[2], x[3]);
  for (int s0 = 0; s0 + 1 < a.segs; s0 += 8) {  // eight ends on their way at once
    float4 e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s0 + i + 1 < a.segs) e[i] = *reinterpret_cast<const float4*>(end + (s0 + i) * slot);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (s0 + i + 1 >= a.segs) break;
      const LinDecay d = s0 + i ? d1 : d0;
      x[0] = fmaf(d.near, x[0], fmaf(d.off, x[0], e[i].x));
      x[1] = fmaf(d.near, x[1], fmaf(d.off, x[1], e[i].y));
      x[2] = fmaf(d.near, x[2], fmaf(d.off, x[2], e[i].z));
      x[3] = fmaf(d.near, x[3], fmaf(d.off, x[3], e[i].w));
      *reinterpret_cast<float4*>(start + (s0 + i + 1) * slot) = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

cudaError_t launch_lin_seg(const LinArgs& a, cudaStream_t st) {
  return launch_k(m3_lin_seg_kernel, dim3((unsigned)(a.np * a.B * a.Hv), LIN_DMAX / 8), 256, 0, st, true, a);
}

cudaError_t launch_lin_tc(const LinArgs& a, cudaStream_t st, int sms) {
  LinMaps maps{};
  for (int i = 0; i < a.np; ++i) {
    const LinPass& p = a.p[i];
    if (!delta_tile_map(&maps.m[i][0], p.q, p.DK, a.Hv / p.qh, a.T, a.B, p.qs) ||
        !delta_tile_map(&maps.m[i][1], p.k, p.DK, a.Hv / p.kh, a.T, a.B, p.ks) ||
        !delta_tile_map(&maps.m[i][2], p.v, p.DV, a.Hv / p.vh, a.T, a.B, p.vs))
      return cudaErrorInvalidValue;
    if (!delta_tile_map(&maps.m[i][3], p.out, p.DV, a.Hv, a.T, a.B, p.os, p.out_f32)) return cudaErrorInvalidValue;
  }
  const int64_t items = (int64_t)a.np * a.B * a.Hv;
  cudaError_t e = cudaSuccess;
  if (a.segs > 1) {  // (the last segment's end is nobody's start)
    e = cudaFuncSetAttribute(m3_lin_tc_kernel<true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    if (e == cudaSuccess)
      e = launch_k(m3_lin_tc_kernel<true, false>, dim3((unsigned)items, (unsigned)(a.segs - 1)), THREADS, SMEM_BYTES, st, false, a, maps);
    if (e == cudaSuccess) e = launch_lin_seg(a, st);
  }
  const auto kern = a.nc <= 8 ? m3_lin_tc_kernel<false, true> : m3_lin_tc_kernel<false, false>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e == cudaSuccess && a.stream) e = cudaMemsetAsync(a.flags, 0, LIN_SMS * 4, st);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = a.stream ? dim3(delta_share_blocks((int64_t)a.B * a.Hv, (sms < LIN_SMS ? sms : LIN_SMS) / a.np) * a.np) : dim3((unsigned)items, (unsigned)a.segs);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  if (a.stream) {  // a block may wait for the state of the one before
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = a.stream || a.segs > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, maps);
}

}  // namespace m3
