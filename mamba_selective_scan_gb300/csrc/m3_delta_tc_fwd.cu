// m3_delta_tc_fwd.cu -- the gated delta rule's forward on the tensor cores:
// bf16 activations, chunks of 64 tokens, f32-grade sums.
#include <initializer_list>

#include "m3_delta_tc.cuh"

namespace m3 {

// nonzero once a kernel here gave up waiting
__device__ unsigned int g_delta_fwd_status;

cudaError_t take_delta_fwd_status(unsigned* out) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_delta_fwd_status, sizeof(v));
  if (e == cudaSuccess && v) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_delta_fwd_status, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}

namespace {

constexpr int CHAIN = 512;                   // threads on the state: a row's columns in quarters
constexpr int THREADS = CHAIN + 64;  // and a warp for the MMAs, one for the copies
constexpr int KQ = 4 * TILE;      // one chunk's K/Q tiles; two stages
constexpr int TP = 2 * KQ;        // T and P, two stages
constexpr int TP_BYTES = (int)sizeof(TcTP);
constexpr int VO = TP + 2 * TP_BYTES;  // V, two stages of two tiles
constexpr int OUT = VO + 4 * TILE;     // a chunk's outputs, for the tile store
constexpr int SMALL = OUT + 2 * TILE;

struct Smem {  // at SMALL
  TcVec vec[3];  // (a chunk's last use is in the next one's step)
  int bad[128];
  uint64_t kq_full[2], v_full[2], mbx, mbq, mbu, mbd, mbo, o_free;
  uint64_t rdy_s, rdy_q, rdy_o, rdy_r, rdy_u, rdy_v;  // one arrival per chain warp
  uint32_t tmem;
};
constexpr size_t SMEM_BYTES = SMALL + sizeof(Smem) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of one block");

// tensor-memory columns
constexpr uint32_t T_S = 0;     // S: per 16 columns k, 8 of hi and 8 of lo; also the 128 columns of U'^T K
constexpr uint32_t T_X = 128;   // S K^T, then U
constexpr uint32_t T_Q = 192;   // S Q^T
constexpr uint32_t T_R = 256;   // R as hi, lo (32 + 32), then U' = U e^{gam_C - gam}
constexpr uint32_t T_U = 320;   // U as hi, lo
constexpr uint32_t T_O = 384;   // U P^T

}  // namespace

// A block walks the chunks of TcWalk.  The state is held transposed, S^T [head_v][head_k], one row per tensor-memory
// lane, so that every product of the chain has the state's rows (M = 128) as
// its A operand in tensor memory and token tiles as B in shared memory, and
// every per-token factor is a column factor:
//
//   X = S^T K^T          R = beta V^T - bfx X        (N = 64 tokens)
//   U = R T^T            U' = U fu
//   S^T = e^{gam_C} S^T + U' K                       (N = head_k)
//   O^T = fq (S^T Q^T) + U P^T
//
// Operands that are not bf16 inputs (S, R, U, T, P) enter as hi + lo, two
// bf16 terms: 2 MMAs against an input, 3 against another pair (lo x lo is
// below f32's own rounding of these sums).  The state itself stays f32 in
// registers, a quarter row per thread.
//
// Roles: warps 0-15 the chain above (a row's columns in quarters), warp 16
// issues its MMAs, warp 17 the copies (T, P and the factors come ready from
// m3_delta_tc_prep_kernel; two stages), so that a full queue stops nobody
// else.  The columns of U'^T K that a thread reads are those its part of S
// goes back to, so the chain needs no barrier among its warps.  A chunk is a
// chain of four dependent products, bound by their latency and the register
// work between them: 2.85 us (32 chunks of 8 x 2048 x 12 heads, 96 blocks: 98
// us).  With checkpoints and every SM at work (4 x 4096 x 40 heads: 257 us, 6.4
// TB/s of reads and writes) HBM is the bound.
__global__ void __launch_bounds__(THREADS, 1)
m3_delta_tc_fwd_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ CUtensorMap mo) {
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Smem& s = *reinterpret_cast<Smem*>(base + SMALL);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // uniform for the compiler too
  const int seg = blockIdx.y;
  const TcWalk walk(a, seg);
  const uint32_t st0 = smem_u32(base);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.kq_full[i], 1);
      mbar_init(&s.v_full[i], 1);
    }
    for (uint64_t* r : {&s.mbx, &s.mbq, &s.mbu, &s.mbd, &s.mbo, &s.o_free}) mbar_init(r, 1);
    for (uint64_t* r : {&s.rdy_s, &s.rdy_q, &s.rdy_o, &s.rdy_r, &s.rdy_u, &s.rdy_v}) mbar_init(r, CHAIN / 32);
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(&s.tmem, 512);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = __shfl_sync(~0u, s.tmem, 0);
  TcWait wait;

  if (warp == CHAIN / 32 + 1) {
    if (elect_one()) {
      int n_kq = 0, n_v = 0;  // loads issued
      auto load_kq = [&](int n) {  // a step's copies, once the stage is free
        if (n >= walk.n || !wait.ok) return;
        ++n_kq;
        const TcStep t = walk.at(n);
        const int c = t.c, b = t.bh / a.Hv, hk = t.bh % a.Hv / a.share;
        const uint32_t st = st0 + (n & 1) * KQ;
        uint64_t* bar = &s.kq_full[n & 1];
        const unsigned char* prep = a.tp + ((size_t)t.bh * a.nc + c) * a.tp_stride;
        mbar_expect_tx(bar, KQ + (uint32_t)sizeof(TcPrep));
        bulk_load(st0 + TP + (n & 1) * TP_BYTES, prep, TP_BYTES, bar);
        bulk_load(smem_u32(&s.vec[n % 3]), prep + TP_BYTES, (uint32_t)sizeof(TcVec), bar);
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          tma_tile(st + blk * 2 * TILE, &mk, blk * 64, hk, c * TC, b, bar);
          tma_tile(st + blk * 2 * TILE + TILE, &mq, blk * 64, hk, c * TC, b, bar);
        }
      };
      auto load_v = [&](int n) {
        if (n >= walk.n || !wait.ok) return;
        ++n_v;
        const TcStep t = walk.at(n);
        mbar_expect_tx(&s.v_full[n & 1], 2 * TILE);
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
          tma_tile(st0 + VO + ((n & 1) * 2 + blk) * TILE, &mv, blk * 64, t.bh % a.Hv, t.c * TC, t.bh / a.Hv, &s.v_full[n & 1]);
      };
      auto store = [&](int n) {  // a step's outputs, which the chain warps left in OUT
        if (!wait.ok) return;
        const TcStep t = walk.at(n);
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
          if (blk * 64 < a.DV)
            tma_tile_store(&mo, st0 + OUT + blk * TILE, blk * 64, t.bh % a.Hv, t.c * TC, t.bh / a.Hv);
        bulk_commit();
        bulk_wait_read();
      };
      grid_dep_wait();  // what the kernels before this one leave is there
      for (int n = 0; n < 2; ++n) {
        load_kq(n);
        load_v(n);
      }
      for (int n = 0; n < walk.n; ++n) {
        // step n's last products are done: so is everything with its tiles
        wait(&s.mbo, n & 1);
        load_kq(n + 2);
        load_v(n + 2);
        wait(&s.rdy_o, n & 1);  // its outputs are in place
        store(n);
        mbar_arrive(&s.o_free);
      }
      bulk_wait_all();
      // after a wait ran out, copies still in flight land before the block's
      // shared memory is given up (bounded)
      if (!wait.ok) {
        for (int i = 1; i <= 2 && i <= n_kq; ++i) mbar_wait(&s.kq_full[(n_kq - i) & 1], (n_kq - i) >> 1 & 1);
        for (int i = 1; i <= 2 && i <= n_v; ++i) mbar_wait(&s.v_full[(n_v - i) & 1], (n_v - i) >> 1 & 1);
      }
    }
    __syncwarp();
  } else if (warp == CHAIN / 32) {
    if (elect_one()) {
      auto mma_state = [&](uint32_t d, uint32_t bt) {  // S (hi, lo) x [64 tokens][128]
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc_mma_ts(tm + d, tm + T_S + ks * 16 + p * 8, tc_desc(bt + (ks >> 2) * 2 * TILE + (ks & 3) * 32, 16, 1024),
                      tc_idesc(128, 64, false, false), p + ks > 0);
      };
      auto mma_tokens = [&](uint32_t d, uint32_t ta, uint32_t bhi, uint32_t blo) {  // (hi, lo) x (hi, lo), K = 64
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc_mma_ts(tm + d, tm + ta + (p == 1 ? 32 : 0) + ks * 8, tc_desc((p == 2 ? blo : bhi) + ks * 32, 16, 1024),
                      tc_idesc(128, 64, false, false), p + ks > 0);
      };
      for (int n = 0; n < walk.n; ++n) {
        const int i = n & 1;
        const uint32_t st = st0 + i * KQ, par = n & 1;
        const uint32_t tp = st0 + TP + i * TP_BYTES;  // T hi, T lo, P hi, P lo
        wait(&s.kq_full[i], (n >> 1) & 1);
        wait(&s.rdy_s, par);  // S is in tensor memory
        tmem_fence_after_sync();
        if (wait.ok) {
          mma_state(T_X, st);
          tc_commit(&s.mbx);
        }
        wait(&s.rdy_r, par);
        if (wait.ok) {
          tmem_fence_after_sync();
          mma_tokens(T_X, T_R, tp, tp + TILE);
          tc_commit(&s.mbu);
        }
        wait(&s.rdy_q, par);  // the last chunk's S^T Q^T is read
        if (wait.ok) {  // behind U: nothing waits for it before the outputs
          tmem_fence_after_sync();
          mma_state(T_Q, st + TILE);
          tc_commit(&s.mbq);
        }
        wait(&s.rdy_u, par);
        wait(&s.mbq, par);  // S is read: its columns may be overwritten
        if (wait.ok) {
          tmem_fence_after_sync();
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ts(tm + T_S, tm + T_R + p * 32 + ks * 8, tc_desc(st + ks * 2048, 2 * TILE, 1024),
                        tc_idesc(128, 128, false, true), p + ks > 0);
          tc_commit(&s.mbd);
        }
        wait(&s.rdy_v, par);
        if (wait.ok) {
          tmem_fence_after_sync();
          mma_tokens(T_O, T_U, tp + 2 * TILE, tp + 3 * TILE);
          tc_commit(&s.mbo);
        }
      }
    }
    __syncwarp();
  } else {
    const int qt = warp >> 2, row = (warp & 3) * 32 + lane;  // quarter; row: the state's head_v index
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const bool live = row < a.DV;
    // this row's element of token 16 qt + j in a [64 tokens][head_v] tile pair
    const uint32_t el = (row >> 6) * TILE + qt * 16 * 128 + (row & 7) * 2, eu = (row & 63) >> 3;
    auto at = [&](int j) { return el + j * 128 + ((eu ^ (j & 7)) << 4); };
    auto vec = [&](int n) -> const TcVec& { return s.vec[n % 3]; };
    float2 S[16];  // S^T[row][32 qt + k]
    if (qt == 0) s.bad[row] = TC;
    bar_sync(1, CHAIN);
    int bad = TC;  // this step's first token (in this quarter) from which the row's outputs are NaN

    auto ready = [&](uint64_t* bar) {  // this warp's tensor-memory accesses so far are done
      tmem_wait_st();
      tmem_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto get_state = [&](const TcStep& t) {  // the state a run starts from
      // the carried state, what the chaining of segments left (the first one's
      // too: the last one's may be written where the carried state is), or a
      // state handed over
      if (t.take && wait.ok) wait.ok = flag_wait(a.flags + t.bh);
      const bool own = t.c > 0 || a.segs > 1;
      const float* src = own ? a.seg_start + ((size_t)t.bh * a.segs + seg) * DMAX * DMAX
                             : a.s_in ? a.s_in + (size_t)t.bh * a.DK * a.DV : nullptr;
      const int ld = own ? DMAX : a.DV;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const int kk = qt * 32 + k;
        const float v = src && (own || (live && kk < a.DK)) ? __ldcg(src + (size_t)kk * ld + row) : 0.0f;
        (k & 1 ? S[k >> 1].y : S[k >> 1].x) = v;
      }
    };
    auto end_state = [&](const TcStep& t) {  // where a run leaves it
      float* dst = nullptr;
      bool own = true;
      if (t.give) {
        dst = a.seg_start + (size_t)t.bh * DMAX * DMAX;
      } else if (a.s_out && t.c == a.nc - 1) {
        dst = a.s_out + (size_t)t.bh * a.DK * a.DV;
        own = false;
      }
      if (dst) {
        const int ld = own ? DMAX : a.DV;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const int kk = qt * 32 + k;
          if (own || (live && kk < a.DK)) dst[(size_t)kk * ld + row] = k & 1 ? S[k >> 1].y : S[k >> 1].x;
        }
      }
      if (t.give) {
        __threadfence();
        bar_sync(1, CHAIN);
        if (tid == 0) flag_set(a.flags + t.bh);
      }
    };
    auto put_state = [&](const TcStep& t) {  // S as hi, lo into tensor memory (and the step's checkpoint)
      uint32_t hi[2][8], lo[8];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int k = 0; k < 8; ++k) split2(S[8 * p + k], hi[p][k], lo[k]);
        tc_st8(tl + T_S + qt * 32 + p * 16, hi[p]);
        tc_st8(tl + T_S + qt * 32 + p * 16 + 8, lo);
      }
      ready(&s.rdy_s);
      if (a.ckpt) {
        unsigned char* ck = reinterpret_cast<unsigned char*>(a.ckpt) + ((size_t)t.bh * a.nc + t.c) * TC_CKPT + row * 16;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<uint4*>(ck + (qt * 4 + p * 2 + u) * 2048) =
                make_uint4(hi[p][4 * u], hi[p][4 * u + 1], hi[p][4 * u + 2], hi[p][4 * u + 3]);
      }
    };
    // x (16 tokens of this row) as hi, lo at column ta (32 + 32 columns)
    auto put_tokens = [&](uint32_t ta, const float2 (&x)[8], unsigned char* ck) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) split2(x[k], hi[k], lo[k]);
      tc_st8(tl + ta + qt * 8, hi);
      tc_st8(tl + ta + 32 + qt * 8, lo);
      if (ck) {
        if (bad < 16) {  // to the gradients such a row's U is NaN from that token on
#pragma unroll
          for (int k = 0; k < 8; ++k) hi[k] |= (2 * k >= bad ? 0x7FFFu : 0u) | (2 * k + 1 >= bad ? 0x7FFF0000u : 0u);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          *reinterpret_cast<uint4*>(ck + (qt * 2 + u) * 2048 + row * 16) = make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]);
          *reinterpret_cast<uint4*>(ck + 16384 + (qt * 2 + u) * 2048 + row * 16) = make_uint4(lo[4 * u], lo[4 * u + 1], lo[4 * u + 2], lo[4 * u + 3]);
        }
      }
    };
    // O of step n: read from T_Q and T_O and rounded, and (later) written to
    // OUT
    __nv_bfloat162 ov[8];
    auto read_outputs = [&](int n) {
      float2 q[8], o[8];
      wait(&s.mbq, n & 1);
      wait(&s.mbo, n & 1);
      tmem_fence_after_sync();
      tc_ld16(tl + T_Q + qt * 16, q);
      tc_ld16(tl + T_O + qt * 16, o);
      const Vec16 fq{&vec(n).fq[qt * 16]};
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __ffma2_rn(fq[j], q[j], o[j]);
      if (bad < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (2 * j >= bad) o[j].x = __int_as_float(0x7FFFFFFF);
          if (2 * j + 1 >= bad) o[j].y = __int_as_float(0x7FFFFFFF);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ov[j] = __floats2bfloat162_rn(o[j].x, o[j].y);
    };
    auto write_outputs = [&](int n) {
      if (n > 0) wait(&s.o_free, (n - 1) & 1);
      const uint32_t ob = st0 + OUT;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(ob + at(2 * j)), "h"(__bfloat16_as_ushort(ov[j].x)) : "memory");
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(ob + at(2 * j + 1)), "h"(__bfloat16_as_ushort(ov[j].y)) : "memory");
      }
      fence_proxy_async();
    };

    TcStep t = walk.at(0);
    grid_dep_wait();  // the segments' states, too
    get_state(t);
    put_state(t);
    for (int n = 0; n < walk.n; ++n) {
      const int i = n & 1;
      const uint32_t vt = st0 + VO + i * 2 * TILE;
      const uint32_t par = n & 1;
      // R = beta V - bfx X
      wait(&s.kq_full[i], (n >> 1) & 1);
      wait(&s.v_full[i], (n >> 1) & 1);
      float2 x[8];
      {
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          uint16_t vr;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(vr) : "r"(vt + at(j)));
          v[j] = vr;
        }
        wait(&s.mbx, par);
        tmem_fence_after_sync();
        tc_ld16(tl + T_X + qt * 16, x);
        float2 chk = f2b(0.0f);
        const Vec16 be{&vec(n).beta[qt * 16]}, bx{&vec(n).bfx[qt * 16]};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 vv = make_float2(__uint_as_float(v[2 * j] << 16), __uint_as_float(v[2 * j + 1] << 16));
          const float2 m = __fmul2_rn(x[j], f2b(-1.0f));
          x[j] = __ffma2_rn(bx[j], m, __fmul2_rn(be[j], vv));
          chk = __ffma2_rn(x[j], f2b(0.0f), chk);  // 0 unless a value is not finite
        }
        // a value that is not finite must not reach earlier tokens through
        // the zeros of T: it is taken out, and every output from its token
        // on becomes NaN
        if (!(chk.x + chk.y == 0.0f)) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float& e = j & 1 ? x[j >> 1].y : x[j >> 1].x;
            if (!(fabsf(e) <= FINITE_MAX)) {
              e = 0.0f;
              atomicMin(&s.bad[row], qt * 16 + j);
            }
          }
        }
      }
      put_tokens(T_R, x, nullptr);
      ready(&s.rdy_r);
      if (n > 0) read_outputs(n - 1);  // while U is made
      ready(&s.rdy_q);
      const TcStep tn = walk.at(n + 1);  // (past the last step: not used)
      wait(&s.mbu, par);
      const int bad_t = s.bad[row];
      bad = bad_t - qt * 16;
      const bool nan_row = bad_t < TC;
      tmem_fence_after_sync();
      tc_ld16(tl + T_X + qt * 16, x);
      {
        const Vec16 fu{&vec(n).fu[qt * 16]};
        float2 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __fmul2_rn(x[j], fu[j]);
        put_tokens(T_R, y, nullptr);
      }
      const float2 ec = f2b(vec(n).ec);
      ready(&s.rdy_u);
      // while the update of S runs
      put_tokens(T_U, x, a.ckpt ? reinterpret_cast<unsigned char*>(a.ckpt) + ((size_t)t.bh * a.nc + t.c) * TC_CKPT + 32768 : nullptr);
      ready(&s.rdy_v);
      if (n > 0) {
        write_outputs(n - 1);
        ready(&s.rdy_o);
      }
      wait(&s.mbd, par);
      tmem_fence_after_sync();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        tc_ld16(tl + T_S + qt * 32 + q * 16, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) S[q * 8 + k] = __ffma2_rn(ec, S[q * 8 + k], x[k]);
      }
      if (nan_row) {
#pragma unroll
        for (int k = 0; k < 16; ++k) S[k] = f2b(__int_as_float(0x7FFFFFFF));
      }
      if (t.last) end_state(t);
      if (n + 1 < walk.n) {
        t = tn;
        if (t.first) {
          bar_sync(1, CHAIN);
          if (qt == 0) s.bad[row] = TC;
          bar_sync(1, CHAIN);
          get_state(t);
        }
        put_state(t);
      }
    }
    read_outputs(walk.n - 1);
    write_outputs(walk.n - 1);
    ready(&s.rdy_o);
  }
  if (!wait.ok) report_timeout(&g_delta_fwd_status, a.status);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0) tmem_dealloc(tm, 512);
}

bool delta_tile_map(CUtensorMap* map, const void* ptr, int D, int H, int64_t T, int64_t B, int64_t stride, bool f32) {
  typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t es = f32 ? 4 : 2;
  const cuuint64_t strides[3] = {(cuuint64_t)D * es, (cuuint64_t)stride * es, (cuuint64_t)T * stride * es};
  const cuuint32_t box[4] = {f32 ? 32u : 64u, 1, TC, 1}, one[4] = {1, 1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------------------
// time segments
// ---------------------------------------------------------------------------
namespace agg {

constexpr int THREADS = CHAIN + 64;
constexpr int KT_ = 2 * TILE;           // one chunk's K tiles; two stages
constexpr int TT_ = 2 * KT_;            // T hi, lo, two stages
constexpr int VT = TT_ + 4 * TILE;      // V, two stages
constexpr int SMALL = VT + 4 * TILE;
struct Smem {  // at SMALL
  TcVec vec[2];
  int bad[2][128];
  uint64_t full[2];
  uint64_t mbx[2], mbu[2], mbd[2], rdy_s[2], rdy_r[2], rdy_u[2];  // by chain; rdy: one arrival per chain warp
  uint32_t tmem;
};
constexpr size_t SMEM_BYTES = SMALL + sizeof(Smem) + 1024;
// tensor-memory columns of a chain (256 each)
constexpr uint32_t A_S = 0, A_X = 128, A_R = 192;

}  // namespace agg

// A segment's effect on the state, S_end = N + Phi^T S_start: the chain of
// m3_delta_tc_fwd_kernel without outputs, twice in one block, from a zero
// state (N) and from the identity with V = 0 (the rows of Phi).  The two use
// the same tiles and take turns: one's products run under the other's
// register work.  With checkpoints Phi is kept for the backward, transposed:
// it takes the adjoint of a segment's end to the adjoint of its start.  3.1 us
// per chunk for both (128 segments of 114 chunks: 350 us); with a block for each, 1 x 65536 x 16 heads took 1.20 ms instead of
// 0.96.
__global__ void __launch_bounds__(agg::THREADS, 1)
m3_delta_tc_agg_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv) {
  using namespace agg;
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  agg::Smem& s = *reinterpret_cast<agg::Smem*>(base + agg::SMALL);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // uniform for the compiler too
  const int bh = blockIdx.x, b = bh / a.Hv, h = bh % a.Hv, hk = h / a.share, seg = blockIdx.y;
  const int c_begin = seg * a.seg_chunks, N = min(a.nc, c_begin + a.seg_chunks) - c_begin;
  const uint32_t st0 = smem_u32(base);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      for (uint64_t* r : {&s.full[i], &s.mbx[i], &s.mbu[i], &s.mbd[i]}) mbar_init(r, 1);
      for (uint64_t* r : {&s.rdy_s[i], &s.rdy_r[i], &s.rdy_u[i]}) mbar_init(r, CHAIN / 32);
    }
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(&s.tmem, 512);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = __shfl_sync(~0u, s.tmem, 0);
  grid_dep_trigger();
  TcWait wait;

  if (warp == CHAIN / 32 + 1) {
    if (elect_one()) {
      int issued = 0;
      auto load = [&](int n) {
        if (n >= N || !wait.ok) return;
        ++issued;
        const int i = n & 1, c = c_begin + n;
        const unsigned char* prep = a.tp + ((size_t)bh * a.nc + c) * a.tp_stride;
        mbar_expect_tx(&s.full[i], 6 * TILE + (uint32_t)sizeof(TcVec));
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          tma_tile(st0 + i * KT_ + blk * TILE, &mk, blk * 64, hk, c * TC, b, &s.full[i]);
          tma_tile(st0 + VT + (i * 2 + blk) * TILE, &mv, blk * 64, h, c * TC, b, &s.full[i]);
        }
        bulk_load(st0 + TT_ + i * 2 * TILE, prep, 2 * TILE, &s.full[i]);
        bulk_load(smem_u32(&s.vec[i]), prep + sizeof(TcTP), (uint32_t)sizeof(TcVec), &s.full[i]);
      };
      load(0);
      load(1);
      for (int n = 0; n < N; ++n) {  // step n's last products are done: so is everything with its tiles
        wait(&s.mbd[0], n & 1);
        wait(&s.mbd[1], n & 1);
        load(n + 2);
      }
      if (!wait.ok)  // as in the other kernels: copies in flight land first
        for (int i = 1; i <= 2 && i <= issued; ++i) mbar_wait(&s.full[(issued - i) & 1], (issued - i) >> 1 & 1);
    }
    __syncwarp();
  } else if (warp == CHAIN / 32) {
    if (elect_one()) {
      for (int n = 0; n < N; ++n) {
        const int i = n & 1;
        const uint32_t par = n & 1, kt = st0 + i * KT_, tt = st0 + TT_ + i * 2 * TILE;
        wait(&s.full[i], (n >> 1) & 1);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          wait(&s.rdy_s[m], par);
          if (!wait.ok) continue;
          tmem_fence_after_sync();
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma_ts(tm + m * 256 + A_X, tm + m * 256 + A_S + ks * 16 + p * 8,
                        tc_desc(kt + (ks >> 2) * TILE + (ks & 3) * 32, 16, 1024), tc_idesc(128, 64, false, false), p + ks > 0);
          tc_commit(&s.mbx[m]);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          wait(&s.rdy_r[m], par);
          if (!wait.ok) continue;
          tmem_fence_after_sync();
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ts(tm + m * 256 + A_X, tm + m * 256 + A_R + (p == 1 ? 32 : 0) + ks * 8,
                        tc_desc(tt + (p == 2 ? TILE : 0) + ks * 32, 16, 1024), tc_idesc(128, 64, false, false), p + ks > 0);
          tc_commit(&s.mbu[m]);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          wait(&s.rdy_u[m], par);
          if (!wait.ok) continue;
          tmem_fence_after_sync();
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ts(tm + m * 256 + A_S, tm + m * 256 + A_R + p * 32 + ks * 8, tc_desc(kt + ks * 2048, TILE, 1024),
                        tc_idesc(128, 128, false, true), p + ks > 0);
          tc_commit(&s.mbd[m]);
        }
      }
    }
    __syncwarp();
  } else {
    const int qt = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t el = (row >> 6) * TILE + qt * 16 * 128 + (row & 7) * 2, eu = (row & 63) >> 3;
    float2 S[2][16];
    if (qt == 0) s.bad[0][row] = s.bad[1][row] = TC;
    bar_sync(1, CHAIN);
    auto ready = [&](uint64_t* bar) {
      tmem_wait_st();
      tmem_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto put_state = [&](int m) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) split2(S[m][8 * p + k], hi[k], lo[k]);
        tc_st8(tl + m * 256 + A_S + qt * 32 + p * 16, hi);
        tc_st8(tl + m * 256 + A_S + qt * 32 + p * 16 + 8, lo);
      }
      ready(&s.rdy_s[m]);
    };
    auto put_tokens = [&](int m, const float2 (&x)[8]) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) split2(x[k], hi[k], lo[k]);
      tc_st8(tl + m * 256 + A_R + qt * 8, hi);
      tc_st8(tl + m * 256 + A_R + 32 + qt * 8, lo);
    };
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        S[m][k] = make_float2(m && qt * 32 + 2 * k == row ? 1.0f : 0.0f, m && qt * 32 + 2 * k + 1 == row ? 1.0f : 0.0f);
      put_state(m);
    }
    for (int n = 0; n < N; ++n) {
      const int i = n & 1;
      const uint32_t par = n & 1, vt = st0 + VT + i * 2 * TILE;
      const TcVec& vec = s.vec[i];
      wait(&s.full[i], (n >> 1) & 1);
#pragma unroll
      for (int m = 0; m < 2; ++m) {  // R = beta V - bfx X (as in the forward kernel)
        float2 x[8];
        uint32_t v[16];
        if (m == 0) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint16_t vr;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(vr) : "r"(vt + el + j * 128 + ((eu ^ (j & 7)) << 4)));
            v[j] = vr;
          }
        }
        wait(&s.mbx[m], par);
        tmem_fence_after_sync();
        tc_ld16(tl + m * 256 + A_X + qt * 16, x);
        float2 chk = f2b(0.0f);
        const Vec16 be{&vec.beta[qt * 16]}, bx{&vec.bfx[qt * 16]};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 y = __fmul2_rn(__fmul2_rn(x[j], f2b(-1.0f)), bx[j]);
          x[j] = m ? y : __ffma2_rn(be[j], make_float2(__uint_as_float(v[2 * j] << 16), __uint_as_float(v[2 * j + 1] << 16)), y);
          chk = __ffma2_rn(x[j], f2b(0.0f), chk);
        }
        if (!(chk.x + chk.y == 0.0f)) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float& e = j & 1 ? x[j >> 1].y : x[j >> 1].x;
            if (!(fabsf(e) <= FINITE_MAX)) {
              e = 0.0f;
              atomicMin(&s.bad[m][row], qt * 16 + j);
            }
          }
        }
        put_tokens(m, x);
        ready(&s.rdy_r[m]);
      }
      const float2 ec = f2b(vec.ec);  // (the factors are free after the arrivals below)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float2 x[8];
        wait(&s.mbu[m], par);
        tmem_fence_after_sync();
        tc_ld16(tl + m * 256 + A_X + qt * 16, x);
        const Vec16 fu{&vec.fu[qt * 16]};
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul2_rn(x[j], fu[j]);
        put_tokens(m, x);
        ready(&s.rdy_u[m]);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const bool nan_row = s.bad[m][row] < TC;
        wait(&s.mbd[m], par);
        tmem_fence_after_sync();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float2 x[8];
          tc_ld16(tl + m * 256 + A_S + qt * 32 + q * 16, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) S[m][q * 8 + k] = __ffma2_rn(ec, S[m][q * 8 + k], x[k]);
        }
        if (nan_row) {
#pragma unroll
          for (int k = 0; k < 16; ++k) S[m][k] = f2b(__int_as_float(0x7FFFFFFF));
        }
        if (n + 1 < N) put_state(m);
      }
    }
    // N as [head_k][row], Phi by its rows (and by its columns for the backward)
    float* end = a.seg_end + ((size_t)bh * a.segs + seg) * DMAX * DMAX;
    float* phi = a.seg_phi + ((size_t)bh * a.segs + seg) * DMAX * DMAX + (size_t)row * DMAX + qt * 32;
#pragma unroll
    for (int k = 0; k < 32; ++k) end[(size_t)(qt * 32 + k) * DMAX + row] = k & 1 ? S[0][k >> 1].y : S[0][k >> 1].x;
#pragma unroll
    for (int k = 0; k < 16; k += 2) *reinterpret_cast<float4*>(phi + 2 * k) = make_float4(S[1][k].x, S[1][k].y, S[1][k + 1].x, S[1][k + 1].y);
    if (a.seg_keep) {
      float* keep = a.seg_keep + ((size_t)bh * a.segs + seg) * DMAX * DMAX;
#pragma unroll
      for (int k = 0; k < 32; ++k) keep[(size_t)(qt * 32 + k) * DMAX + row] = k & 1 ? S[1][k >> 1].y : S[1][k >> 1].x;
    }
  }
  if (!wait.ok) report_timeout(&g_delta_fwd_status, a.status);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0) tmem_dealloc(tm, 512);
}

// A segment's start state from the ones before: start[s+1] = N_s + Phi_s^T
// start[s], 16 columns of the state per block, f32.  rev: the adjoint's, from
// the last segment to the first.  The segments' Phi (64 KB each) do not depend
// on the states, so each arrives by one bulk copy while the one before is
// used.  A thread has four by four values over a quarter of the rows, so that
// shared memory is read twice per sixteen products: 16 heads of nine segments
// 25 us (38 with four values over all rows), latency and that way through
// shared memory; two blocks per SM, Phi by halves, were no faster.
constexpr int SEG_PHI = DMAX * DMAX * 4;
constexpr size_t SEG_SMEM = 2 * SEG_PHI + 4 * 16 * DMAX * 4;  // and the quarters' sums [4][16][128]
__global__ void __launch_bounds__(512) m3_delta_seg_kernel(const __grid_constant__ DeltaArgs a, const float* first, bool rev) {
  extern __shared__ __align__(128) unsigned char raw[];
  __shared__ __align__(16) float S[DMAX][16];
  __shared__ __align__(8) uint64_t full[2];
  const int tid = threadIdx.x, bh = blockIdx.x, k = tid & (DMAX - 1), vq = (tid >> 7) * 4, v = blockIdx.y * 16 + vq;
  const int lane = tid & 31, vg = (tid >> 5 & 3) * 4;
  float* part = reinterpret_cast<float*>(raw + 2 * SEG_PHI);
  auto where = [&](int n) { return ((size_t)bh * a.segs + (rev ? a.segs - 1 - n : n)) * DMAX * DMAX; };
  const float* phis = rev ? a.seg_keep : a.seg_phi;
  int n_phi = 0;  // loads issued
  auto load = [&](int n) {
    if (n + 1 >= a.segs) return;
    ++n_phi;
    mbar_expect_tx(&full[n & 1], SEG_PHI);
    bulk_load(smem_u32(raw) + (n & 1) * SEG_PHI, phis + where(n), SEG_PHI, &full[n & 1]);
  };
  grid_dep_trigger();
  grid_dep_wait();
  if (tid == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    mbar_init_fence();
    load(0);
    load(1);
  }
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (first && k < a.DK && v < a.DV) x = *reinterpret_cast<const float4*>(first + ((size_t)bh * a.DK + k) * a.DV + v);
  *reinterpret_cast<float4*>(&S[k][vq]) = x;
  *reinterpret_cast<float4*>(a.seg_start + where(0) + (size_t)k * DMAX + v) = x;
  TcWait wait;
  for (int n = 0; n + 1 < a.segs; ++n) {
    x = *reinterpret_cast<const float4*>(a.seg_end + where(n) + (size_t)k * DMAX + v);
    __syncthreads();  // S
    wait(&full[n & 1], (n >> 1) & 1);
    // a quarter of the rows per 128 threads, four by four values per thread
    const float* phi = reinterpret_cast<const float*>(raw + (n & 1) * SEG_PHI) + (tid >> 7) * 32 * DMAX + lane * 4;  // Phi[r][..]
    const float* sr = &S[(tid >> 7) * 32][vg];
    float2 acc[4][2] = {};
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
      const float4 y = *reinterpret_cast<const float4*>(sr + r * 16), f = *reinterpret_cast<const float4*>(phi + r * DMAX);
      const float yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][0] = __ffma2_rn(make_float2(f.x, f.y), f2b(yv[i]), acc[i][0]);
        acc[i][1] = __ffma2_rn(make_float2(f.z, f.w), f2b(yv[i]), acc[i][1]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(part + ((tid >> 7) * 16 + vg + i) * DMAX + lane * 4) =
          make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
    __syncthreads();  // the quarters; S and Phi are read
    if (tid == 0 && wait.ok) load(n + 2);
    auto sum = [&](int i) {
      const float* q = part + (vq + i) * DMAX + k;
      return (q[0] + q[16 * DMAX]) + (q[32 * DMAX] + q[48 * DMAX]);
    };
    x.x += sum(0); x.y += sum(1); x.z += sum(2); x.w += sum(3);
    *reinterpret_cast<float4*>(&S[k][vq]) = x;
    *reinterpret_cast<float4*>(a.seg_start + where(n + 1) + (size_t)k * DMAX + v) = x;
  }
  if (!wait.ok)  // as in the other kernels: copies in flight land first
    for (int i = 1; i <= 2 && i <= n_phi; ++i) mbar_wait(&full[(n_phi - i) & 1], (n_phi - i) >> 1 & 1);
  if (!wait.ok) report_timeout(&g_delta_fwd_status, a.status);
}

cudaError_t launch_delta_seg(const DeltaArgs& a, const float* first, bool rev, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(m3_delta_seg_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SEG_SMEM);
  if (e != cudaSuccess) return e;
  return launch_k(m3_delta_seg_kernel, dim3((unsigned)(a.B * a.Hv), DMAX / 16), 512, SEG_SMEM, st, true, a, first, rev);
}

cudaError_t launch_delta_tc_fwd(const DeltaArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mo;
  if (!delta_tile_map(&mq, a.q, a.DK, a.Hk, a.T, a.B, a.qs) || !delta_tile_map(&mk, a.k, a.DK, a.Hk, a.T, a.B, a.ks) ||
      !delta_tile_map(&mv, a.v, a.DV, a.Hv, a.T, a.B, a.vs) ||
      !delta_tile_map(&mo, a.o, a.DV, a.Hv, a.T, a.B, (int64_t)a.Hv * a.DV))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  const unsigned heads = (unsigned)(a.B * a.Hv);
  if (a.segs > 1) {
    e = cudaFuncSetAttribute(m3_delta_tc_agg_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)agg::SMEM_BYTES);
    if (e == cudaSuccess)
      // (the last segment's effect is wanted by the backward only)
      // (not launched ahead of the end of the kernel before: blocks that come up one by one as SMs get free run 4 % slower)
      e = launch_k(m3_delta_tc_agg_kernel, dim3(heads, (unsigned)(a.segs - (a.seg_keep ? 0 : 1))), agg::THREADS, agg::SMEM_BYTES, st, false, a, mk, mv);
    if (e == cudaSuccess) e = launch_delta_seg(a, a.s_in, false, st);
  }
  if (e == cudaSuccess) e = cudaFuncSetAttribute(m3_delta_tc_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e == cudaSuccess && a.stream) e = cudaMemsetAsync(a.flags, 0, (size_t)heads * 4, st);
  if (e == cudaSuccess) e = launch_delta_blocks(m3_delta_tc_fwd_kernel, a, THREADS, SMEM_BYTES, st, true, mq, mk, mv, mo);
  return e;
}

}  // namespace m3
