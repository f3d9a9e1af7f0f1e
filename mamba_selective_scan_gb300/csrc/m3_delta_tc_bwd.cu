// m3_delta_tc_bwd.cu -- the gated delta rule's backward on the tensor cores:
// the reverse pass over the chunks (the state's adjoint), and the gradients
// of every chunk from it.
#include <initializer_list>

#include "m3_delta_tc.cuh"

namespace m3 {

// nonzero once a kernel here gave up waiting
__device__ unsigned int g_delta_bwd_status;

cudaError_t take_delta_bwd_status(unsigned* out) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_delta_bwd_status, sizeof(v));
  if (e == cudaSuccess && v) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_delta_bwd_status, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}

// ---------------------------------------------------------------------------
// reverse pass
// ---------------------------------------------------------------------------
namespace rev {

constexpr int CHAIN = 512;
constexpr int THREADS = CHAIN + 64;
constexpr int KQ = 4 * TILE;      // one chunk's K/Q tiles; two stages
constexpr int PREP = 2 * KQ;      // TcPrep, two stages
constexpr int PREP_STAGE = 34 * 1024;
constexpr int VO = PREP + 2 * PREP_STAGE;  // dO, two stages of two tiles; a chunk's dV takes its dO's place
constexpr int SMALL = VO + 4 * TILE;

struct Smem {  // at SMALL
  uint64_t kq_full[2], v_full[2], mbx, mbz, mbu, mbd;
  uint64_t rdy_s, rdy_y, rdy_r, rdy_u;  // one arrival per chain warp
  uint32_t tmem;
};
constexpr size_t SMEM_BYTES = SMALL + sizeof(Smem) + 1024;

// tensor-memory columns
constexpr uint32_t T_S = 0;    // dS: per 16 columns k, 8 of hi and 8 of lo; also the 128 columns of its update
constexpr uint32_t T_X = 128;  // dS^T K^T, then dR
constexpr uint32_t T_Z = 192;  // dO^T P
constexpr uint32_t T_R = 256;  // dU as hi, lo (32 + 32), then -bfx dR
constexpr uint32_t T_Y = 320;  // fq dO as hi, lo

}  // namespace rev

// The forward's chain backwards, with dS^T [head_v][head_k] in its place (see
// m3_delta_tc_fwd_kernel for the layout, the two-term operands and the roles):
//
//   dU = fu (dS^T K^T) + dO^T P       dR = dU T          (N = 64 tokens)
//   dV = beta dR
//   dS^T = e^{gam_C} dS^T - (bfx dR) K + (fq dO^T) Q     (N = head_k)
//
// It leaves dS (at each chunk's end) and dR for the gradients' kernel, which
// has no order among chunks.  AGG: a segment's effect on the adjoint, from
// zero (the transition is the forward's, transposed).
//
// Bound like the forward by a chunk's dependent products, 4.3 us (24 chunks of
// 36 heads one after the other: 104 us), and with every SM at work by what it
// reads and writes (194 KB per chunk and head; 4 x 4096 x 40 heads: 336 us,
// 5.9 TB/s).
template <bool AGG>
__global__ void __launch_bounds__(rev::THREADS, 1)
m3_delta_tc_rev_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ CUtensorMap mq,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap md,
                       const __grid_constant__ CUtensorMap mv) {
  using namespace rev;
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Smem& s = *reinterpret_cast<Smem*>(base + SMALL);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // uniform for the compiler too
  // the walk's steps count chunks from the end: of the head, or of a segment
  // (segments from the last one)
  const int seg = a.stream ? 0 : a.segs - 1 - (int)blockIdx.y;
  const int c_seg = seg * a.seg_chunks, n_seg = min(a.nc, c_seg + a.seg_chunks) - c_seg;
  TcWalk walk(a, 0);
  if (!a.stream) walk.n = walk.len_a = n_seg;
  auto chunk = [&](const TcStep& t) { return a.stream ? a.nc - 1 - t.c : c_seg + n_seg - 1 - t.c; };
  const uint32_t st0 = smem_u32(base);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.kq_full[i], 1);
      mbar_init(&s.v_full[i], 1);
    }
    for (uint64_t* r : {&s.mbx, &s.mbz, &s.mbu, &s.mbd}) mbar_init(r, 1);
    for (uint64_t* r : {&s.rdy_s, &s.rdy_y, &s.rdy_r, &s.rdy_u}) mbar_init(r, CHAIN / 32);
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
      int n_kq = 0, n_v = 0;  // loads issued
      auto load_kq = [&](int n) {  // a step's copies, once the stage is free
        if (n >= walk.n || !wait.ok) return;
        ++n_kq;
        const TcStep t = walk.at(n);
        const int c = chunk(t), b = t.bh / a.Hv, hk = t.bh % a.Hv / a.share;
        const uint32_t st = st0 + (n & 1) * KQ;
        uint64_t* bar = &s.kq_full[n & 1];
        mbar_expect_tx(bar, KQ + (uint32_t)sizeof(TcPrep));
        bulk_load(st0 + PREP + (n & 1) * PREP_STAGE, a.tp + ((size_t)t.bh * a.nc + c) * a.tp_stride, (uint32_t)sizeof(TcPrep), bar);
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
          tma_tile(st0 + VO + ((n & 1) * 2 + blk) * TILE, &md, blk * 64, t.bh % a.Hv, chunk(t) * TC, t.bh / a.Hv, &s.v_full[n & 1]);
      };
      auto store = [&](int n) {  // a step's dV, which the chain warps left in place of its inputs
        if (AGG || !wait.ok) return;
        const TcStep t = walk.at(n);
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
          if (blk * 64 < a.DV)
            tma_tile_store(&mv, st0 + VO + ((n & 1) * 2 + blk) * TILE, blk * 64, t.bh % a.Hv, chunk(t) * TC, t.bh / a.Hv);
        bulk_commit();
        bulk_wait_read();
      };
      for (int n = 0; n < 2; ++n) {
        load_kq(n);
        load_v(n);
      }
      for (int n = 0; n <= walk.n; ++n) {
        // step n - 1 is done with its tiles, its results are in place
        wait(&s.rdy_s, n & 1);
        if (n == 0) continue;
        load_kq(n + 1);
        store(n - 1);
        load_v(n + 1);
      }
      if (!AGG) bulk_wait_all();
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
      for (int n = 0; n < walk.n; ++n) {
        const int i = n & 1;
        const uint32_t st = st0 + i * KQ, par = n & 1;
        const uint32_t tp = st0 + PREP + i * PREP_STAGE;  // T hi, T lo, P hi, P lo
        wait(&s.kq_full[i], (n >> 1) & 1);
        wait(&s.rdy_s, par);  // dS is in tensor memory, the last chunk is done with
        tmem_fence_after_sync();
        if (wait.ok) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma_ts(tm + T_X, tm + T_S + ks * 16 + p * 8, tc_desc(st + (ks >> 2) * 2 * TILE + (ks & 3) * 32, 16, 1024),
                        tc_idesc(128, 64, false, false), p + ks > 0);
          tc_commit(&s.mbx);
        }
        wait(&s.v_full[i], (n >> 1) & 1);
        if (wait.ok) {  // dO^T P: dO [64 tokens][head_v] as an M-major A, P [i][j] as an N-major B
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ss(tm + T_Z, tc_desc(st0 + VO + i * 2 * TILE + ks * 2048, TILE, 1024), tc_desc(tp + (2 + p) * TILE + ks * 2048, 16, 1024),
                        tc_idesc(128, 64, true, true), p + ks > 0);
          tc_commit(&s.mbz);
        }
        wait(&s.rdy_y, par);
        wait(&s.mbx, par);  // dS is read: its columns may be overwritten
        if (wait.ok) {  // the update's first half, which needs no dR
          tmem_fence_after_sync();
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ts(tm + T_S, tm + T_Y + p * 32 + ks * 8, tc_desc(st + TILE + ks * 2048, 2 * TILE, 1024),
                        tc_idesc(128, 128, false, true), p + ks > 0);
        }
        wait(&s.rdy_r, par);
        if (wait.ok) {
          tmem_fence_after_sync();
#pragma unroll
          for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ts(tm + T_X, tm + T_R + (p == 1 ? 32 : 0) + ks * 8, tc_desc(tp + (p == 2 ? TILE : 0) + ks * 2048, 16, 1024),
                        tc_idesc(128, 64, false, true), p + ks > 0);
          tc_commit(&s.mbu);
        }
        wait(&s.rdy_u, par);
        if (wait.ok) {
          tmem_fence_after_sync();
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc_mma_ts(tm + T_S, tm + T_R + p * 32 + ks * 8, tc_desc(st + ks * 2048, 2 * TILE, 1024),
                        tc_idesc(128, 128, false, true), true);
          tc_commit(&s.mbd);
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
    auto vec = [&](int n) -> const TcVec& { return reinterpret_cast<const TcPrep*>(base + PREP + (n & 1) * PREP_STAGE)->vec; };
    float2 S[16];  // dS^T[row][32 qt + k]

    auto ready = [&](uint64_t* bar) {  // this warp's tensor-memory accesses so far are done
      tmem_wait_st();
      tmem_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto get_state = [&](const TcStep& t) {  // the adjoint a run starts from
      if (AGG) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          S[k] = f2b(0.0f);
        return;
      }
      if (t.take && wait.ok) wait.ok = flag_wait(a.flags + t.bh);
      const bool own = chunk(t) < a.nc - 1 || a.segs > 1;  // (of the last segment too: see the forward)
      const float* src = own ? a.seg_start + ((size_t)t.bh * a.segs + seg) * DMAX * DMAX
                             : a.ds_out ? a.ds_out + (size_t)t.bh * a.DK * a.DV : nullptr;
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
      if (AGG) {
        dst = a.seg_end + ((size_t)t.bh * a.segs + seg) * DMAX * DMAX;
      } else if (t.give) {
        dst = a.seg_start + (size_t)t.bh * DMAX * DMAX;
      } else if (a.ds_in && chunk(t) == 0) {
        dst = a.ds_in + (size_t)t.bh * a.DK * a.DV;
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
    auto put_state = [&](const TcStep& t) {  // dS as hi, lo into tensor memory, and kept for the step's gradients
      uint32_t hi[2][8], lo[2][8];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int k = 0; k < 8; ++k) split2(S[8 * p + k], hi[p][k], lo[p][k]);
        tc_st8(tl + T_S + qt * 32 + p * 16, hi[p]);
        tc_st8(tl + T_S + qt * 32 + p * 16 + 8, lo[p]);
      }
      ready(&s.rdy_s);
      if (!AGG) {
        unsigned char* ck = a.bwd + ((size_t)t.bh * a.nc + chunk(t)) * TC_BWD + row * 16;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int o = (qt * 4 + p * 2 + u) * 2048;
            *reinterpret_cast<uint4*>(ck + o) = make_uint4(hi[p][4 * u], hi[p][4 * u + 1], hi[p][4 * u + 2], hi[p][4 * u + 3]);
            *reinterpret_cast<uint4*>(ck + 32768 + o) = make_uint4(lo[p][4 * u], lo[p][4 * u + 1], lo[p][4 * u + 2], lo[p][4 * u + 3]);
          }
      }
    };
    // x (16 tokens of this row) as hi, lo at column ta (32 + 32 columns; or
    // only into ck)
    auto put_tokens = [&](uint32_t ta, const float2 (&x)[8], unsigned char* ck) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) split2(x[k], hi[k], lo[k]);
      if (ta != ~0u) {
        tc_st8(tl + ta + qt * 8, hi);
        tc_st8(tl + ta + 32 + qt * 8, lo);
      }
      if (ck) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          *reinterpret_cast<uint4*>(ck + (qt * 2 + u) * 2048 + row * 16) = make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]);
          *reinterpret_cast<uint4*>(ck + 16384 + (qt * 2 + u) * 2048 + row * 16) = make_uint4(lo[4 * u], lo[4 * u + 1], lo[4 * u + 2], lo[4 * u + 3]);
        }
      }
    };

    TcStep t = walk.at(0);
    if (!AGG) grid_dep_wait();  // the segments' adjoints are there (the rest is the forward's, or the caller's)
    get_state(t);
    put_state(t);
    for (int n = 0; n < walk.n; ++n) {
      const int i = n & 1;
      const uint32_t vt = st0 + VO + i * 2 * TILE;
      const uint32_t par = n & 1;
      float2 x[8];
      wait(&s.kq_full[i], (n >> 1) & 1);
      wait(&s.v_full[i], (n >> 1) & 1);
      {  // fq dO
        const Reg16 fq{&vec(n).fq[qt * 16]};
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          uint16_t vr;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(vr) : "r"(vt + at(j)));
          v[j] = vr;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = __fmul2_rn(make_float2(__uint_as_float(v[2 * j] << 16), __uint_as_float(v[2 * j + 1] << 16)), fq[j]);
        put_tokens(T_Y, x, nullptr);
        ready(&s.rdy_y);
      }
      wait(&s.mbx, par);
      wait(&s.mbz, par);
      tmem_fence_after_sync();
      tc_ld16(tl + T_X + qt * 16, x);
      {
        const Reg16 fu{&vec(n).fu[qt * 16]};
        float2 z[8];
        tc_ld16(tl + T_Z + qt * 16, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __ffma2_rn(x[j], fu[j], z[j]);
      }
      put_tokens(T_R, x, nullptr);
      ready(&s.rdy_r);
      const TcStep tn = walk.at(n + 1);  // (past the last step: not used)
      wait(&s.mbu, par);
      tmem_fence_after_sync();
      tc_ld16(tl + T_X + qt * 16, x);
      {
        const Reg16 bx{&vec(n).bfx[qt * 16]};
        float2 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __fmul2_rn(__fmul2_rn(x[j], f2b(-1.0f)), bx[j]);
        put_tokens(T_R, y, nullptr);
      }
      const float2 ec = f2b(vec(n).ec);
      float2 be[8];
      {
        const Reg16 v{&vec(n).beta[qt * 16]};
#pragma unroll
        for (int j = 0; j < 8; ++j) be[j] = v[j];  // (the factors are free after this arrival)
      }
      ready(&s.rdy_u);
      if (!AGG) {  // dV in place of dO, and dR for the gradients, while the update of dS runs
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 o = __fmul2_rn(be[j], x[j]);
          const __nv_bfloat162 v = __floats2bfloat162_rn(o.x, o.y);
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(vt + at(2 * j)), "h"(__bfloat16_as_ushort(v.x)) : "memory");
          asm volatile("st.shared.b16 [%0], %1;" ::"r"(vt + at(2 * j + 1)), "h"(__bfloat16_as_ushort(v.y)) : "memory");
        }
        fence_proxy_async();
        put_tokens(~0u, x, a.bwd + ((size_t)t.bh * a.nc + chunk(t)) * TC_BWD + 65536);
      }
      wait(&s.mbd, par);
      tmem_fence_after_sync();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        tc_ld16(tl + T_S + qt * 32 + q * 16, x);
#pragma unroll
        for (int k = 0; k < 8; ++k) S[q * 8 + k] = __ffma2_rn(ec, S[q * 8 + k], x[k]);
      }
      if (t.last) end_state(t);
      if (n + 1 < walk.n) {
        t = tn;
        if (t.first) get_state(t);
        put_state(t);
      } else {
        ready(&s.rdy_s);  // the last dV is in place
      }
    }
  }
  if (!wait.ok) report_timeout(&g_delta_bwd_status, a.status);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0) tmem_dealloc(tm, 512);
}

cudaError_t launch_delta_tc_rev(const DeltaArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, md, mv;
  if (!delta_tile_map(&mq, a.q, a.DK, a.Hk, a.T, a.B, a.qs) || !delta_tile_map(&mk, a.k, a.DK, a.Hk, a.T, a.B, a.ks) ||
      !delta_tile_map(&md, a.d_o, a.DV, a.Hv, a.T, a.B, (int64_t)a.Hv * a.DV) ||
      !delta_tile_map(&mv, a.dv, a.DV, a.Hv, a.T, a.B, a.dvs))
    return cudaErrorInvalidValue;
  auto go = [&](auto agg, auto fin) {
    cudaError_t e = cudaSuccess;
    const unsigned heads = (unsigned)(a.B * a.Hv);
    if (a.segs > 1) {
      e = cudaFuncSetAttribute(agg, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)rev::SMEM_BYTES);
      if (e == cudaSuccess)
        e = launch_k(agg, dim3(heads, (unsigned)(a.segs - 1)), rev::THREADS, rev::SMEM_BYTES, st, false, a, mq, mk, md, mv);
      if (e == cudaSuccess) e = launch_delta_seg(a, a.ds_out, true, st);
    }
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fin, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)rev::SMEM_BYTES);
    if (e == cudaSuccess && a.stream) e = cudaMemsetAsync(a.flags, 0, (size_t)heads * 4, st);
    if (e == cudaSuccess) e = launch_delta_blocks(fin, a, rev::THREADS, rev::SMEM_BYTES, st, a.segs > 1, mq, mk, md, mv);
    return e;
  };
  return go(m3_delta_tc_rev_kernel<true>, m3_delta_tc_rev_kernel<false>);
}

// ---------------------------------------------------------------------------
// gradients of a chunk
// ---------------------------------------------------------------------------
namespace grad {

constexpr int EPI = 512;
constexpr int THREADS = EPI + 32;
// shared-memory offsets
constexpr int KQ = 0;            // K, Q, K, Q tiles as in a stage
constexpr int DO = 4 * TILE;     // dO, two tiles; the tile before each is read (and ignored) with it
constexpr int S0 = 6 * TILE;     // S^T
constexpr int U = S0 + 32768;    // U^T hi, lo
constexpr int DS = U + 32768;    // dS^T hi, lo; in the place of lo later P2 hi, lo and A2 hi, lo
constexpr int DR = DS + 65536;   // dR^T hi, lo
constexpr int SMALL = DR + 32768;
constexpr int P2 = DS + 32768, A2 = P2 + 2 * TILE;

struct Smem {  // at SMALL
  float gam[TC], lo[TC], nkp[TC], nkm[TC];  // gam + lo: the gates' sum; nk (1 + lo), nk (1 - lo)
  float beta[TC], eg[TC], nk[TC], nq[TC], bfx[TC], fu[TC], fq[TC], cq[TC], ck[TC], gd[TC], d[TC], z[TC];
  float ss[4][2 * TC];
  float row_p[4][TC], col_p[2][TC];  // sums of dP o P: per column quarter, per warp
  float col_a[4][TC], row_a[2][TC];  // sums of dA o A (row_a without beta)
  float dot[3][4][TC];               // Q.(dO S0^T), K.(dR S0^T), K.(U dS^T): per warp of 32 head_k
  float red[2][16];  // (by turns: the next item's may be written before this one's are summed)
  float ec;
  GateSum tot;
  uint64_t ds, dl, us, kq;           // arrived: dS hi; dS lo; U, dR, dO, S0; K, Q
  uint64_t mb1, mb2, mb3;            // done: K Q^T (and all before it); G, dP, Yo, Y, Z; the products with P2 and A2
  uint64_t rdy0, rdy1, rdya;   // see the issuing warp
  uint32_t tmem;
};
constexpr size_t SMEM_BYTES = SMALL + sizeof(Smem) + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of one block");

// tensor-memory columns
constexpr uint32_t T_YO = 0, T_Y = 64, T_Z = 128, T_DQ = 192, T_DK = 256, T_G = 320, T_DP = 384, T_KQ = 448;

}  // namespace grad

// One head's chunk; a block takes the value heads of a key head's chunk one
// after the other.
struct GradItem {
  uint32_t group;  // (there are fewer than 2^31)
  int b, hk, m, c, h;
  size_t at;  // batch row x value head x chunk
  __device__ __forceinline__ GradItem(const DeltaArgs& a, uint32_t g) { set(a, g); }
  __device__ __forceinline__ void set(const DeltaArgs& a, uint32_t g) {
    group = g;
    const int bk = (int)(g / (uint32_t)a.nc);
    c = (int)(g - (uint32_t)bk * a.nc);
    b = bk / a.Hk;
    hk = bk % a.Hk;
    m = 0;
    h = hk * a.share;
    at = ((size_t)b * a.Hv + h) * a.nc + c;
  }
  __device__ __forceinline__ void next(const DeltaArgs& a) {
    if (++m < a.share) {
      ++h;
      at += a.nc;
    } else {
      set(a, group + gridDim.x);
    }
  }
};

// The 16 values of every lane summed over the warp: lane l returns the sum of
// value l / 2.
__device__ __forceinline__ float reduce16(float (&v)[16], int lane) {
#pragma unroll
  for (int w = 8, o = 16; w >= 1; w >>= 1, o >>= 1)
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const bool up = (lane & o) != 0;
      const float send = up ? v[j] : v[j + w], keep = up ? v[j + w] : v[j];
      v[j] = keep + __shfl_xor_sync(~0u, send, o);
    }
  return v[0] + __shfl_xor_sync(~0u, v[0], 1);
}

// Persistent blocks, one (chunk, head) at a time, in any order.  With the
// chunk's start state S0, U, dR and the adjoint dS at its end (q and k
// normalised, D as in m3_delta.cuh):
//
//   G = dR U^T          dA = -G below the diagonal     dbeta_i = G_ii / beta_i
//   dP = dO U^T         P2 = scale dP o D on and below it
//   A2 = dA o beta D
//   dQ = scale e^gam (dO S0^T) + P2 K
//   dK = e^{gam_C - gam} (U dS^T) - beta e^gam (dR S0^T) + P2^T Q + (A2 + A2^T) K
//
// and the exponents' shares, whose suffix sums are dg.  The products with
// S0 and dS stand transposed (head_k in the lanes, tokens in the columns), so
// the tiles the other kernels wrote serve as M-major operands as they are and
// no half of an MMA is idle; only G^T and dP share their lanes' two halves.
// S0 enters with one bf16 term, everything else that is not an input with two:
// dq, dg and dbeta are those of a start state rounded to bf16.  In the 2-norm
// over 300 tokens that puts dq at 1.9e-3 and dg at 2.0e-3, where their own
// rounding to bf16 gives 1.7e-3 and 2.0e-3 (over one token 2.4e-3 and 3.3e-3
// against 1.8e-3 and 2.1e-3).  A second term is 32 KB more per item to keep,
// write and read, for which shared memory has no place.
//
// 210 KB come in and 32 KB go out per item, so the next item's tiles are
// fetched as soon as the first products have read this one's.  The sums over
// the heads of a key head stay in tensor memory.  4 x 4096 x 40 heads: 425 us,
// 12600 cycles an item, 5.4 TB/s.  Shared memory is the bound: the products'
// operands keep its data path busy 6000 cycles an item, the epilogues' reads,
// writes and shuffles 6700, besides what the copies write.
template <bool L2>
__global__ void __launch_bounds__(grad::THREADS, 1)
m3_delta_tc_grad_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ CUtensorMap mq,
                        const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap md) {
  using namespace grad;
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Smem& s = *reinterpret_cast<Smem*>(base + SMALL);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(~0u, tid >> 5, 0);  // uniform for the compiler too
  const uint32_t groups = (uint32_t)a.B * a.Hk * a.nc;  // (batch row, key head, chunk), `share` items each
  const uint32_t sb = smem_u32(base);

  if (tid == 0) {
    for (uint64_t* r : {&s.ds, &s.dl, &s.us, &s.kq, &s.mb1, &s.mb2, &s.mb3}) mbar_init(r, 1);
    for (uint64_t* r : {&s.rdy0, &s.rdy1, &s.rdya}) mbar_init(r, EPI / 32);
    mbar_init_fence();
  }
  if (warp == 0) tmem_alloc(&s.tmem, 512);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tm = __shfl_sync(~0u, s.tmem, 0);
  TcWait wait;

  if (warp == EPI / 32) {
    if (elect_one()) {
      uint32_t n_ds = 0, n_dl = 0, n_us = 0, n_kq = 0;  // loads issued
      auto load_ds = [&](const GradItem& it) {
        ++n_ds;
        mbar_expect_tx(&s.ds, 32768);
        bulk_load(sb + DS, a.bwd + it.at * TC_BWD, 32768, &s.ds);
      };
      auto load_dl = [&](const GradItem& it) {
        ++n_dl;
        mbar_expect_tx(&s.dl, 32768);
        bulk_load(sb + DS + 32768, a.bwd + it.at * TC_BWD + 32768, 32768, &s.dl);
      };
      auto load_us = [&](const GradItem& it) {
        ++n_us;
        mbar_expect_tx(&s.us, 3 * 32768 + 2 * TILE);
        bulk_load(sb + S0, reinterpret_cast<const unsigned char*>(a.ckpt_in) + it.at * TC_CKPT, 65536, &s.us);  // and U
        bulk_load(sb + DR, a.bwd + it.at * TC_BWD + 65536, 32768, &s.us);
        for (int blk = 0; blk < 2; ++blk) tma_tile(sb + DO + blk * TILE, &md, blk * 64, it.h, it.c * TC, it.b, &s.us);
      };
      auto load_kq = [&](const GradItem& it) {
        ++n_kq;
        mbar_expect_tx(&s.kq, 4 * TILE);
        for (int blk = 0; blk < 2; ++blk) {
          tma_tile(sb + KQ + blk * 2 * TILE, &mk, blk * 64, it.hk, it.c * TC, it.b, &s.kq);
          tma_tile(sb + KQ + blk * 2 * TILE + TILE, &mq, blk * 64, it.hk, it.c * TC, it.b, &s.kq);
        }
      };
      // a product of `steps` steps of 16 in K; operand descriptors by step
      auto mma = [&](uint32_t d, int steps, uint32_t idesc, bool first, auto da, auto db) {
#pragma unroll
        for (int ks = 0; ks < steps; ++ks) tc_mma_ss(tm + d, da(ks), db(ks), idesc, !(first && ks == 0));
      };
      auto kept = [&](int at) { return [=](int ks) { return tc_desc_plain(sb + at + ks * 256); }; };
      auto mn = [&](int at, int lbo) { return [=](int ks) { return tc_desc(sb + at + ks * 2048, lbo, 1024); }; };
      auto kmaj = [&](int at, int blk) { return [=](int ks) { return tc_desc(sb + at + (ks >> 2) * blk + (ks & 3) * 32, 16, 1024); }; };
      constexpr uint32_t NN = tc_idesc(128, 64, false, false), NM = tc_idesc(128, 64, false, true),
                         MN = tc_idesc(128, 64, true, false), MM = tc_idesc(128, 64, true, true);
      GradItem it(a, blockIdx.x);
      grid_dep_wait();  // the reverse pass is done
      load_us(it);
      load_ds(it);
      load_dl(it);
      load_kq(it);
      uint32_t pkq = 0;
      for (uint32_t n = 0; it.group < groups; ++n) {
        const uint32_t par = n & 1;
        const int m = it.m;
        // while the last item's outputs are still being written
        wait(&s.us, par);
        wait(&s.ds, par);
        if (n > 0) wait(&s.rdya, par ^ 1);  // its G, dP, Yo, Y, Z, K and Q are read
        if (wait.ok) {
          tmem_fence_after_sync();
          mma(T_G, 8, MM, true, kept(U), kept(DR));
          mma(T_G, 8, MM, false, kept(U + 16384), kept(DR));
          mma(T_G, 8, MM, false, kept(U), kept(DR + 16384));
          mma(T_DP, 8, NM, true, kmaj(DO - TILE, TILE), kept(U));
          mma(T_DP, 8, NM, false, kmaj(DO - TILE, TILE), kept(U + 16384));
          mma(T_Z, 8, MM, true, kept(DS), kept(U));
          mma(T_Z, 8, MM, false, kept(DS), kept(U + 16384));
          mma(T_YO, 8, MN, true, kept(S0), kmaj(DO, TILE));
          mma(T_Y, 8, MM, true, kept(S0), kept(DR));
          mma(T_Y, 8, MM, false, kept(S0), kept(DR + 16384));
        }
        wait(&s.dl, par);
        if (wait.ok) {
          mma(T_Z, 8, MM, false, kept(DS + 32768), kept(U));
          tc_commit(&s.mb2);
        }
        if (m == 0) {
          wait(&s.kq, pkq);
          pkq ^= 1;
          if (wait.ok) {
            tmem_fence_after_sync();
            mma(T_KQ, 8, NN, true, kmaj(KQ, 2 * TILE), kmaj(KQ, 2 * TILE));
          }
        }
        if (wait.ok) tc_commit(&s.mb1);
        it.next(a);
        const bool more = it.group < groups;
        // the next item's tiles as soon as this one's have been read
        wait(&s.mb2, par);
        wait(&s.rdy0, par);  // the inner product has read S0 and dS
        if (more && wait.ok) {
          load_us(it);
          load_ds(it);
        }
        wait(&s.rdy1, par);  // P2 and A2 are in place
        if (wait.ok) {
          tmem_fence_after_sync();
          for (int p = 0; p < 2; ++p) {
            mma(T_DQ, 4, MN, p + m == 0, mn(KQ, 2 * TILE), kmaj(P2 + p * TILE, 0));
            mma(T_DK, 4, MM, p + m == 0, mn(KQ + TILE, 2 * TILE), mn(P2 + p * TILE, 16));
            mma(T_DK, 4, MN, false, mn(KQ, 2 * TILE), kmaj(A2 + p * TILE, 0));
            mma(T_DK, 4, MM, false, mn(KQ, 2 * TILE), mn(A2 + p * TILE, 16));
          }
          tc_commit(&s.mb3);
        }
        wait(&s.mb3, par);
        if (more && wait.ok) load_dl(it);
        if (more && it.m == 0) {  // (else K and Q are the next item's too)
          wait(&s.rdya, par);     // and read
          if (wait.ok) load_kq(it);
        }
      }
      if (!wait.ok) {  // as in the other kernels: copies in flight land first
        if (n_ds) mbar_wait(&s.ds, (n_ds - 1) & 1);
        if (n_dl) mbar_wait(&s.dl, (n_dl - 1) & 1);
        if (n_us) mbar_wait(&s.us, (n_us - 1) & 1);
        if (n_kq) mbar_wait(&s.kq, (n_kq - 1) & 1);
      }
    }
    __syncwarp();
  } else {
    const int qt = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
    const uint32_t tl = tm + ((uint32_t)(wq * 32) << 16) + qt * 16;
    auto ready = [&](uint64_t* bar) {
      tmem_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // elements `row` (a head_k index) of tokens 2 j and 2 j + 1 of this
    // quarter, K (0) or Q (1), as their bf16 pair
    const uint32_t el = sb + KQ + (row >> 6) * 2 * TILE + (row & 7) * 2;
    auto tok = [&](int q, int j) {
      uint16_t v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v[e]) : "r"(el + q * TILE + sw(qt * 16 + 2 * j + e, (row & 63) >> 3)));
      return (uint32_t)v[0] | (uint32_t)v[1] << 16;
    };
    auto wide = [](uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u)); };
    uint32_t par = 0, pkq = 0;
    for (GradItem it(a, blockIdx.x); it.group < groups; it.next(a), par ^= 1) {
      const int c = it.c, b = it.b, h = it.h;
      const int64_t tok0 = (int64_t)b * a.T + c * TC;  // the chunk's first token
      const int n = min(TC, a.T - c * TC);
      GateSum g = {0.0f, 0.0f};  // (in powers of two)
      float beta = 0.0f;
      if (tid < n) {
        g.h = LOG2E * clamp_g(__bfloat162float(static_cast<const __nv_bfloat16*>(a.g)[(tok0 + tid) * a.Hv + h]));
        beta = __bfloat162float(static_cast<const __nv_bfloat16*>(a.beta)[(tok0 + tid) * a.Hv + h]);
      }
      // <dS, S0>
      wait(&s.us, par);
      wait(&s.ds, par);
      wait(&s.dl, par);
      {
        float acc = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int at = (tid + u * EPI) * 16;
          const uint4 x = *reinterpret_cast<const uint4*>(base + S0 + at), y = *reinterpret_cast<const uint4*>(base + DS + at),
                      z = *reinterpret_cast<const uint4*>(base + DS + 32768 + at);
          const uint32_t xv[4] = {x.x, x.y, x.z, x.w}, yv[4] = {y.x, y.y, y.z, y.w}, zv[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc = fmaf(__uint_as_float(xv[j] << 16), __uint_as_float(yv[j] << 16) + __uint_as_float(zv[j] << 16), acc);
            acc = fmaf(__uint_as_float(xv[j] & 0xFFFF0000u),
                       __uint_as_float(yv[j] & 0xFFFF0000u) + __uint_as_float(zv[j] & 0xFFFF0000u), acc);
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(~0u, acc, o);
        if (lane == 0) s.red[par][warp] = acc;
      }
      ready(&s.rdy0);
      if (it.m == 0) {
        wait(&s.kq, pkq);
        pkq ^= 1;
      }
      if (L2 && it.m == 0) {  // (the heads of a key head share its norms)
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint4 x;
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                       : "r"(sb + KQ + (qt >> 1) * (2 * TILE) + sw(row, (qt & 1) * 4 + u)));
          const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float(q[j] << 16), hi = __uint_as_float(q[j] & 0xFFFF0000u);
            s0 = fmaf(lo, lo, s0);
            s1 = fmaf(hi, hi, s1);
          }
        }
        s.ss[qt][row] = s0 + s1;
      }
      if (warp < 2) {
        g = gate_scan(g, lane);
        if (tid == 31) s.tot = g;
      }
      bar_sync(1, EPI);
      if (warp < 2) {
        if (warp == 1) g = gate_add(s.tot, g);
        g.l *= LN2;  // (in powers of e from here on)
        s.gam[tid] = g.h;
        s.lo[tid] = g.l;
        s.beta[tid] = beta;
        float nk = 1.0f, nq = 1.0f;
        if (L2) {
          nk = it.m ? s.nk[tid] : rsqrtf((s.ss[0][tid] + s.ss[1][tid]) + (s.ss[2][tid] + s.ss[3][tid]) + DELTA_L2_EPS);
          nq = it.m ? s.nq[tid]
                    : rsqrtf((s.ss[0][TC + tid] + s.ss[1][TC + tid]) + (s.ss[2][TC + tid] + s.ss[3][TC + tid]) + DELTA_L2_EPS);
        }
        const float eg = ex2(g.h) * (1.0f + g.l);
        s.eg[tid] = eg;
        s.nk[tid] = nk;
        s.nkp[tid] = nk * (1.0f + g.l);
        s.nkm[tid] = nk * (1.0f - g.l);
        s.nq[tid] = nq;
        s.bfx[tid] = beta * eg * nk;
        s.fq[tid] = a.scale * eg * nq;
      }
      bar_sync(1, EPI);
      if (warp < 2) {
        s.fu[tid] = ex2(s.gam[TC - 1] - g.h) * (1.0f + (s.lo[TC - 1] - g.l)) * s.nk[tid];
        if (tid == 0) s.ec = ex2(s.gam[TC - 1]) * (1.0f + s.lo[TC - 1]);
      }
      wait(&s.mb1, par);
      tmem_fence_after_sync();
      {
        const int r = row & (TC - 1), c0 = qt * 16;
        const float2 gr = f2b(s.gam[r]);
        const Reg16 gc{&s.gam[c0]}, nc{wq < 2 ? &s.nkp[c0] : &s.nkm[c0]}, bc{&s.beta[c0]};
        float2 v[8], k[8];
        float sum[16];
        unsigned char* tile = base + grad::P2;
        if (wq < 2) {  // G^T: row j = r, columns i
          tc_ld16(tl + T_G, v);
          tc_ld16(tl + T_KQ, k);
          if (r >> 4 == qt) {
#pragma unroll
            for (int m = 0; m < 16; ++m)
              if (c0 + m == r) s.gd[r] = m & 1 ? v[m >> 1].y : v[m >> 1].x;
          }
          const float2 f = f2b(-s.nkm[r]);
          float2 col = f2b(0.0f);
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float2 e = ex2x2(__ffma2_rn(gr, f2b(-1.0f), gc[m]));
            float2 x = __fmul2_rn(__fmul2_rn(__fmul2_rn(nc[m], f), e), v[m]);  // dA o D
            x.x = c0 + 2 * m > r ? x.x : 0.0f;
            x.y = c0 + 2 * m + 1 > r ? x.y : 0.0f;
            v[m] = __fmul2_rn(x, bc[m]);
            k[m] = __fmul2_rn(k[m], x);
            col = __ffma2_rn(k[m], bc[m], col);
            sum[2 * m] = k[m].x;
            sum[2 * m + 1] = k[m].y;
          }
          s.col_a[qt][r] = col.x + col.y;
          const float t = reduce16(sum, lane);
          if (!(lane & 1)) s.row_a[wq][c0 + (lane >> 1)] = t;
          tile += 2 * TILE;
        } else {  // dP: row i = r, columns j
          tc_ld16(tl + T_DP, v);
          tc_ld16(tl + T_KQ, k);
          const float2 f = f2b(a.scale * s.nq[r] * (1.0f + s.lo[r]));
          float2 rs = f2b(0.0f);
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float2 e = ex2x2(__ffma2_rn(gc[m], f2b(-1.0f), gr));
            float2 x = __fmul2_rn(__fmul2_rn(__fmul2_rn(nc[m], f), e), v[m]);
            x.x = c0 + 2 * m <= r ? x.x : 0.0f;
            x.y = c0 + 2 * m + 1 <= r ? x.y : 0.0f;
            v[m] = x;
            k[m] = __fmul2_rn(k[m], x);
            rs = __fadd2_rn(rs, k[m]);
            sum[2 * m] = k[m].x;
            sum[2 * m + 1] = k[m].y;
          }
          s.row_p[qt][r] = rs.x + rs.y;
          const float t = reduce16(sum, lane);
          if (!(lane & 1)) s.col_p[wq - 2][c0 + (lane >> 1)] = t;
        }
        wait(&s.mb2, par);  // dS is read (so has the inner product, two barriers ago)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint4 hi, lo;
          split2(v[4 * u], hi.x, lo.x);
          split2(v[4 * u + 1], hi.y, lo.y);
          split2(v[4 * u + 2], hi.z, lo.z);
          split2(v[4 * u + 3], hi.w, lo.w);
          const uint32_t at = sw(r, qt * 2 + u);
          *reinterpret_cast<uint4*>(tile + at) = hi;
          *reinterpret_cast<uint4*>(tile + TILE + at) = lo;
        }
      }
      fence_proxy_async();
      ready(&s.rdy1);
      // the products with the states, and their rows' dots with Q and K
      wait(&s.mb2, par);
      tmem_fence_after_sync();
      float2 dq[8], dk[8];
      uint32_t qv[8], kv[8];  // (kept: shared memory is busy with the next item's products when they are wanted again)
      {
        float y[16];
        float2 x[8];
        tc_ld16(tl + T_YO, dq);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          qv[j] = tok(1, j);
          const float2 p = __fmul2_rn(dq[j], wide(qv[j]));
          y[2 * j] = p.x;
          y[2 * j + 1] = p.y;
        }
        float t = reduce16(y, lane);
        if (!(lane & 1)) s.dot[0][wq][qt * 16 + (lane >> 1)] = t;
        tc_ld16(tl + T_Y, dk);
        tc_ld16(tl + T_Z, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) kv[j] = tok(0, j);
        ready(&s.rdya);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 p = __fmul2_rn(dk[j], wide(kv[j]));
          y[2 * j] = p.x;
          y[2 * j + 1] = p.y;
        }
        t = reduce16(y, lane);
        if (!(lane & 1)) s.dot[1][wq][qt * 16 + (lane >> 1)] = t;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 p = __fmul2_rn(x[j], wide(kv[j]));
          y[2 * j] = p.x;
          y[2 * j + 1] = p.y;
        }
        t = reduce16(y, lane);
        if (!(lane & 1)) s.dot[2][wq][qt * 16 + (lane >> 1)] = t;
        bar_sync(1, EPI);
        const Reg16 fq{&s.fq[qt * 16]}, fu{&s.fu[qt * 16]}, bx{&s.bfx[qt * 16]};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dq[j] = __fmul2_rn(dq[j], fq[j]);
          dk[j] = __ffma2_rn(fu[j], x[j], __fmul2_rn(__fmul2_rn(dk[j], f2b(-1.0f)), bx[j]));
        }
      }
      if (warp < 2) {  // per-token sums: dbeta, the normalisations' parts, the exponent's share
        const int i = tid;
        float dot[3];
#pragma unroll
        for (int m = 0; m < 3; ++m) dot[m] = (s.dot[m][0][i] + s.dot[m][1][i]) + (s.dot[m][2][i] + s.dot[m][3][i]);
        const float rp = (s.row_p[0][i] + s.row_p[1][i]) + (s.row_p[2][i] + s.row_p[3][i]), cp = s.col_p[0][i] + s.col_p[1][i];
        const float ca = (s.col_a[0][i] + s.col_a[1][i]) + (s.col_a[2][i] + s.col_a[3][i]), rah = s.row_a[0][i] + s.row_a[1][i];
        const float be = s.beta[i], ra = be * rah;
        const float yo = s.fq[i] * dot[0], y = s.bfx[i] * dot[1], z = s.fu[i] * dot[2];
        s.cq[i] = L2 ? -s.nq[i] * s.nq[i] * (yo + rp) : 0.0f;
        s.ck[i] = L2 ? -s.nk[i] * s.nk[i] * (z - y + cp + ra + ca) : 0.0f;
        s.d[i] = (rp - cp) + (ra - ca) + yo - y - z;
        s.z[i] = z;
        if (i < n) {
          float db = s.gd[i] / be;
          if (!(fabsf(be) > 1e-20f)) {
            // U holds nothing of a token that writes nothing: from
            // dR.(v - e^gam S0^T k) - (below the diagonal of D K K^T) G
            const unsigned char* dr = a.bwd + it.at * TC_BWD + 65536;
            const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v) + (tok0 + i) * a.vs + (int64_t)h * a.DV;
            float rv = 0.0f;
            for (int m = 0; m < a.DV; ++m) {
              const uint32_t at = (i >> 3) * 2048 + m * 16 + (i & 7) * 2;
              const float x = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(dr + at)) +
                              __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(dr + 16384 + at));
              rv = fmaf(x, __bfloat162float(vp[m]), rv);
            }
            db = rv - s.eg[i] * s.nk[i] * dot[1] + rah;
          }
          static_cast<__nv_bfloat16*>(a.dbeta)[(tok0 + i) * a.Hv + h] = __float2bfloat16_rn(db);
        }
      }
      bar_sync(1, EPI);
      if (warp == EPI / 32 - 1) {  // dg: suffix sums, tokens lane and lane + 32
        float d[2] = {s.d[lane], s.d[lane + 32]}, w = s.z[lane] + s.z[lane + 32], in = lane < 16 ? s.red[par][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          w += __shfl_xor_sync(~0u, w, o);
          in += __shfl_xor_sync(~0u, in, o);
        }
        if (lane == 31) d[1] += fmaf(s.ec, in, w);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x = __shfl_down_sync(~0u, d[0], o), y = __shfl_down_sync(~0u, d[1], o);
          if (lane + o < 32) {
            d[0] += x;
            d[1] += y;
          }
        }
        d[0] += __shfl_sync(~0u, d[1], 0);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (lane + 32 * e < n)
            static_cast<__nv_bfloat16*>(a.dg)[(tok0 + lane + 32 * e) * a.Hv + h] = __float2bfloat16_rn(d[e]);
      }
      wait(&s.mb3, par);
      tmem_fence_after_sync();
      {
        float2 x[8];
        tc_ld16(tl + T_DQ, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) dq[j] = __fadd2_rn(dq[j], x[j]);
        tc_ld16(tl + T_DK, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) dk[j] = __fadd2_rn(dk[j], x[j]);
        if (L2) {
          const Reg16 cq{&s.cq[qt * 16]}, ck{&s.ck[qt * 16]};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dq[j] = __ffma2_rn(cq[j], wide(qv[j]), dq[j]);  // (cq, ck are negative)
            dk[j] = __ffma2_rn(ck[j], wide(kv[j]), dk[j]);
          }
        }
      }
      // value heads that share a key head: their sum so far goes back to where
      // the next one's products with P2 and A2 are added to it
      if (it.m + 1 < a.share) {
        auto put = [&](uint32_t at, const float2 (&v)[8]) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint32_t x[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              x[2 * j] = __float_as_uint(v[4 * p + j].x);
              x[2 * j + 1] = __float_as_uint(v[4 * p + j].y);
            }
            tc_st8(tl + at + p * 8, x);
          }
        };
        put(T_DQ, dq);
        put(T_DK, dk);
        tmem_wait_st();  // (behind this thread's next arrival at rdy1)
        continue;
      }
      tmem_fence_before_sync();
      // out, two neighbours of a token at a time: an even lane takes the even
      // tokens of its pair of rows, the odd lane the odd ones
      const int row2 = row & ~1, odd = row & 1;
      const bool in = row2 < a.DK;  // (head_k is even)
      __nv_bfloat16* qp = static_cast<__nv_bfloat16*>(a.dq) + (tok0 + qt * 16 + odd) * a.dqs + (int64_t)it.hk * a.DK + row2;
      __nv_bfloat16* kp = static_cast<__nv_bfloat16*>(a.dk) + (tok0 + qt * 16 + odd) * a.dks + (int64_t)it.hk * a.DK + row2;
      const int left = n - qt * 16 - odd;
#pragma unroll
      for (int j = 0; j < 8; ++j, qp += 2 * a.dqs, kp += 2 * a.dks) {
        const float oq = __shfl_xor_sync(~0u, odd ? dq[j].x : dq[j].y, 1), ok = __shfl_xor_sync(~0u, odd ? dk[j].x : dk[j].y, 1);
        const __nv_bfloat162 q2 = odd ? __floats2bfloat162_rn(oq, dq[j].y) : __floats2bfloat162_rn(dq[j].x, oq);
        const __nv_bfloat162 k2 = odd ? __floats2bfloat162_rn(ok, dk[j].y) : __floats2bfloat162_rn(dk[j].x, ok);
        if (in && 2 * j < left) {
          *reinterpret_cast<__nv_bfloat162*>(qp) = q2;
          *reinterpret_cast<__nv_bfloat162*>(kp) = k2;
        }
      }
    }
  }
  if (!wait.ok) report_timeout(&g_delta_bwd_status, a.status);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  if (warp == 0) tmem_dealloc(tm, 512);
}

cudaError_t launch_delta_tc_grad(const DeltaArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, md;
  if (!delta_tile_map(&mq, a.q, a.DK, a.Hk, a.T, a.B, a.qs) || !delta_tile_map(&mk, a.k, a.DK, a.Hk, a.T, a.B, a.ks) ||
      !delta_tile_map(&md, a.d_o, a.DV, a.Hv, a.T, a.B, (int64_t)a.Hv * a.DV))
    return cudaErrorInvalidValue;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  auto kern = a.l2 ? m3_delta_tc_grad_kernel<true> : m3_delta_tc_grad_kernel<false>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)grad::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t groups = (int64_t)a.B * a.Hk * a.nc;
  if (sms > TC_BLOCKS) sms = TC_BLOCKS;
  return launch_k(kern, dim3((unsigned)(groups < sms ? groups : sms)), grad::THREADS, grad::SMEM_BYTES, st, true, a, mq, mk, md);
}

}  // namespace m3
