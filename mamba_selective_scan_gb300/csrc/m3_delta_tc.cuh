// m3_delta_tc.cuh -- shared by the tensor-core kernels of the gated delta
// rule (bf16 activations, chunks of 64 tokens): tcgen05 helpers, operand
// layouts in shared memory, and the way through heads and chunks.
#pragma once

#include "m3_delta.cuh"

namespace m3 {


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
// What the chain kernels keep for the gradients is [16-byte unit][128 rows
// (head_v)][8 elements] without a swizzle (a warp whose lanes are rows writes
// whole lines): an M- or N-major operand whose rows are K, units 2048 bytes
// apart, 8 rows 128 bytes apart; a step of 16 in K is 256 bytes.
__device__ __forceinline__ uint64_t tc_desc_plain(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(2048 >> 4) << 32 | 1ull << 46;
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
// values 2 j and 2 j + 1 of 16 consecutive shared-memory floats, as pairs: read
// where they are used, or (16-byte aligned) at once by half as many loads,
// where the registers allow it
struct Vec16 {
  const float* p;
  __device__ __forceinline__ float2 operator[](int j) const { return *reinterpret_cast<const float2*>(p + 2 * j); }
};
struct Reg16 {
  float2 x[8];
  __device__ __forceinline__ explicit Reg16(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = reinterpret_cast<const float4*>(p)[i];
      x[2 * i] = make_float2(t.x, t.y);
      x[2 * i + 1] = make_float2(t.z, t.w);
    }
  }
  __device__ __forceinline__ float2 operator[](int j) const { return x[j]; }
};
// byte offset of the 16-byte unit u of row r in a swizzled tile
__device__ __forceinline__ uint32_t sw(uint32_t r, uint32_t u) { return r * 128 + ((u ^ (r & 7)) << 4); }

// ---- shared memory ----
// A chunk's inputs are tiles [64 tokens][64 columns].  K and Q alternate (K of
// columns 0-63, Q of 0-63, K of 64-127, Q of 64-127), so that K over Q is one
// operand of 128 rows whose column halves are 2 tiles apart.
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
struct TcPrep {  // what the preparing kernel leaves for one chunk and head
  TcTP tp;
  TcVec vec;
};
static_assert(sizeof(TcPrep) <= TC_PREP && sizeof(TcPrep) % 16 == 0, "one bulk copy");

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
// Which (head, chunk) a block works on at each step.  Either one run of
// chunks of one head (a time segment), or, when there are more heads than
// SMs, an equal share of all chunks of all heads: block s of G has the range
// [s, s + 1) / G of the heads' chunks laid end to end.  It starts with the
// first chunks of the head that the next block ends, hands that head's state
// on, goes through its whole heads, and ends with the last chunks of the
// head that the block before began.  There are no more blocks than heads, so a
// share is at least a head long: a head has two blocks at most, and the part
// handed on is never longer than what its receiver does before it.
struct TcStep {
  int bh, c;          // head (batch row x value head), chunk
  bool first, last;   // of a run
  bool take, give;    // the run starts from, or ends in, a state handed over
};
inline unsigned delta_share_blocks(int64_t heads, int sms) { return (unsigned)(heads < sms ? heads : sms); }
struct TcWalk {
  int nc, n, len_a, whole, h0, c0, ha, ca;
  bool stream;
  __device__ __forceinline__ TcWalk(const DeltaArgs& a, int seg)
      : TcWalk(a.stream, (int64_t)a.B * a.Hv, a.nc, blockIdx.x, gridDim.x, seg, a.seg_chunks) {}
  __host__ __device__ __forceinline__ TcWalk(bool shares, int64_t heads, int chunks, unsigned block, unsigned blocks, int seg,
                                             int seg_chunks) {
    nc = chunks;
    stream = shares;
    if (stream) {
      const int64_t total = heads * nc;
      const int64_t r0 = total * block / blocks, r1 = total * (block + 1) / blocks;
      const int hs = (int)(r0 / nc);
      c0 = (int)(r0 % nc);
      ha = (int)(r1 / nc);
      len_a = (int)(r1 % nc);
      ca = 0;
      h0 = c0 ? hs : hs - 1;  // whole heads are h0 + 1 ...
      whole = ha - h0 - 1;
      n = (int)(r1 - r0);
    } else {
      ha = (int)block;
      ca = seg * seg_chunks;
      len_a = n = (nc < ca + seg_chunks ? nc : ca + seg_chunks) - ca;
      h0 = c0 = whole = 0;
    }
  }
  __host__ __device__ __forceinline__ TcStep at(int i) const {
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

// One chunk's tiles of a [B, T, H, D] tensor as [64 tokens][64 columns],
// 128-byte swizzle; columns past D and tokens past T arrive as zeros.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int col, int head, int tok, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(tok), "r"(b), "r"(smem_u32(bar)) : "memory");
}

// An untiled copy of `bytes` (a multiple of 16) into shared memory
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
// The same tile back (only columns below D and tokens below T are written)
__device__ __forceinline__ void tma_tile_store(const CUtensorMap* map, uint32_t src, int col, int head, int tok, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(col), "r"(head), "r"(tok), "r"(b) : "memory");
}

// The chain kernels' grid: a block per (head, segment), or one per SM (and not
// more than heads) in equal shares.  Those wait for a state that the block before hands over, so
// they are launched cooperatively (all of them resident at once).  Otherwise,
// with `pdl`, the blocks may come up while the kernel before them ends.
template <typename... Args, typename... Vals>
cudaError_t launch_delta_blocks(void (*kern)(Args...), const DeltaArgs& a, int threads, size_t smem, cudaStream_t st, bool pdl,
                                Vals... maps) {
  cudaLaunchConfig_t cfg{};
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  cfg.gridDim = a.stream ? dim3(delta_share_blocks((int64_t)a.B * a.Hv, sms)) : dim3((unsigned)(a.B * a.Hv), (unsigned)a.segs);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  if (a.stream) {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = a.stream || pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a, maps...);
}

}  // namespace m3
