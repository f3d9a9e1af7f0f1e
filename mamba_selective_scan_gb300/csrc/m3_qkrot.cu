// m3_qkrot.cu -- queries and keys on their way into attention: the norm of
// each head (root mean square, with a weight) and the rotation by position in
// one pass, forward and backward: kernels, validation and the C entry points.
//
//   forward   n = x r w,  r = 1 / sqrt(mean(x^2) + eps)
//             pair (a, b) of n -> (a c - b s, a s + b c),  c, s = cos, sin of position * inv_freq
//   backward  dn = dy turned back,  d_w = sum dn x r
//             dx = r (dn w - x r^2 mean(dn w x))
//
// Every value is read once and written once.  A thread owns both halves of its
// pairs (two vectors of 16 bytes), so the rotation is arithmetic in registers
// and the sum of squares two to four shuffles.  Forward, HBM is the bound: 4 x
// 4096 tokens with 40 + 40 heads of 128 take 115 us, 5.8 TB/s.  Backward, the
// arithmetic of the sums counts too: 8 x 2048 with 12 + 12 heads take 61 us (4.9
// TB/s, issue slots 59 % busy), and 6 us more the sum of the blocks' shares of
// the weights' gradients.
//
// Angles.  position * inv_freq in f32 is off by 0.03 radians at position 10^6.
// Here the frequency becomes turns per position as a 64-bit fraction, and its
// product with the integer position, modulo a turn, is one integer
// multiplication without any rounding: at position p the angle is off by at most
// p 2^-63 turns, for the fraction's own rounding.  A block makes the cosines and
// sines of its tokens once, for all heads.

#include <initializer_list>

#include "m3_delta.cuh"  // sm_count

namespace m3 {
namespace {

constexpr int ROT_DMAX = 256;       // head size, at most
constexpr int ROT_THREADS = 256;
constexpr int ROT_WARPS = ROT_THREADS / 32;
constexpr int ROT_BLOCKS = 456;     // share rows of the backward's workspace (and its blocks), at most

struct RotSide {      // queries, or keys
  const void *x, *dy; // [tokens][heads][D], heads dense; dy: the gradient of the output
  void* y;            // output, or the gradient of x
  int64_t xs, dys, ys;  // elements between tokens
  const float* w;
  float* dw;
  int heads, groups, its, units;  // groups of heads a warp takes at once; units of `its` groups per token
  int blocks;
};
struct RotArgs {
  RotSide side[2];
  const float* freq;
  const int64_t* pos;
  int64_t pos_bs;     // between batch rows (0: the same for all)
  float* part;        // [blocks][D]
  int64_t tokens;
  int T, D, R;        // R pairs turn
  int np, group;      // slots per head, lanes per head
  int accumulate;
  float eps;
};

// turns per position as a 64-bit fraction: 1 / (2 pi) in three parts of 28 bits,
// whose products with a float are exact in a double (one double's product would
// be off by 2^-56 turns at a radian per position, 8e-6 radians at position 2^36)
__device__ __forceinline__ uint64_t turn_step(float freq) {
  const double part[3] = {0x1.45f306cp-3, 0x1.c9c882ap-31, 0x1.4fe13aap-61};
  uint64_t sum = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    double t = (double)freq * part[i];
    t -= rint(t);
    sum += (uint64_t)__double2ll_rn(t * 18446744073709551616.0);
  }
  return sum;
}
// cos and sin of that many positions' turn: the angle within an eighth of the
// nearest quarter turn, and Taylor's series there (to x^9 and x^10: the next
// terms are below 2e-9)
__device__ __forceinline__ float2 turn_of(int64_t pos, uint64_t step) {
  const uint64_t ph = (uint64_t)pos * step;                     // of a turn, in 2^-64
  const int quad = (int)((ph + (1ull << 61)) >> 62);
  const int rest = (int)((int64_t)(ph - ((uint64_t)quad << 62)) >> 30);  // in 2^-34
  const float x = (float)rest * (6.2831853071795864769f * 0x1p-34f), z = x * x;
  const float s = x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880.0f, -1.0f / 5040.0f), 1.0f / 120.0f), -1.0f / 6.0f), 1.0f);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800.0f, 1.0f / 40320.0f), -1.0f / 720.0f), 1.0f / 24.0f), -0.5f), 1.0f);
  const float a = quad & 1 ? -s : c, b = quad & 1 ? c : s;
  return quad & 2 ? make_float2(-a, -b) : make_float2(a, b);
}

// VEC consecutive values as they are in memory
template <typename T, int VEC> struct Raw;
template <> struct Raw<float, 4> { float4 v; };
template <> struct Raw<float, 1> { float v; };
template <> struct Raw<__nv_bfloat16, 8> { uint4 v; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 v; };
// and as f32
__device__ __forceinline__ void open(const Raw<float, 4>& r, float (&v)[4]) { v[0] = r.v.x; v[1] = r.v.y; v[2] = r.v.z; v[3] = r.v.w; }
__device__ __forceinline__ void open(const Raw<float, 1>& r, float (&v)[1]) { v[0] = r.v; }
__device__ __forceinline__ void open(const Raw<__nv_bfloat16, 1>& r, float (&v)[1]) { v[0] = __bfloat162float(r.v); }
__device__ __forceinline__ void open(const Raw<__nv_bfloat16, 8>& r, float (&v)[8]) {
  const uint32_t x[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(x[i] << 16);
    v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void put(float* p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[1]) { *p = __float2bfloat16_rn(v[0]); }
__device__ __forceinline__ void put(float* p, const float (&v)[4]) { *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[8]) {
  __nv_bfloat162 t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
}
// The pairs of a slot's two vectors: first values p, second values q, two
// pairs to a float2 (of a vector of one value the second half stays 0)
template <int VEC> struct Pairs {
  static constexpr int N = VEC > 1 ? VEC / 2 : 1;
  float2 p[N], q[N];
  __device__ __forceinline__ float& first(int j) { return j & 1 ? p[j >> 1].y : p[j >> 1].x; }
  __device__ __forceinline__ float& second(int j) { return j & 1 ? q[j >> 1].y : q[j >> 1].x; }
  // value i of vector h: halves of a head, or neighbours
  template <bool IL> __device__ __forceinline__ float& at(int h, int i) {
    if (!IL || VEC == 1) return h ? second(i) : first(i);
    const int e = h * VEC + i;
    return e & 1 ? second(e >> 1) : first(e >> 1);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = q[j] = f2b(0.0f);
  }
  template <bool IL, typename T> __device__ __forceinline__ void take(const Raw<T, VEC> (&r)[2]) {
    if (VEC == 1) zero();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[VEC];
      open(r[h], v);
#pragma unroll
      for (int i = 0; i < VEC; ++i) at<IL>(h, i) = v[i];
    }
  }
  template <bool IL, typename T> __device__ __forceinline__ void give(T* dst, int h) {
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = at<IL>(h, i);
    put(dst, v);
  }
};
__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }

// Slot u of a head: the elements e0 .. e0 + VEC and e1 .. e1 + VEC, and the
// pairs u VEC .. of the table.  Half-split: the slots below R / VEC hold the
// two halves of their pairs, the ones behind what is not turned.  Neighbours:
// 2 VEC elements in a row.
template <int VEC, bool IL> __device__ __forceinline__ void slot_at(const RotArgs& a, int u, int& e0, int& e1) {
  const int turned = a.R / VEC;
  if (IL || u >= turned) {
    e0 = (IL ? 2 * u : 2 * turned + 2 * (u - turned)) * VEC;
    e1 = e0 + VEC;
  } else {
    e0 = u * VEC;
    e1 = a.R + u * VEC;
  }
}

// A unit of work is a token and `its` groups of its heads: a warp takes 32 /
// group heads at a time, with the token's cosines and sines (and the weights)
// in registers and the next groups' values on their way, across units.  A
// warp makes its token's cosines and sines itself, so no barrier stands
// between units.  Blocks take the queries or the keys.  PART: not all of a head
// turns (4 x 4096 with 40 + 40 heads, half turned, 122 -> 124 us forward; as a
// condition in one kernel for all it cost the backward of 8 x 2048 with 12 + 12
// heads a third, 66 -> 86 us).
template <typename T, int VEC, int NS, bool IL, bool BWD, bool PART>
__global__ void __launch_bounds__(ROT_THREADS, 2) m3_qkrot_kernel(const __grid_constant__ RotArgs a) {
  constexpr int ROW = VEC > 1 ? ROT_DMAX / 2 : 32 * NS;  // pairs of a head, at most
  __shared__ __align__(16) float2 cs_all[ROT_WARPS][ROW];
  __shared__ uint64_t steps[ROT_DMAX / 2];
  __shared__ float lost[ROT_DMAX / 2];  // NaN where a frequency is not finite, else 0
  extern __shared__ float comb[];       // backward: [warps][D]
  const bool keys = blockIdx.x >= (unsigned)a.side[0].blocks;
  const RotSide& sd = a.side[keys];
  const int block = keys ? blockIdx.x - a.side[0].blocks : blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.group, at_once = 32 / group, u0 = lane % group, sub = lane / group;
  const int row = a.np * VEC;  // pairs of a head
  const float inv = 1.0f / (float)a.D;
  float2* cs = cs_all[warp];
  using P = Pairs<VEC>;
  constexpr int N = P::N;
  int e0[NS], e1[NS];
  bool l0[NS], l1[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int u = u0 + i * group;
    slot_at<VEC, IL>(a, u, e0[i], e1[i]);
    l0[i] = u < a.np && e0[i] < a.D;
    l1[i] = u < a.np && e1[i] < a.D;
    if (!l0[i]) e0[i] = 0;
    if (!l1[i]) e1[i] = 0;
  }
  P w[NS];
  auto weights = [&]() {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      w[i].zero();
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        w[i].template at<IL>(0, j) = sd.w ? sd.w[e0[i] + j] : 1.0f;
        w[i].template at<IL>(1, j) = sd.w ? sd.w[e1[i] + j] : 1.0f;
      }
    }
  };
  if (BWD) weights();
  // PART: x of slot i's pairs 2 j and 2 j + 1 that turn, 0 of those that do not: a
  // value (or a weight) that is not finite stays out of the one it shares a pair with
  auto turned = [&](int i, int j, float2 x) {
    if (!PART) return x;
    const int m = (u0 + i * group) * VEC + 2 * j;
    return make_float2(m < a.R ? x.x : 0.0f, m + 1 < a.R ? x.y : 0.0f);
  };
  P dw[BWD ? NS : 1];
#pragma unroll
  for (int i = 0; i < (BWD ? NS : 1); ++i) dw[i].zero();
  for (int m = threadIdx.x; m < a.R; m += ROT_THREADS) {
    const float f = a.freq[m];
    steps[m] = turn_step(f);
    lost[m] = f * 0.0f;
  }
  __syncthreads();

  // the values of a group of a token's heads (what no fetch fills stays zero)
  struct Values {
    Raw<T, VEC> x[NS][2], y[BWD ? NS : 1][2];
    __device__ __forceinline__ void zero() {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        x[i][0] = x[i][1] = Raw<T, VEC>{};
        if constexpr (BWD) y[i][0] = y[i][1] = Raw<T, VEC>{};
      }
    }
  };
  constexpr int AHEAD = BWD ? 1 : 2;  // groups on their way (backward, two would not fit the registers)
  Values val[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) val[k].zero();
  auto fetch = [&](Values& r, int64_t tok, int g) {
    const int h = g * at_once + sub;
    const int at = h * a.D;
    const T* xp = static_cast<const T*>(sd.x) + tok * sd.xs + at;
    const T* yp = static_cast<const T*>(sd.dy) + tok * sd.dys + at;
    if (h < sd.heads) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (l0[i]) r.x[i][0] = *reinterpret_cast<const Raw<T, VEC>*>(xp + e0[i]);
        if (l1[i]) r.x[i][1] = *reinterpret_cast<const Raw<T, VEC>*>(xp + e1[i]);
        if constexpr (BWD) {
          if (l0[i]) r.y[i][0] = *reinterpret_cast<const Raw<T, VEC>*>(yp + e0[i]);
          if (l1[i]) r.y[i][1] = *reinterpret_cast<const Raw<T, VEC>*>(yp + e1[i]);
        }
      }
    } else {
      r.zero();
    }
  };
  // this warp's units: `step` apart, counted as token (batch row b, time t) and
  // part of its groups
  struct Unit {
    int64_t tok, pos;
    int b, t, part, g0, g1;
  };
  const int64_t step = (int64_t)sd.blocks * ROT_WARPS;
  const int64_t step_tok = step / sd.units;
  const int step_part = (int)(step % sd.units), step_b = (int)(step_tok / a.T), step_t = (int)(step_tok % a.T);
  auto place = [&](Unit& r) {
    if (r.tok >= a.tokens) {
      r.g0 = r.g1 = 0;
      return;
    }
    r.g0 = r.part * sd.its;
    r.g1 = min(r.g0 + sd.its, sd.groups);
    if (a.R > 0) r.pos = a.pos[r.b * a.pos_bs + r.t];
  };
  Unit now;
  {
    const int64_t first = (int64_t)block * ROT_WARPS + warp;
    now.tok = first / sd.units;
    now.part = (int)(first % sd.units);
    now.b = (int)(now.tok / a.T);
    now.t = (int)(now.tok % a.T);
    now.pos = 0;
    place(now);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (now.g0 + k < now.g1) fetch(val[k], now.tok, now.g0 + k);
  }
  while (now.tok < a.tokens) {
    Unit then = now;
    then.tok += step_tok;
    then.b += step_b;
    then.t += step_t;
    then.part += step_part;
    if (then.part >= sd.units) {
      then.part -= sd.units;
      ++then.tok;
      ++then.t;
    }
    if (then.t >= a.T) {
      then.t -= a.T;
      ++then.b;
    }
    place(then);
    __syncwarp();
    for (int m = lane; m < row; m += 32) {
      float2 c = make_float2(1.0f, 0.0f);
      if (m < a.R) {
        c = turn_of(now.pos, steps[m]);
        c.x += lost[m];
        c.y += lost[m];
      }
      cs[m] = c;
    }
    __syncwarp();
    // cosines and sines; forward, times the weights: of the first value and
    // of the second in either output
    if (!BWD) weights();  // (there again for each unit: no registers in between)
    float2 co[NS][N], si[NS][N], wc[BWD ? 1 : NS][N], ws[BWD ? 1 : NS][N];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float2* tb = cs + (l0[i] ? u0 + i * group : 0) * VEC;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float2 c0 = tb[2 * j], c1 = VEC > 1 ? tb[2 * j + 1] : f2b(0.0f);
        co[i][j] = make_float2(c0.x, c1.x);
        si[i][j] = make_float2(c0.y, c1.y);
        if constexpr (!BWD) {
          wc[i][j] = __fmul2_rn(w[i].q[j], co[i][j]);
          ws[i][j] = turned(i, j, neg2(__fmul2_rn(w[i].q[j], si[i][j])));
          co[i][j] = __fmul2_rn(w[i].p[j], co[i][j]);
          si[i][j] = turned(i, j, __fmul2_rn(w[i].p[j], si[i][j]));
        }
      }
    }
    T* op = static_cast<T*>(sd.y) + now.tok * sd.ys;
    auto work = [&](int g, int k) {  // group g, and its values' place for the one that comes AHEAD of it
      Values& r = val[k];
      const int h = g * at_once + sub;
      const bool live = h < sd.heads;
      P v[NS], u[BWD ? NS : 1];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        v[i].template take<IL, T>(r.x[i]);
        if constexpr (BWD) u[i].template take<IL, T>(r.y[i]);
      }
      if (g + AHEAD < now.g1) fetch(r, now.tok, g + AHEAD);
      else if (then.g0 + k < then.g1) fetch(r, then.tok, then.g0 + k);
      float2 s2 = f2b(0.0f);
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) s2 = __ffma2_rn(v[i].p[j], v[i].p[j], __ffma2_rn(v[i].q[j], v[i].q[j], s2));
      float ss = s2.x + s2.y;
      for (int o = 1; o < group; o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
      const float rn = live ? rsqrtf(ss * inv + a.eps) : 0.0f;  // (no head: 1 / sqrt(0) with eps 0)
      const float2 r2 = f2b(rn);
      if constexpr (!BWD) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float2 p = __fmul2_rn(v[i].p[j], r2), q = __fmul2_rn(v[i].q[j], r2);
            v[i].p[j] = __ffma2_rn(p, co[i][j], __fmul2_rn(turned(i, j, q), ws[i][j]));
            v[i].q[j] = __ffma2_rn(turned(i, j, p), si[i][j], __fmul2_rn(q, wc[i][j]));
          }
      } else {
        // u = r dn w,  dx = u - x r^2 mean(u x)
        float2 d2 = f2b(0.0f);
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float2 p = __fmul2_rn(u[i].p[j], r2), q = __fmul2_rn(u[i].q[j], r2);
            const float2 np = __ffma2_rn(p, co[i][j], __fmul2_rn(turned(i, j, q), si[i][j]));
            const float2 nq = __ffma2_rn(q, co[i][j], __fmul2_rn(turned(i, j, p), neg2(si[i][j])));
            dw[i].p[j] = __ffma2_rn(np, v[i].p[j], dw[i].p[j]);
            dw[i].q[j] = __ffma2_rn(nq, v[i].q[j], dw[i].q[j]);
            u[i].p[j] = __fmul2_rn(np, w[i].p[j]);
            u[i].q[j] = __fmul2_rn(nq, w[i].q[j]);
            d2 = __ffma2_rn(u[i].p[j], v[i].p[j], __ffma2_rn(u[i].q[j], v[i].q[j], d2));
          }
        float dot = d2.x + d2.y;
        for (int o = 1; o < group; o <<= 1) dot += __shfl_xor_sync(~0u, dot, o);
        const float2 m = f2b(-dot * inv * rn * rn);
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j) {
            v[i].p[j] = __ffma2_rn(v[i].p[j], m, u[i].p[j]);
            v[i].q[j] = __ffma2_rn(v[i].q[j], m, u[i].q[j]);
          }
      }
      T* dst = op + h * a.D;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        if (live && l0[i]) v[i].template give<IL>(dst + e0[i], 0);
        if (live && l1[i]) v[i].template give<IL>(dst + e1[i], 1);
      }
    };
#pragma unroll 1
    for (int g = now.g0; g < now.g1; g += AHEAD) {
      work(g, 0);
      if constexpr (AHEAD > 1) {
        if (g + 1 < now.g1) work(g + 1, 1);
        else if (g == now.g0 && then.g0 + 1 < then.g1) fetch(val[1], then.tok, then.g0 + 1);  // (of more groups the last pair fetched it)
      }
    }
    now = then;
  }
  if constexpr (BWD) {
    // this block's share of the weight's gradient: lanes that hold the same
    // slots, then the warps, in a fixed order
    grid_dep_trigger();
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int j = 0; j < 2 * VEC; ++j) {
        float d = dw[i].template at<IL>(j / VEC, j % VEC);
        for (int o = group; o < 32; o <<= 1) d += __shfl_xor_sync(~0u, d, o);
        if (sub == 0 && (j < VEC ? l0[i] : l1[i])) comb[warp * a.D + (j < VEC ? e0[i] + j : e1[i] + j - VEC)] = d;
      }
    __syncthreads();
    for (int k = threadIdx.x; k < a.D; k += ROT_THREADS) {
      float d = 0.0f;
      for (int m = 0; m < ROT_WARPS; ++m) d += comb[m * a.D + k];
      a.part[(size_t)blockIdx.x * a.D + k] = d;
    }
  }
}

// The weights' gradients: the blocks' shares [blocks][D] added over the
// blocks, 32 columns per block, the rows over 32 warps and a fixed tree.
__global__ void __launch_bounds__(1024) m3_qkrot_wgrad_kernel(const __grid_constant__ RotArgs a) {
  __shared__ float sh[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  const RotSide& sd = a.side[blockIdx.y];
  const float* part = a.part + (blockIdx.y ? (size_t)a.side[0].blocks * a.D : 0) + c;
  grid_dep_wait();
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < a.D) {
    int r = warp;
    for (; r + 96 < sd.blocks; r += 128)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += part[(size_t)(r + 32 * i) * a.D];
    for (; r < sd.blocks; r += 32) s[0] += part[(size_t)r * a.D];
  }
  sh[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  float t = sh[lane][warp];  // column blockIdx.x * 32 + warp
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
  const int cc = blockIdx.x * 32 + warp;
  if (lane == 0 && cc < a.D && sd.dw) sd.dw[cc] = a.accumulate ? sd.dw[cc] + t : t;
}

m3_status rot_validate(const m3_qkrot_dims* d, m3_dtype act) {
  if (!d) return M3_ERR_NULL;
  if (act != M3_F32 && act != M3_BF16) return M3_ERR_UNSUPPORTED;
  if (d->batch < 0 || d->seq_len < 0 || d->q_heads < 1 || d->k_heads < 1) return M3_ERR_DIMS;
  if (d->head_dim < 2) return M3_ERR_DIMS;  // of a single value the norm leaves its sign, and a gradient that is all cancellation
  if (d->batch > (int64_t)1 << 30 || d->seq_len > (int64_t)1 << 30 || d->batch * d->seq_len > (int64_t)1 << 33) return M3_ERR_DIMS;
  if (d->q_heads > 65535 || d->k_heads > 65535 || !(d->eps >= 0.0f)) return M3_ERR_DIMS;
  if (d->reserved != 0) return M3_ERR_DIMS;
  if (d->head_dim > ROT_DMAX) return M3_ERR_UNSUPPORTED;
  if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 2) return M3_ERR_DIMS;
  if ((d->interleaved != 0 && d->interleaved != 1) || (d->accumulate_param_grads != 0 && d->accumulate_param_grads != 1))
    return M3_ERR_DIMS;
  if (d->position_stride != 0 && (d->position_stride < d->seq_len || d->position_stride > (int64_t)1 << 40)) return M3_ERR_DIMS;
  const int64_t qw = d->q_heads * d->head_dim, kw = d->k_heads * d->head_dim;
  const struct { int64_t stride, width; } rows[] = {{d->q_stride, qw}, {d->k_stride, kw}, {d->q_out_stride, qw}, {d->k_out_stride, kw},
                                                    {d->dq_stride, qw}, {d->dk_stride, kw}, {d->dq_out_stride, qw}, {d->dk_out_stride, kw}};
  for (const auto& r : rows)
    if (r.stride != 0 && (r.stride < r.width || r.stride > (int64_t)1 << 24)) return M3_ERR_DIMS;
  return M3_OK;
}

int64_t rot_parts(const m3_qkrot_dims* d) {
  return d->batch && d->seq_len ? ROT_BLOCKS : 0;
}

RotArgs rot_args(const m3_qkrot_dims* d, const void* q, const void* k, const float* wq, const float* wk, const int64_t* pos,
                 const float* freq) {
  RotArgs a{};
  const int64_t qw = d->q_heads * d->head_dim, kw = d->k_heads * d->head_dim;
  a.side[0].x = q; a.side[1].x = k;
  a.side[0].xs = d->q_stride ? d->q_stride : qw;
  a.side[1].xs = d->k_stride ? d->k_stride : kw;
  a.side[0].w = wq; a.side[1].w = wk;
  a.side[0].heads = (int)d->q_heads; a.side[1].heads = (int)d->k_heads;
  a.pos = pos; a.freq = freq;
  a.pos_bs = d->position_stride;
  a.tokens = d->batch * d->seq_len;
  a.T = (int)d->seq_len;
  a.D = (int)d->head_dim; a.R = (int)d->rot_dim / 2;
  a.eps = d->eps;
  a.accumulate = d->accumulate_param_grads;
  return a;
}

template <typename T, int VEC, int NS, bool IL, bool BWD, bool PART>
cudaError_t rot_go(RotArgs& a, cudaStream_t s) {
  auto kern = m3_qkrot_kernel<T, VEC, NS, IL, BWD, PART>;
  int sms = 0, occ = 0;
  const size_t smem = BWD ? (size_t)ROT_WARPS * a.D * 4 : 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, ROT_THREADS, smem);
  if (e != cudaSuccess) return e;
  int64_t blocks = (int64_t)sms * (occ < 1 ? 1 : occ);
  if (BWD && blocks > ROT_BLOCKS) blocks = ROT_BLOCKS;
  if (blocks < 2) blocks = 2;
  // blocks by the sides' work; groups per unit: a token's, but no fewer units
  // than a side's warps
  const int at_once = 32 / a.group;
  int64_t all = 0, left = blocks;
  for (RotSide& sd : a.side) all += sd.groups = (sd.heads + at_once - 1) / at_once;
  for (int i = 0; i < 2; ++i) {
    RotSide& sd = a.side[i];
    int64_t n = i ? left : (blocks * sd.groups + all / 2) / all;
    if (i == 0 && n > blocks - 1) n = blocks - 1;
    if (n < 1) n = 1;
    left -= n;
    const int64_t its = sd.groups * a.tokens / (n * ROT_WARPS);
    sd.its = its < 1 ? 1 : its > sd.groups ? sd.groups : (int)its;
    sd.units = (sd.groups + sd.its - 1) / sd.its;
    const int64_t need = (a.tokens * sd.units + ROT_WARPS - 1) / ROT_WARPS;
    sd.blocks = (int)(n < need ? n : need);
  }
  e = launch_k(kern, dim3((unsigned)(a.side[0].blocks + a.side[1].blocks)), ROT_THREADS, smem, s, false, a);
  if (BWD && e == cudaSuccess)
    e = launch_k(m3_qkrot_wgrad_kernel, dim3((unsigned)((a.D + 31) / 32), 2), 1024, 0, s, true, a);
  return e;
}

template <typename T, bool IL, bool BWD, bool PART>
cudaError_t rot_pick(RotArgs& a, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int v = vec ? V : 1;
  a.np = (a.D + 2 * v - 1) / (2 * v);
  a.group = 1;
  while (a.group < a.np && a.group < 32) a.group *= 2;
  const int per = (a.np + a.group - 1) / a.group;
  if (vec) return rot_go<T, V, 1, IL, BWD, PART>(a, s);
  if (per == 1) return rot_go<T, 1, 1, IL, BWD, PART>(a, s);
  if (per == 2) return rot_go<T, 1, 2, IL, BWD, PART>(a, s);
  return rot_go<T, 1, 4, IL, BWD, PART>(a, s);
}
template <typename T, bool BWD>
cudaError_t rot_launch(RotArgs a, bool vec, bool il, cudaStream_t s) {
  if (2 * a.R == a.D) return il ? rot_pick<T, true, BWD, false>(a, vec, s) : rot_pick<T, false, BWD, false>(a, vec, s);
  return il ? rot_pick<T, true, BWD, true>(a, vec, s) : rot_pick<T, false, BWD, true>(a, vec, s);
}

// 16-byte vectors: heads and tokens of every tensor start on 16 bytes, and a
// half-split rotation's halves do
bool rot_vec(const m3_qkrot_dims* d, int es, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> strides) {
  const int v = 16 / es;
  if (d->head_dim % v) return false;
  if (!d->interleaved && d->rot_dim / 2 % v) return false;
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return false;
  for (const int64_t x : strides)
    if (x % v) return false;
  return true;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

m3_status m3scan_qkrot_plan(const m3_qkrot_dims* dims, m3_dtype act, m3_qkrot_plan* out) {
  const m3_status st = rot_validate(dims, act);
  if (st != M3_OK) return st;
  if (!out) return M3_ERR_NULL;
  out->workspace_bytes = STATUS_BYTES + rot_parts(dims) * dims->head_dim * 4;
  return M3_OK;
}

m3_status m3scan_qkrot_fwd(const m3_qkrot_dims* dims, m3_dtype act, const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const int64_t* positions, const float* inv_freq, void* q_out,
                           void* k_out, m3_stream_t stream) {
  const m3_status st = rot_validate(dims, act);
  if (st != M3_OK) return st;
  const int es = act == M3_BF16 ? 2 : 4;
  for (const void* p : {q, k, (const void*)q_out, (const void*)k_out})
    if (!aligned(p, es)) return M3_ERR_ALIGN;
  for (const void* p : {(const void*)q_weight, (const void*)k_weight, (const void*)inv_freq})
    if (!aligned(p, 4)) return M3_ERR_ALIGN;
  if (!aligned(positions, 8)) return M3_ERR_ALIGN;
  if (dims->batch == 0 || dims->seq_len == 0) return M3_OK;
  if (!q || !k || !q_out || !k_out) return M3_ERR_NULL;
  if (dims->rot_dim > 0 && (!positions || !inv_freq)) return M3_ERR_NULL;
  RotArgs a = rot_args(dims, q, k, q_weight, k_weight, positions, inv_freq);
  a.side[0].y = q_out; a.side[1].y = k_out;
  a.side[0].ys = dims->q_out_stride ? dims->q_out_stride : dims->q_heads * dims->head_dim;
  a.side[1].ys = dims->k_out_stride ? dims->k_out_stride : dims->k_heads * dims->head_dim;
  const bool vec = rot_vec(dims, es, {q, k, q_out, k_out}, {a.side[0].xs, a.side[1].xs, a.side[0].ys, a.side[1].ys});
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = act == M3_BF16 ? rot_launch<__nv_bfloat16, false>(a, vec, dims->interleaved, s)
                                       : rot_launch<float, false>(a, vec, dims->interleaved, s);
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

m3_status m3scan_qkrot_bwd(const m3_qkrot_dims* dims, m3_dtype act, const void* dq_out, const void* dk_out, const void* q,
                           const void* k, const float* q_weight, const float* k_weight, const int64_t* positions,
                           const float* inv_freq, void* dq, void* dk, float* d_q_weight, float* d_k_weight,
                           void* workspace, size_t workspace_bytes, m3_stream_t stream) {
  const m3_status st = rot_validate(dims, act);
  if (st != M3_OK) return st;
  const int es = act == M3_BF16 ? 2 : 4;
  for (const void* p : {dq_out, dk_out, q, k, (const void*)dq, (const void*)dk})
    if (!aligned(p, es)) return M3_ERR_ALIGN;
  for (const void* p : {(const void*)q_weight, (const void*)k_weight, (const void*)inv_freq, (const void*)d_q_weight, (const void*)d_k_weight})
    if (!aligned(p, 4)) return M3_ERR_ALIGN;
  if (!aligned(positions, 8)) return M3_ERR_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dims->batch == 0 || dims->seq_len == 0) {  // no tokens: zero sums
    if (!dims->accumulate_param_grads)
      for (float* g : {d_q_weight, d_k_weight})
        if (g && note(cudaMemsetAsync(g, 0, (size_t)dims->head_dim * 4, s)) != cudaSuccess) return M3_ERR_CUDA;
    return M3_OK;
  }
  if (!dq_out || !dk_out || !q || !k || !dq || !dk) return M3_ERR_NULL;
  if (dims->rot_dim > 0 && (!positions || !inv_freq)) return M3_ERR_NULL;
  m3_qkrot_plan pl;
  m3scan_qkrot_plan(dims, act, &pl);
  if (!workspace || (int64_t)workspace_bytes < pl.workspace_bytes) return M3_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return M3_ERR_ALIGN;
  RotArgs a = rot_args(dims, q, k, q_weight, k_weight, positions, inv_freq);
  const int64_t qw = dims->q_heads * dims->head_dim, kw = dims->k_heads * dims->head_dim;
  a.side[0].dy = dq_out; a.side[1].dy = dk_out;
  a.side[0].y = dq; a.side[1].y = dk;
  a.side[0].dys = dims->dq_out_stride ? dims->dq_out_stride : qw;
  a.side[1].dys = dims->dk_out_stride ? dims->dk_out_stride : kw;
  a.side[0].ys = dims->dq_stride ? dims->dq_stride : qw;
  a.side[1].ys = dims->dk_stride ? dims->dk_stride : kw;
  a.side[0].dw = d_q_weight; a.side[1].dw = d_k_weight;
  a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + STATUS_BYTES);
  const bool vec = rot_vec(dims, es, {dq_out, dk_out, q, k, dq, dk},
                           {a.side[0].xs, a.side[1].xs, a.side[0].dys, a.side[1].dys, a.side[0].ys, a.side[1].ys});
  const cudaError_t e = act == M3_BF16 ? rot_launch<__nv_bfloat16, true>(a, vec, dims->interleaved, s)
                                       : rot_launch<float, true>(a, vec, dims->interleaved, s);
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

}  // extern "C"
