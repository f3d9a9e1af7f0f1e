// m3_qkrot.cu -- queries and keys on their way into attention: the norm of
// each head (root mean square, with a weight) and the rotation by position in
// one pass, forward and backward: kernels, validation and the C entry points.
//
//   forward   n = x r w,  r = 1 / sqrt(mean(x^2) + eps)
//             pair (a, b) of n -> (a c - b s, a s + b c),  c, s = cos, sin of position * inv_freq
//   backward  dn = dy turned back,  d_w = sum dn x r
//             dx = r (dn w - x r^2 mean(dn w x))
//
// Both are bound by HBM: every value is read once and written once.  A thread
// owns both halves of its pairs (two vectors of 16 bytes), so the rotation is
// arithmetic in registers and the sum of squares two to four shuffles.
//
// Angles.  position * inv_freq in f32 is off by 0.03 radians at position 10^6.
// Here the frequency becomes turns per position as a 64-bit fraction, and its
// product with the integer position, modulo a turn, is one integer
// multiplication without any rounding: at position p the angle is off by p
// 2^-65 turns for the fraction's own rounding.  A block makes the cosines and
// sines of its tokens once, for all heads.

#include <initializer_list>

#include "m3_delta.cuh"  // sm_count

namespace m3 {
namespace {

constexpr int ROT_DMAX = 256;       // head size, at most
constexpr int ROT_THREADS = 256;
constexpr int ROT_WARPS = ROT_THREADS / 32;
constexpr int ROT_BLOCKS = 608;     // share rows of the backward's workspace (and its blocks), at most
constexpr int ROT_TABLE = 1024;     // pairs of (cos, sin) that a block keeps

struct RotArgs {
  const void *q, *k, *dqo, *dko;  // [tokens][heads][D], heads dense
  void *qo, *ko;                  // outputs: q_out and k_out, or dq and dk
  int64_t qs, ks, dqos, dkos, qos, kos;  // elements between tokens
  const float *wq, *wk, *freq;
  const int64_t* pos;
  int64_t pos_bs;                 // between batch rows (0: the same for all)
  float *part, *dwq, *dwk;        // [blocks][2][D]
  int64_t tokens;
  int T, Hq, Hk, D, R;            // R pairs turn
  int np, per, group;             // slots per head, slots per thread, lanes per head
  int tb;                         // tokens per table
  int nparts, accumulate;
  float eps;
};

// cos and sin of position * freq
__device__ __forceinline__ float2 turn_of(int64_t pos, float freq) {
  if (!(fabsf(freq) <= 3.4028235e38f)) return f2b(__int_as_float(0x7FFFFFFF));
  double t = (double)freq * 0.15915494309189533577;  // turns per position
  t -= rint(t);
  const int64_t step = __double2ll_rn(t * 18446744073709551616.0);
  const uint64_t ph = (uint64_t)pos * (uint64_t)step;       // of a turn, in 2^-64
  const uint64_t near = ph + (1ull << 61);
  const int quad = (int)(near >> 62);                       // the nearest quarter turn
  const int64_t rest = (int64_t)(ph - ((uint64_t)quad << 62));  // within an eighth
  float s, c;
  sincospif((float)rest * 0x1p-63f, &s, &c);
  if (quad & 1) {
    const float x = c;
    c = -s;
    s = x;
  }
  if (quad & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c, s);
}

template <int VEC> __device__ __forceinline__ void ldr(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) v[0] = *p;
  else {
    const float4 t = *reinterpret_cast<const float4*>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  }
}
template <int VEC> __device__ __forceinline__ void ldr(const __nv_bfloat16* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) v[0] = __bfloat162float(*p);
  else {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    const uint32_t x[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(x[i] << 16);
      v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
    }
  }
}
template <int VEC> __device__ __forceinline__ void str(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) *p = v[0];
  else *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <int VEC> __device__ __forceinline__ void str(__nv_bfloat16* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) *p = __float2bfloat16_rn(v[0]);
  else {
    __nv_bfloat162 t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
  }
}

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

// Work is (token, group of heads): a warp takes 32 / group heads at a time.
// A block goes through tables of tb tokens with a grid stride.
template <typename T, int VEC, int NS, bool IL, bool BWD>
__global__ void __launch_bounds__(ROT_THREADS) m3_qkrot_kernel(const __grid_constant__ RotArgs a) {
  __shared__ __align__(16) float2 cs[ROT_TABLE];
  extern __shared__ float comb[];  // backward: [warps][2][D]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.group, heads_at_once = 32 / group, u0 = lane % group, sub = lane / group;
  const int qg = (a.Hq + heads_at_once - 1) / heads_at_once, kg = (a.Hk + heads_at_once - 1) / heads_at_once;
  const int per_tok = qg + kg, row = a.np * VEC;  // table entries per token
  const float inv = 1.0f / (float)a.D;
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
  float dw[BWD ? 2 : 1][NS][2][VEC];
  if constexpr (BWD) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[w][i][0][j] = dw[w][i][1][j] = 0.0f;
  }
  for (int64_t tok0 = (int64_t)blockIdx.x * a.tb; tok0 < a.tokens; tok0 += (int64_t)gridDim.x * a.tb) {
    const int nt = (int)min((int64_t)a.tb, a.tokens - tok0);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * row; i += ROT_THREADS) {
      const int m = i % row;
      const int64_t tok = tok0 + i / row;
      cs[i] = m < a.R ? turn_of(a.pos[tok / a.T * a.pos_bs + tok % a.T], a.freq[m]) : make_float2(1.0f, 0.0f);
    }
    __syncthreads();
    for (int w = warp; w < nt * per_tok; w += ROT_WARPS) {
      const int t = w / per_tok, g = w % per_tok;
      const bool isk = g >= qg;
      const int h = (isk ? g - qg : g) * heads_at_once + sub;
      const bool live = h < (isk ? a.Hk : a.Hq);
      const int64_t tok = tok0 + t;
      const T* src = static_cast<const T*>(isk ? a.k : a.q) + tok * (isk ? a.ks : a.qs) + (int64_t)(live ? h : 0) * a.D;
      T* dst = static_cast<T*>(isk ? a.ko : a.qo) + tok * (isk ? a.kos : a.qos) + (int64_t)(live ? h : 0) * a.D;
      const float* wt = isk ? a.wk : a.wq;
      float x[NS][2][VEC], y[NS][2][VEC];
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[i][0][j] = x[i][1][j] = 0.0f;
        if (live && l0[i]) ldr<VEC>(src + e0[i], x[i][0]);
        if (live && l1[i]) ldr<VEC>(src + e1[i], x[i][1]);
      }
      if constexpr (BWD) {
        const T* up = static_cast<const T*>(isk ? a.dko : a.dqo) + tok * (isk ? a.dkos : a.dqos) + (int64_t)(live ? h : 0) * a.D;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) y[i][0][j] = y[i][1][j] = 0.0f;
          if (live && l0[i]) ldr<VEC>(up + e0[i], y[i][0]);
          if (live && l1[i]) ldr<VEC>(up + e1[i], y[i][1]);
        }
      }
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(x[i][0][j], x[i][0][j], fmaf(x[i][1][j], x[i][1][j], ss));
      for (int o = 1; o < group; o <<= 1) ss += __shfl_xor_sync(~0u, ss, o);
      const float r = live ? rsqrtf(ss * inv + a.eps) : 0.0f;  // (no head: 1 / sqrt(0) with eps 0)
      if constexpr (!BWD) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          float w0[VEC], w1[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) w0[j] = w1[j] = 1.0f;
          if (wt) {
            ldr<VEC == 1 ? 1 : 4>(wt + e0[i], reinterpret_cast<float(&)[VEC == 1 ? 1 : 4]>(w0));
            ldr<VEC == 1 ? 1 : 4>(wt + e1[i], reinterpret_cast<float(&)[VEC == 1 ? 1 : 4]>(w1));
            if constexpr (VEC == 8) {
              ldr<4>(wt + e0[i] + 4, reinterpret_cast<float(&)[4]>(w0[4]));
              ldr<4>(wt + e1[i] + 4, reinterpret_cast<float(&)[4]>(w1[4]));
            }
          }
          const int u = l0[i] ? u0 + i * group : 0;
          const float2* tb = cs + t * row + u * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            x[i][0][j] = x[i][0][j] * r * w0[j];
            x[i][1][j] = x[i][1][j] * r * w1[j];
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float2 c = tb[j];
            float &p = IL && VEC > 1 ? x[i][2 * j / VEC][2 * j % VEC] : x[i][0][j];
            float &q = IL && VEC > 1 ? x[i][2 * j / VEC][2 * j % VEC + 1] : x[i][1][j];
            const float aa = p * c.x - q * c.y, bb = p * c.y + q * c.x;
            p = aa;
            q = bb;
          }
          if (live && l0[i]) str<VEC>(dst + e0[i], x[i][0]);
          if (live && l1[i]) str<VEC>(dst + e1[i], x[i][1]);
        }
      } else {
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          float w0[VEC], w1[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) w0[j] = w1[j] = 1.0f;
          if (wt) {
            ldr<VEC == 1 ? 1 : 4>(wt + e0[i], reinterpret_cast<float(&)[VEC == 1 ? 1 : 4]>(w0));
            ldr<VEC == 1 ? 1 : 4>(wt + e1[i], reinterpret_cast<float(&)[VEC == 1 ? 1 : 4]>(w1));
            if constexpr (VEC == 8) {
              ldr<4>(wt + e0[i] + 4, reinterpret_cast<float(&)[4]>(w0[4]));
              ldr<4>(wt + e1[i] + 4, reinterpret_cast<float(&)[4]>(w1[4]));
            }
          }
          const int u = l0[i] ? u0 + i * group : 0;
          const float2* tb = cs + t * row + u * VEC;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float2 c = tb[j];
            float &p = IL && VEC > 1 ? y[i][2 * j / VEC][2 * j % VEC] : y[i][0][j];
            float &q = IL && VEC > 1 ? y[i][2 * j / VEC][2 * j % VEC + 1] : y[i][1][j];
            const float aa = p * c.x + q * c.y, bb = q * c.x - p * c.y;
            p = aa;
            q = bb;
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float a0 = y[i][0][j] * x[i][0][j] * r, a1 = y[i][1][j] * x[i][1][j] * r;
            if (isk) {
              dw[1][i][0][j] += a0;
              dw[1][i][1][j] += a1;
            } else {
              dw[0][i][0][j] += a0;
              dw[0][i][1][j] += a1;
            }
            dot = fmaf(a0, w0[j], fmaf(a1, w1[j], dot));
            y[i][0][j] *= w0[j];
            y[i][1][j] *= w1[j];
          }
        }
        for (int o = 1; o < group; o <<= 1) dot += __shfl_xor_sync(~0u, dot, o);
        const float m = dot * inv * r;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            y[i][0][j] = r * (y[i][0][j] - x[i][0][j] * m);
            y[i][1][j] = r * (y[i][1][j] - x[i][1][j] * m);
          }
          if (live && l0[i]) str<VEC>(dst + e0[i], y[i][0]);
          if (live && l1[i]) str<VEC>(dst + e1[i], y[i][1]);
        }
      }
    }
  }
  if constexpr (BWD) {
    // this block's share of the weights' gradients: lanes that hold the same
    // slots, then the warps, in a fixed order
    grid_dep_trigger();
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float s0 = dw[w][i][0][j], s1 = dw[w][i][1][j];
          for (int o = group; o < 32; o <<= 1) {
            s0 += __shfl_xor_sync(~0u, s0, o);
            s1 += __shfl_xor_sync(~0u, s1, o);
          }
          if (sub == 0 && l0[i]) comb[(warp * 2 + w) * a.D + e0[i] + j] = s0;
          if (sub == 0 && l1[i]) comb[(warp * 2 + w) * a.D + e1[i] + j] = s1;
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += ROT_THREADS) {
      float s = 0.0f;
      for (int w = 0; w < ROT_WARPS; ++w) s += comb[w * 2 * a.D + c];
      a.part[(size_t)blockIdx.x * 2 * a.D + c] = s;
    }
  }
}

// The weights' gradients: the blocks' shares [nparts][2][D] added over the
// blocks, 32 columns per block, the rows over 32 warps and a fixed tree.
__global__ void __launch_bounds__(1024) m3_qkrot_wgrad_kernel(const __grid_constant__ RotArgs a) {
  __shared__ float sh[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane, n2 = 2 * a.D;
  grid_dep_wait();
  float s = 0.0f;
  if (c < n2)
    for (int r = warp; r < a.nparts; r += 32) s += a.part[(size_t)r * n2 + c];
  sh[warp][lane] = s;
  __syncthreads();
  float t = sh[lane][warp];  // column blockIdx.x * 32 + warp
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(~0u, t, o);
  const int cc = blockIdx.x * 32 + warp;
  if (lane == 0 && cc < n2) {
    float* o = cc < a.D ? a.dwq : a.dwk;
    if (o) {
      o += cc < a.D ? cc : cc - a.D;
      *o = a.accumulate ? *o + t : t;
    }
  }
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
  const int64_t n = d->batch * d->seq_len;
  return n < ROT_BLOCKS ? n : ROT_BLOCKS;
}

RotArgs rot_args(const m3_qkrot_dims* d, const float* wq, const float* wk, const int64_t* pos, const float* freq) {
  RotArgs a{};
  const int64_t qw = d->q_heads * d->head_dim, kw = d->k_heads * d->head_dim;
  a.qs = d->q_stride ? d->q_stride : qw;
  a.ks = d->k_stride ? d->k_stride : kw;
  a.wq = wq; a.wk = wk; a.pos = pos; a.freq = freq;
  a.pos_bs = d->position_stride;
  a.tokens = d->batch * d->seq_len;
  a.T = (int)d->seq_len; a.Hq = (int)d->q_heads; a.Hk = (int)d->k_heads;
  a.D = (int)d->head_dim; a.R = (int)d->rot_dim / 2;
  a.eps = d->eps;
  a.accumulate = d->accumulate_param_grads;
  return a;
}

template <typename T, int VEC, int NS, bool IL, bool BWD>
cudaError_t rot_go(RotArgs& a, cudaStream_t s) {
  auto kern = m3_qkrot_kernel<T, VEC, NS, IL, BWD>;
  int sms = 0, occ = 0;
  const size_t smem = BWD ? (size_t)ROT_WARPS * 2 * a.D * 4 : 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, ROT_THREADS, smem);
  if (e != cudaSuccess) return e;
  // tokens per table: as many as it holds, but no fewer blocks than fit the GPU at once
  int64_t blocks = (int64_t)sms * (occ < 1 ? 1 : occ);
  if (BWD && blocks > ROT_BLOCKS) blocks = ROT_BLOCKS;
  const int64_t row = (int64_t)a.np * VEC;
  int64_t tb = ROT_TABLE / row, fill = (a.tokens + blocks - 1) / blocks;
  if (tb > fill) tb = fill;
  if (tb < 1) tb = 1;
  a.tb = (int)tb;
  const int64_t need = (a.tokens + tb - 1) / tb;
  if (blocks > need) blocks = need;
  a.nparts = (int)blocks;
  e = launch_k(kern, dim3((unsigned)blocks), ROT_THREADS, smem, s, false, a);
  if (BWD && e == cudaSuccess)
    e = launch_k(m3_qkrot_wgrad_kernel, dim3((unsigned)((2 * a.D + 31) / 32)), 1024, 0, s, true, a);
  return e;
}

template <typename T, bool BWD>
cudaError_t rot_launch(RotArgs a, bool vec, bool il, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int v = vec ? V : 1;
  a.np = (a.D + 2 * v - 1) / (2 * v);
  a.group = 1;
  while (a.group < a.np && a.group < 32) a.group *= 2;
  a.per = (a.np + a.group - 1) / a.group;
  if (vec) return il ? rot_go<T, V, 1, true, BWD>(a, s) : rot_go<T, V, 1, false, BWD>(a, s);
  if (a.per == 1) return il ? rot_go<T, 1, 1, true, BWD>(a, s) : rot_go<T, 1, 1, false, BWD>(a, s);
  if (a.per == 2) return il ? rot_go<T, 1, 2, true, BWD>(a, s) : rot_go<T, 1, 2, false, BWD>(a, s);
  return il ? rot_go<T, 1, 4, true, BWD>(a, s) : rot_go<T, 1, 4, false, BWD>(a, s);
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
  out->workspace_bytes = STATUS_BYTES + rot_parts(dims) * 2 * dims->head_dim * 4;
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
  RotArgs a = rot_args(dims, q_weight, k_weight, positions, inv_freq);
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  a.qos = dims->q_out_stride ? dims->q_out_stride : dims->q_heads * dims->head_dim;
  a.kos = dims->k_out_stride ? dims->k_out_stride : dims->k_heads * dims->head_dim;
  const bool vec = rot_vec(dims, es, {q, k, q_out, k_out, q_weight, k_weight}, {a.qs, a.ks, a.qos, a.kos});
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
  RotArgs a = rot_args(dims, q_weight, k_weight, positions, inv_freq);
  const int64_t qw = dims->q_heads * dims->head_dim, kw = dims->k_heads * dims->head_dim;
  a.q = q; a.k = k; a.dqo = dq_out; a.dko = dk_out; a.qo = dq; a.ko = dk;
  a.dqos = dims->dq_out_stride ? dims->dq_out_stride : qw;
  a.dkos = dims->dk_out_stride ? dims->dk_out_stride : kw;
  a.qos = dims->dq_stride ? dims->dq_stride : qw;
  a.kos = dims->dk_stride ? dims->dk_stride : kw;
  a.dwq = d_q_weight; a.dwk = d_k_weight;
  a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + STATUS_BYTES);
  const bool vec = rot_vec(dims, es, {dq_out, dk_out, q, k, dq, dk, q_weight, k_weight}, {a.qs, a.ks, a.dqos, a.dkos, a.qos, a.kos});
  const cudaError_t e = act == M3_BF16 ? rot_launch<__nv_bfloat16, true>(a, vec, dims->interleaved, s)
                                       : rot_launch<float, true>(a, vec, dims->interleaved, s);
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

}  // extern "C"
