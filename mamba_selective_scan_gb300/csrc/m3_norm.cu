// m3_norm.cu -- layer norm over the last dimension, forward and backward,
// with the f32 residual stream of a pre-norm block: kernels, validation and
// the C entry points.
//
//   forward   r = x + residual;  y = (r - mean) rstd w + b
//             mean = sum r / dim,  rstd = 1 / sqrt(sum (r - mean)^2 / dim + eps)
//   backward  xh = (r - mean) rstd,  e = dy w
//             dr = rstd (e - mean(e) - xh mean(e xh)) + d_residual_out
//             d_w = sum_rows dy xh,  d_b = sum_rows dy
//
// Both are bound by HBM: every input is read and every output written once.
// A row is held in registers by W warps (W = 1..16), so the variance is the
// sum of squared deviations from the mean of the same registers, and all
// sums are f32.  The backward's blocks walk rows with a grid stride, each
// thread keeping the weight and bias gradient of its own columns in
// registers; a block's shares are one row of the workspace, and a second
// kernel adds the rows in a fixed order (identical bits on every call).
// Forward of 16384 x 2560 bf16 with its residual stream: 85 us, 89 % of the
// measured copy bandwidth.  Backward of 16384 x 768: 39 us (78 %), then 6.5 us
// for the sums of 912 blocks' shares (608 blocks: 45 us, 1216: 39).

#include <initializer_list>

#include "m3_delta.cuh"

namespace m3 {

constexpr int NORM_W_MAX = 16;        // warps that share a row, at most
constexpr int NORM_DIM_MAX = 16384;   // dim % 8 == 0 and 16-byte aligned rows
constexpr int NORM_DIM_MAX1 = 8192;   // any other dim
constexpr int NORM_BWD_BLOCKS = 912;  // share rows of the backward's workspace (and its blocks), at most

struct NormArgs {
  const void *x, *dy;
  const float *residual, *w, *b, *mean_in, *rstd_in, *d_res_out;
  void *y, *dx;
  float *res_out, *mean, *rstd, *d_res, *part, *dw, *db;
  int64_t rows;
  int dim, wpr, accumulate, nparts;
  float eps;
};

// VEC consecutive elements to and from f32 registers (VEC 1, 4 or 8; the
// vector forms need 16-byte aligned rows)
template <int VEC> __device__ __forceinline__ void ldv(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) v[0] = *p;
  else
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 t = *reinterpret_cast<const float4*>(p + i);
      v[i] = t.x; v[i + 1] = t.y; v[i + 2] = t.z; v[i + 3] = t.w;
    }
}
template <int VEC> __device__ __forceinline__ void ldv(const __nv_bfloat16* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) v[0] = __bfloat162float(*p);
  else {
    __nv_bfloat162 t[VEC / 2];
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(t) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(t) = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float2 f = __bfloat1622float2(t[i]);
      v[2 * i] = f.x; v[2 * i + 1] = f.y;
    }
  }
}
template <int VEC> __device__ __forceinline__ void stv(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) *p = v[0];
  else
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int VEC> __device__ __forceinline__ void stv(__nv_bfloat16* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) *p = __float2bfloat16_rn(v[0]);
  else {
    __nv_bfloat162 t[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) t[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(t);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(t);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
// Sum over the W warps of a row (every thread of the block calls it; `slot`
// alternates so that one barrier a call is enough).
__device__ __forceinline__ float row_sum(float v, float (*sh)[32], int slot, int warp, int lane, int W) {
  v = warp_sum(v);
  if (W == 1) return v;
  if (lane == 0) sh[slot][warp] = v;
  __syncthreads();
  const int base = warp / W * W;
  float s = 0.0f;
  for (int i = 0; i < W; ++i) s += sh[slot][base + i];
  return s;
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(512) m3_norm_fwd_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float sh[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = a.wpr, R = (blockDim.x >> 5) / W;
  const int64_t row = (int64_t)blockIdx.x * R + warp / W;
  const bool live = row < a.rows;
  const int c0 = ((warp % W) * 32 + lane) * VEC, step = W * 32 * VEC;
  const size_t base = (size_t)(live ? row : 0) * a.dim;
  float v[NV][VEC];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * step;
    if (live && c < a.dim) {
      ldv<VEC>(static_cast<const T*>(a.x) + base + c, v[i]);
      if (a.residual) {
        float r[VEC];
        ldv<VEC>(a.residual + base + c, r);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) s += v[i][j];
  }
  const float inv = 1.0f / (float)a.dim;
  const float mean = row_sum(s, sh, 0, warp, lane, W) * inv;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * step;
    if (live && c < a.dim) {
      if (a.res_out) stv<VEC>(a.res_out + base + c, v[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] -= mean;
        q = fmaf(v[i][j], v[i][j], q);
      }
    }
  }
  const float rstd = rsqrtf(row_sum(q, sh, 1, warp, lane, W) * inv + a.eps);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * step;
    if (c < a.dim) {
      float w[VEC], b[VEC];
      ldv<VEC>(a.w + c, w);
      if (a.b) ldv<VEC>(a.b + c, b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = fmaf(v[i][j] * rstd, w[j], a.b ? b[j] : 0.0f);
      stv<VEC>(static_cast<T*>(a.y) + base + c, v[i]);
    }
  }
  if (warp % W == 0 && lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// X: the type of the normalised input (the activation dtype, or f32 for the
// residual stream).
template <typename T, typename X, int VEC, int NV>
__global__ void __launch_bounds__(512) m3_norm_bwd_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ float comb[];  // [R][2][dim] when R > 1
  __shared__ float sh[4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = a.wpr, R = (blockDim.x >> 5) / W;
  const int c0 = ((warp % W) * 32 + lane) * VEC, step = W * 32 * VEC;
  float dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.0f;
  const float inv = 1.0f / (float)a.dim;
  int slot = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.rows; r0 += (int64_t)gridDim.x * R) {
    const int64_t row = r0 + warp / W;
    const bool live = row < a.rows;
    const size_t base = (size_t)(live ? row : 0) * a.dim;
    const float mean = live ? a.mean_in[row] : 0.0f, rstd = live ? a.rstd_in[row] : 0.0f;
    float xh[NV][VEC], e[NV][VEC], up[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (live && c < a.dim) {
        ldv<VEC>(static_cast<const X*>(a.x) + base + c, xh[i]);
        ldv<VEC>(static_cast<const T*>(a.dy) + base + c, e[i]);
        if (a.d_res_out) ldv<VEC>(a.d_res_out + base + c, up[i]);
      }
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (live && c < a.dim) {
        float w[VEC];
        ldv<VEC>(a.w + c, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = (xh[i][j] - mean) * rstd;
          xh[i][j] = h;
          dw[i][j] = fmaf(e[i][j], h, dw[i][j]);
          db[i][j] += e[i][j];
          const float g = e[i][j] * w[j];
          e[i][j] = g;
          s1 += g;
          s2 = fmaf(g, h, s2);
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (W > 1) {
      if (lane == 0) {
        sh[slot][warp] = s1;
        sh[slot + 1][warp] = s2;
      }
      __syncthreads();
      const int b0 = warp / W * W;
      s1 = s2 = 0.0f;
      for (int i = 0; i < W; ++i) {
        s1 += sh[slot][b0 + i];
        s2 += sh[slot + 1][b0 + i];
      }
      slot ^= 2;
    }
    s1 *= inv;
    s2 *= inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (live && c < a.dim) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float g = rstd * (e[i][j] - s1 - xh[i][j] * s2);
          e[i][j] = a.d_res_out ? g + up[i][j] : g;
        }
        stv<VEC>(static_cast<T*>(a.dx) + base + c, e[i]);
        if (a.d_res) stv<VEC>(a.d_res + base + c, e[i]);
      }
    }
  }
  grid_dep_trigger();
  // this block's share of the weight and bias gradients: one row [2][dim]
  float* out = a.part + (size_t)blockIdx.x * 2 * a.dim;
  if (R == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (c < a.dim) {
        stv<VEC>(out + c, dw[i]);
        stv<VEC>(out + a.dim + c, db[i]);
      }
    }
    return;
  }
  float* mine = comb + (size_t)(warp / W) * 2 * a.dim;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * step;
    if (c < a.dim) {
      stv<VEC>(mine + c, dw[i]);
      stv<VEC>(mine + a.dim + c, db[i]);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.dim; c += blockDim.x) {
    float s = 0.0f;
    for (int r = 0; r < R; ++r) s += comb[(size_t)r * 2 * a.dim + c];
    out[c] = s;
  }
}

// d_weight and d_bias: the shares [nparts][2][dim] added over nparts, 32
// columns per block, the rows over 32 warps and a fixed tree over the warps.
__global__ void __launch_bounds__(1024) m3_norm_wgrad_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float sh[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane, n2 = 2 * a.dim;
  grid_dep_wait();
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < n2) {
    int r = warp;
    for (; r + 96 < a.nparts; r += 128)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += a.part[(size_t)(r + 32 * i) * n2 + c];
    for (; r < a.nparts; r += 32) s[0] += a.part[(size_t)r * n2 + c];
  }
  sh[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  const float t = warp_sum(sh[lane][warp]);  // column blockIdx.x * 32 + warp
  const int cc = blockIdx.x * 32 + warp;
  if (lane == 0 && cc < n2) {
    float* o = cc < a.dim ? a.dw : a.db;
    if (o) {
      o += cc < a.dim ? cc : cc - a.dim;
      *o = a.accumulate ? *o + t : t;
    }
  }
}

namespace {

// Warps per row and vectors per thread: the fewest warps whose threads hold
// the row in at most `nv_max` vectors each (fewer warps need fewer barriers).
bool norm_shape(int dim, int vec, int nv_max, int* wpr, int* nv) {
  const int nvec = dim / vec;
  for (int w = 1; w <= NORM_W_MAX; w *= 2) {
    const int n = (nvec + w * 32 - 1) / (w * 32);
    if (n <= nv_max) {
      *wpr = w;
      *nv = n < 1 ? 1 : n;
      return true;
    }
  }
  return false;
}

m3_status norm_validate(const m3_norm_dims* d, m3_dtype act) {
  if (!d) return M3_ERR_NULL;
  if (act != M3_F32 && act != M3_BF16) return M3_ERR_UNSUPPORTED;
  if (d->rows < 0 || d->dim < 0 || d->rows > ((int64_t)1 << 31) - 1 || !(d->eps >= 0.0f)) return M3_ERR_DIMS;
  if (d->accumulate_param_grads != 0 && d->accumulate_param_grads != 1) return M3_ERR_DIMS;
  if (d->dim > (d->dim % 8 ? NORM_DIM_MAX1 : NORM_DIM_MAX)) return M3_ERR_UNSUPPORTED;
  return M3_OK;
}

template <typename T, int VEC>
cudaError_t fwd_nv(const NormArgs& a, int nv, dim3 grid, unsigned block, cudaStream_t s) {
  switch (nv) {
    case 1: m3_norm_fwd_kernel<T, VEC, 1><<<grid, block, 0, s>>>(a); break;
    case 2: m3_norm_fwd_kernel<T, VEC, 2><<<grid, block, 0, s>>>(a); break;
    case 3: m3_norm_fwd_kernel<T, VEC, 3><<<grid, block, 0, s>>>(a); break;
    case 4: m3_norm_fwd_kernel<T, VEC, 4><<<grid, block, 0, s>>>(a); break;
    default:
      if constexpr (VEC == 8) return cudaErrorInvalidValue;  // 16 warps x 4 vectors hold every dim
      else if (nv <= 8) m3_norm_fwd_kernel<T, VEC, 8><<<grid, block, 0, s>>>(a);
      else if (VEC == 1 && nv <= 16) m3_norm_fwd_kernel<T, 1, 16><<<grid, block, 0, s>>>(a);
      else return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_norm_fwd(NormArgs a, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  int nv = 0;
  bool ok;
  if (vec) {
    ok = norm_shape(a.dim, V, 4, &a.wpr, &nv) || norm_shape(a.dim, V, 8, &a.wpr, &nv);
  } else {
    ok = norm_shape(a.dim, 1, 4, &a.wpr, &nv) || norm_shape(a.dim, 1, 8, &a.wpr, &nv) ||
         norm_shape(a.dim, 1, 16, &a.wpr, &nv);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int R = a.wpr >= 4 ? 1 : 4 / a.wpr;
  const unsigned block = 32 * a.wpr * R;
  const dim3 grid((unsigned)((a.rows + R - 1) / R));
  return vec ? fwd_nv<T, V>(a, nv, grid, block, s) : fwd_nv<T, 1>(a, nv, grid, block, s);
}

template <typename T, typename X, int VEC>
void (*bwd_kernel_nv(int nv))(const NormArgs) {
  if constexpr (VEC == 1) {
    if (nv == 4) return m3_norm_bwd_kernel<T, X, 1, 4>;
    if (nv == 8) return m3_norm_bwd_kernel<T, X, 1, 8>;
    return m3_norm_bwd_kernel<T, X, 1, 16>;
  } else {
    if (nv == 1) return m3_norm_bwd_kernel<T, X, VEC, 1>;
    if (nv == 2) return m3_norm_bwd_kernel<T, X, VEC, 2>;
    if (nv == 4) return m3_norm_bwd_kernel<T, X, VEC, 4>;
    return m3_norm_bwd_kernel<T, X, VEC, 8>;
  }
}

template <typename T, typename X>
cudaError_t launch_norm_bwd(NormArgs a, bool vec, cudaStream_t s) {
  // 16-byte rows: the fewest vectors per thread, in as many warps as that
  // takes (a thread keeps five values for each column: 16384 x 768 bf16 with
  // its residual stream runs in 39 us with 6 warps x 1 vector, 47 us with 2 x
  // 3).  Others: four columns per thread (4099 x 1003 f32: 16 us with 8 warps
  // x 4, 25 us with 16 x 2, whose rows have too few loads in flight)
  int nv = 0, sms = 0, occ = 0;
  const int nvec = a.dim / (vec ? 4 : 1);
  for (int n : {vec ? 1 : 4, vec ? 2 : 8, vec ? 4 : 16, 8})
    if (!nv && nvec <= NORM_W_MAX * 32 * n) nv = n;
  if (!nv) return cudaErrorInvalidValue;
  a.wpr = (nvec + 32 * nv - 1) / (32 * nv);
  if (a.wpr < 1) a.wpr = 1;
  const int R = a.wpr >= 8 ? 1 : 8 / a.wpr;
  const unsigned block = 32 * a.wpr * R;
  // R > 1: at most 8 / W rows of W * 32 * 4 columns (one vector per thread), 8 KB of shares
  const size_t smem = R > 1 ? (size_t)R * 2 * a.dim * 4 : 0;
  auto kern = vec ? bwd_kernel_nv<T, X, 4>(nv) : bwd_kernel_nv<T, X, 1>(nv);
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, (int)block, smem);
  if (e != cudaSuccess) return e;
  int64_t grid = (int64_t)sms * (occ < 1 ? 1 : occ);
  const int64_t need = (a.rows + R - 1) / R;
  if (grid > need) grid = need;
  if (grid > NORM_BWD_BLOCKS) grid = NORM_BWD_BLOCKS;
  a.nparts = (int)grid;
  e = launch_k(kern, dim3((unsigned)grid), block, smem, s, false, a);
  if (e != cudaSuccess) return e;
  return launch_k(m3_norm_wgrad_kernel, dim3((unsigned)((2 * a.dim + 31) / 32)), 1024, 0, s, true, a);
}

// 16-byte vectors: every row of every array starts on a 16-byte boundary
bool norm_vec(const m3_norm_dims* d, std::initializer_list<const void*> ptrs) {
  if (d->dim % 8) return false;
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return false;
  return true;
}

int64_t norm_parts(const m3_norm_dims* d) { return d->rows < NORM_BWD_BLOCKS ? d->rows : NORM_BWD_BLOCKS; }

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

m3_status m3scan_norm_plan(const m3_norm_dims* dims, m3_dtype act, m3_norm_plan* out) {
  const m3_status st = norm_validate(dims, act);
  if (st != M3_OK) return st;
  if (!out) return M3_ERR_NULL;
  out->workspace_bytes = STATUS_BYTES + norm_parts(dims) * 2 * dims->dim * 4;
  return M3_OK;
}

m3_status m3scan_norm_fwd(const m3_norm_dims* dims, m3_dtype act, const void* x, const float* residual,
                          const float* weight, const float* bias, void* y, float* residual_out,
                          float* mean, float* rstd, m3_stream_t stream) {
  const m3_status st = norm_validate(dims, act);
  if (st != M3_OK) return st;
  if (dims->rows == 0 || dims->dim == 0) return M3_OK;
  if (!x || !weight || !y) return M3_ERR_NULL;
  const size_t ea = act == M3_BF16 ? 2 : 4;
  if (!aligned(x, ea) || !aligned(y, ea)) return M3_ERR_ALIGN;
  for (const void* p : {(const void*)residual, (const void*)weight, (const void*)bias,
                        (const void*)residual_out, (const void*)mean, (const void*)rstd})
    if (!aligned(p, 4)) return M3_ERR_ALIGN;
  const bool vec = norm_vec(dims, {x, residual, weight, bias, y, residual_out});
  if (!vec && dims->dim > NORM_DIM_MAX1) return M3_ERR_ALIGN;
  NormArgs a{};
  a.x = x; a.residual = residual; a.w = weight; a.b = bias; a.y = y; a.res_out = residual_out;
  a.mean = mean; a.rstd = rstd; a.rows = dims->rows; a.dim = (int)dims->dim; a.eps = dims->eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = act == M3_BF16 ? launch_norm_fwd<__nv_bfloat16>(a, vec, s) : launch_norm_fwd<float>(a, vec, s);
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

m3_status m3scan_norm_bwd(const m3_norm_dims* dims, m3_dtype act, const void* dy, const void* normed,
                          m3_dtype normed_dtype, const float* weight, const float* mean,
                          const float* rstd, const float* d_residual_out, void* dx, float* d_residual,
                          float* d_weight, float* d_bias, void* workspace, size_t workspace_bytes,
                          m3_stream_t stream) {
  m3_status st = norm_validate(dims, act);
  if (st != M3_OK) return st;
  if (normed_dtype != act && normed_dtype != M3_F32) return M3_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dims->dim == 0) return M3_OK;
  if (dims->rows == 0) {  // no rows: zero sums
    if (!dims->accumulate_param_grads)
      for (float* g : {d_weight, d_bias})
        if (g && note(cudaMemsetAsync(g, 0, (size_t)dims->dim * 4, s)) != cudaSuccess) return M3_ERR_CUDA;
    return M3_OK;
  }
  if (!dy || !normed || !weight || !mean || !rstd || !dx) return M3_ERR_NULL;
  const size_t ea = act == M3_BF16 ? 2 : 4;
  if (!aligned(dy, ea) || !aligned(dx, ea) || !aligned(normed, normed_dtype == M3_BF16 ? 2 : 4)) return M3_ERR_ALIGN;
  for (const void* p : {(const void*)weight, (const void*)mean, (const void*)rstd, (const void*)d_residual_out,
                        (const void*)d_residual, (const void*)d_weight, (const void*)d_bias})
    if (!aligned(p, 4)) return M3_ERR_ALIGN;
  const bool vec = norm_vec(dims, {dy, normed, weight, d_residual_out, dx, d_residual});
  if (!vec && dims->dim > NORM_DIM_MAX1) return M3_ERR_ALIGN;
  m3_norm_plan pl;
  m3scan_norm_plan(dims, act, &pl);
  if (!workspace || (int64_t)workspace_bytes < pl.workspace_bytes) return M3_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return M3_ERR_ALIGN;
  NormArgs a{};
  a.dy = dy; a.x = normed; a.w = weight; a.mean_in = mean; a.rstd_in = rstd; a.d_res_out = d_residual_out;
  a.dx = dx; a.d_res = d_residual; a.dw = d_weight; a.db = d_bias;
  a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + STATUS_BYTES);
  a.rows = dims->rows; a.dim = (int)dims->dim; a.accumulate = dims->accumulate_param_grads;
  cudaError_t e;
  if (act == M3_F32) e = launch_norm_bwd<float, float>(a, vec, s);
  else if (normed_dtype == M3_F32) e = launch_norm_bwd<__nv_bfloat16, float>(a, vec, s);
  else e = launch_norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

}  // extern "C"
