// m3_delta_api.cu -- the C entry points of the gated delta rule: validation,
// the launch plan and the launch sequences.
#include <math.h>

#include <atomic>
#include <initializer_list>

#include "m3_delta.cuh"

namespace m3 {

cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev >= 0 && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

namespace {

m3_status delta_validate(const m3_delta_dims* d, m3_dtype act) {
  if (!d) return M3_ERR_NULL;
  if (act != M3_F32 && act != M3_BF16) return M3_ERR_UNSUPPORTED;
  if (d->batch < 0 || d->seq_len < 0 || d->k_heads < 1 || d->v_heads < 1) return M3_ERR_DIMS;
  if (d->batch > 65535 || d->seq_len > (int64_t)1 << 30 || d->v_heads > 65535) return M3_ERR_DIMS;
  if (d->batch * d->v_heads > (int64_t)1 << 24) return M3_ERR_DIMS;
  if (d->batch * d->seq_len > (int64_t)1 << 33) return M3_ERR_DIMS;
  if (d->v_heads % d->k_heads != 0) return M3_ERR_UNSUPPORTED;
  if (d->head_k < 8 || d->head_v < 8 || d->head_k > DMAX || d->head_v > DMAX || d->head_k % 8 || d->head_v % 8)
    return M3_ERR_UNSUPPORTED;
  if (!isfinite(d->scale)) return M3_ERR_DIMS;
  if (d->qk_l2norm != 0 && d->qk_l2norm != 1) return M3_ERR_DIMS;
  const int es = act == M3_BF16 ? 2 : 4;
  const int64_t kw = d->k_heads * d->head_k, vw = d->v_heads * d->head_v;
  const struct { int64_t stride, width; } rows[] = {{d->q_stride, kw}, {d->k_stride, kw}, {d->v_stride, vw},
                                                    {d->dq_stride, kw}, {d->dk_stride, kw}, {d->dv_stride, vw}};
  for (const auto& r : rows) {
    if (r.stride != 0 && (r.stride < r.width || r.stride > (int64_t)1 << 24)) return M3_ERR_DIMS;
    if (r.stride * es % 16 != 0) return M3_ERR_ALIGN;
  }
  return M3_OK;
}

// Time segments of the tensor-core chains.  A block per (head, segment) runs
// one chunk in a unit of time (2.8 us in the forward); with S segments, first
// the effect of the S - 1 earlier ones is found (1.1 units per chunk), then a
// kernel chains them (eight blocks per head, 1.1 units per segment), then all
// S run; the two extra launches and their first loads are three units.  The
// count with the least total is taken, with at least four chunks per segment.
// 1 x 65536 x 16 heads: 19 segments, 0.88 ms, where one would take 1024
// chunks one after the other, some 3 ms; 36 heads of 24 chunks: four segments,
// forward and backward 94 and 129 us against 107 and 155 in one.
void delta_segments(int64_t heads, int nc, int* segs, int* seg_chunks) {
  constexpr int64_t SMS = 152;
  double best = 0.0;
  *segs = 1;
  *seg_chunks = nc < 1 ? 1 : nc;
  for (int want = 1; want <= 64 && want * 4 <= (nc > 4 ? nc : 4); ++want) {
    const int m = (nc + want - 1) / want;
    if (m < 1) break;
    const int S = (nc + m - 1) / m;
    const double fin = (double)((heads * S + SMS - 1) / SMS) * m;
    const double agg = S > 1 ? (double)((heads * (S - 1) + SMS - 1) / SMS) * m * 1.1 +
                                     (double)((heads * 8 + SMS - 1) / SMS) * (S - 1) * 1.1 + 3.0 : 0.0;
    if (want == 1 || fin + agg < best - 1e-9) {
      best = fin + agg;
      *segs = S;
      *seg_chunks = m;
    }
  }
}

m3_status delta_plan(const m3_delta_dims* d, m3_dtype act, DeltaPlan* p) {
  const m3_status st = delta_validate(d, act);
  if (st != M3_OK) return st;
  p->B = (int)d->batch; p->T = (int)d->seq_len;
  p->Hk = (int)d->k_heads; p->Hv = (int)d->v_heads;
  p->DK = (int)d->head_k; p->DV = (int)d->head_v;
  const bool tc = act == M3_BF16;  // the tensor-core kernels
  p->chunk = tc ? 64 : 32;
  p->nc = (p->T + p->chunk - 1) / p->chunk;
  const size_t chunks = (size_t)p->B * p->Hv * p->nc;
  if (chunks > 0x7FFFFFFF) return M3_ERR_DIMS;  // one block each
  p->ckpt_bytes = chunks * (tc ? TC_CKPT : (size_t)p->DK * p->DV * 4);
  size_t off = STATUS_BYTES;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  p->segs = 1;
  p->seg_chunks = p->nc;
  // more heads than SMs: equal shares of all chunks, a block per SM
  const int64_t heads = (int64_t)p->B * p->Hv;
  p->stream = tc && heads > 152 && p->nc > 0;
  if (tc && !p->stream) delta_segments(heads, p->nc, &p->segs, &p->seg_chunks);
  const size_t seg_bytes = p->segs > 1 ? (size_t)p->B * p->Hv * p->segs * DMAX * DMAX * 4 : 0;
  p->o_keep = p->ckpt_bytes;  // the segments' transitions, behind the chunks' checkpoints
  p->ckpt_bytes += seg_bytes;
  p->o_end = take(seg_bytes);
  p->o_phi = take(seg_bytes);
  p->o_start = take(p->stream ? (size_t)heads * DMAX * DMAX * 4 : seg_bytes);
  p->o_flags = take(p->stream ? (size_t)heads * 4 : 0);
  // T, P and factors of a forward without checkpoints; what the backward
  // keeps takes their place
  const size_t mark = off;
  p->o_tp = take(tc ? chunks * TC_PREP : 0);
  p->fwd_ws_bytes = off;
  off = mark;
  p->o_bwd = take(chunks * (tc ? TC_BWD : F32_KEPT));
  const bool shared = p->Hv != p->Hk;
  const size_t share_bytes = shared && !tc ? (size_t)p->B * p->T * p->Hv * p->DK * 4 : 0;
  p->o_pdq = take(share_bytes);
  p->o_pdk = take(share_bytes);
  p->ws_bytes = off > p->fwd_ws_bytes ? off : p->fwd_ws_bytes;
  const bool empty = p->B == 0 || p->T == 0;
  const int walk = p->segs > 1 ? 3 : 1;  // (shares: and a memset of their flags)
  p->fwd_launches = empty ? 0 : walk + (tc ? 1 : 0);
  p->bwd_launches = empty ? 0 : tc ? walk + 1 : shared ? 4 : 3;
  return M3_OK;
}

DeltaArgs delta_args(const m3_delta_dims* d, const DeltaPlan& p) {
  DeltaArgs a{};
  a.B = p.B; a.T = p.T; a.Hk = p.Hk; a.Hv = p.Hv; a.DK = p.DK; a.DV = p.DV;
  a.share = p.Hv / p.Hk;
  a.chunk = p.chunk; a.nc = p.nc;
  const int64_t kw = (int64_t)p.Hk * p.DK, vw = (int64_t)p.Hv * p.DV;
  a.qs = d->q_stride ? d->q_stride : kw;
  a.ks = d->k_stride ? d->k_stride : kw;
  a.vs = d->v_stride ? d->v_stride : vw;
  a.dqs = d->dq_stride ? d->dq_stride : kw;
  a.dks = d->dk_stride ? d->dk_stride : kw;
  a.dvs = d->dv_stride ? d->dv_stride : vw;
  a.scale = d->scale != 0.0f ? d->scale : 1.0f / sqrtf((float)p.DK);
  a.l2 = d->qk_l2norm;
  return a;
}

// The workspace's parts
void delta_ws(DeltaArgs& a, const DeltaPlan& p, void* workspace) {
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.status = static_cast<unsigned*>(workspace);
  a.pdq = reinterpret_cast<float*>(ws + p.o_pdq);
  a.pdk = reinterpret_cast<float*>(ws + p.o_pdk);
  a.stream = p.stream;
  a.flags = reinterpret_cast<unsigned*>(ws + p.o_flags);
  a.segs = p.segs; a.seg_chunks = p.seg_chunks;
  a.seg_end = reinterpret_cast<float*>(ws + p.o_end);
  a.seg_phi = reinterpret_cast<float*>(ws + p.o_phi);
  a.seg_start = reinterpret_cast<float*>(ws + p.o_start);
  a.bwd = ws + p.o_bwd;
  // in the checkpoints, where there are some
  const void* ck = a.ckpt ? a.ckpt : a.ckpt_in;
  a.tp = ck ? static_cast<unsigned char*>(const_cast<void*>(ck)) + 65536 : ws + p.o_tp;
  a.tp_stride = ck ? TC_CKPT : TC_PREP;
  a.seg_keep = ck ? reinterpret_cast<float*>(static_cast<unsigned char*>(const_cast<void*>(ck)) + p.o_keep) : nullptr;
}

// `aligned` for a list; NULL passes (presence is checked apart)
bool all_aligned(std::initializer_list<const void*> ptrs, size_t n) {
  for (const void* q : ptrs)
    if (q && !aligned(q, n)) return false;
  return true;
}

// No tokens: the state passes through (zero where there is none)
m3_status pass_state(const float* in, float* out, size_t bytes, cudaStream_t s) {
  if (!out || bytes == 0 || in == out) return M3_OK;
  const cudaError_t e = in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, s)
                           : cudaMemsetAsync(out, 0, bytes, s);
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

m3_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need) return M3_ERR_WORKSPACE;
  return aligned(ws, 256) ? M3_OK : M3_ERR_ALIGN;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

m3_status m3scan_delta_plan(const m3_delta_dims* dims, m3_dtype act, m3_delta_plan* out) {
  if (!out) return M3_ERR_NULL;
  DeltaPlan p;
  const m3_status st = delta_plan(dims, act, &p);
  if (st != M3_OK) return st;
  out->chunk = p.chunk;
  out->n_chunks = p.nc;
  out->ckpt_bytes = (int64_t)p.ckpt_bytes;
  out->workspace_bytes = (int64_t)p.ws_bytes;
  out->fwd_workspace_bytes = (int64_t)p.fwd_ws_bytes;
  out->fwd_launches = p.fwd_launches;
  out->bwd_launches = p.bwd_launches;
  return M3_OK;
}

m3_status m3scan_delta_fwd(const m3_delta_dims* dims, m3_dtype act, const void* q, const void* k,
                           const void* v, const void* g, const void* beta, const float* state,
                           void* o, float* state_out, float* ckpt, void* workspace,
                           size_t workspace_bytes, m3_stream_t stream) {
  DeltaPlan p;
  m3_status st = delta_plan(dims, act, &p);
  if (st != M3_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!all_aligned({q, k, v, o, state, state_out, ckpt}, 16) || !all_aligned({g, beta}, act == M3_BF16 ? 2 : 4))
    return M3_ERR_ALIGN;
  if (p.B == 0 || p.T == 0)
    return pass_state(state, state_out, (size_t)p.B * p.Hv * p.DK * p.DV * 4, s);
  if (!q || !k || !v || !g || !beta || !o) return M3_ERR_NULL;
  st = check_workspace(workspace, workspace_bytes, p.fwd_ws_bytes);
  if (st != M3_OK) return st;
  int sms = 0;
  if (note(sm_count(&sms)) != cudaSuccess) return M3_ERR_CUDA;
  DeltaArgs a = delta_args(dims, p);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.s_in = state;
  a.o = o; a.s_out = state_out; a.ckpt = ckpt;
  delta_ws(a, p, workspace);
  cudaError_t e;
  if (act == M3_BF16) {
    e = launch_delta_tc_prep(a, s);
    if (e == cudaSuccess) e = launch_delta_tc_fwd(a, s);
  } else {
    e = launch_delta_rec<float>(a, s, sms);
  }
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

m3_status m3scan_delta_decode(const m3_delta_dims* dims, m3_dtype act, const void* q, const void* k,
                              const void* v, const void* g, const void* beta, float* state, void* o,
                              m3_stream_t stream) {
  DeltaPlan p;
  m3_status st = delta_plan(dims, act, &p);
  if (st != M3_OK) return st;
  if (!all_aligned({q, k, v, o, state}, 16) || !all_aligned({g, beta}, act == M3_BF16 ? 2 : 4)) return M3_ERR_ALIGN;
  if (p.B == 0 || p.T == 0) return M3_OK;
  if (!q || !k || !v || !g || !beta || !o || !state) return M3_ERR_NULL;
  int sms = 0;
  if (note(sm_count(&sms)) != cudaSuccess) return M3_ERR_CUDA;
  DeltaArgs a = delta_args(dims, p);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.s_in = state; a.s_out = state; a.o = o;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = act == M3_BF16 ? launch_delta_rec<__nv_bfloat16>(a, s, sms) : launch_delta_rec<float>(a, s, sms);
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

m3_status m3scan_delta_bwd(const m3_delta_dims* dims, m3_dtype act, const void* q, const void* k,
                           const void* v, const void* g, const void* beta, const float* ckpt,
                           const void* d_o, const float* d_state_out, void* dq, void* dk, void* dv,
                           void* dg, void* dbeta, float* d_state, void* workspace,
                           size_t workspace_bytes, m3_stream_t stream) {
  DeltaPlan p;
  m3_status st = delta_plan(dims, act, &p);
  if (st != M3_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!all_aligned({q, k, v, ckpt, d_o, d_state_out, dq, dk, dv, d_state}, 16) ||
      !all_aligned({g, beta, dg, dbeta}, act == M3_BF16 ? 2 : 4))
    return M3_ERR_ALIGN;
  if (p.B == 0 || p.T == 0)
    return pass_state(d_state_out, d_state, (size_t)p.B * p.Hv * p.DK * p.DV * 4, s);
  if (!q || !k || !v || !g || !beta || !ckpt || !d_o || !dq || !dk || !dv || !dg || !dbeta) return M3_ERR_NULL;
  st = check_workspace(workspace, workspace_bytes, p.ws_bytes);
  if (st != M3_OK) return st;
  DeltaArgs a = delta_args(dims, p);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.ckpt_in = ckpt; a.d_o = d_o; a.ds_out = d_state_out;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.ds_in = d_state;
  delta_ws(a, p, workspace);
  cudaError_t e;
  if (act == M3_BF16) {
    e = launch_delta_tc_rev(a, s);
    if (e == cudaSuccess) e = launch_delta_tc_grad(a, s);
  } else {
    e = launch_delta_bwd(a, s);
    if (e == cudaSuccess && a.share > 1) e = launch_delta_share(a, s);
  }
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

}  // extern "C"
