// m3_lin_api.cu -- the C entry points of linear attention with a decay for
// each head: validation, the launch plan and the launch sequences.
#include <math.h>

#include <initializer_list>

#include "m3_delta.cuh"  // sm_count
#include "m3_lin.cuh"

namespace m3 {
namespace {

struct LinPlan {
  int B, T, Hk, Hv, DK, DV, share;
  size_t fwd_ws_bytes, ws_bytes;
  size_t o_pdq, o_pdk, o_dstate;  // workspace offsets
  bool tc;                        // the tensor-core kernels
  int nc;
  struct Walk {                   // of the forward (one pass), of the backward (three)
    bool stream;
    int segs, seg_chunks;
    size_t o_start, o_end, o_flags;
  } walk[2];
  int fwd_launches, bwd_launches;
};

m3_status lin_validate(const m3_linattn_dims* d, m3_dtype act) {
  if (!d) return M3_ERR_NULL;
  if (act != M3_F32 && act != M3_BF16) return M3_ERR_UNSUPPORTED;
  if (d->batch < 0 || d->seq_len < 0 || d->k_heads < 1 || d->v_heads < 1) return M3_ERR_DIMS;
  if (d->batch > 65535 || d->seq_len > (int64_t)1 << 30 || d->v_heads > 65535) return M3_ERR_DIMS;
  if (d->batch * d->v_heads > (int64_t)1 << 24) return M3_ERR_DIMS;
  if (d->batch * d->seq_len > (int64_t)1 << 33) return M3_ERR_DIMS;
  if (d->v_heads % d->k_heads != 0) return M3_ERR_UNSUPPORTED;
  if (d->head_k < 8 || d->head_v < 8 || d->head_k > LIN_DMAX || d->head_v > LIN_DMAX || d->head_k % 8 || d->head_v % 8)
    return M3_ERR_UNSUPPORTED;
  if (!isfinite(d->scale)) return M3_ERR_DIMS;
  if (d->reserved != 0) return M3_ERR_DIMS;
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

// Time segments of the tensor-core kernels for few items.  A block per (item,
// segment) takes a unit of time per chunk (1.2 us) and eight to come up and to
// end; with S segments, first the ends of the S - 1 earlier ones are found (0.8
// units per chunk, two more), then a kernel chains them, then all S run.  The
// count with the least total is taken, with at least three chunks per segment.
// 16 heads of 1024 chunks: nine segments, 266 us, where one takes 1200 and eight
// 282; 24 of 128: six, 70, where one takes 163 and seven 87; 12 of 16: five, 26,
// where one takes 30; 48 of 32: three, 46, where one takes 49 and two 54; 72 of
// 64: one, 88, where two take 93.
//
// f32: a block takes 32 columns, so there are four per (item, segment).  A unit
// is 64 tokens of an SM with three blocks at work for each of them, 7.6 us; one
// or two alone take 1.5 and 2.4 units together, the ends half of that.  Training
// passes: 1 x 2000 x 1 head, 32 segments: 76 us, one 692; 1 x 300 x 8, five: 87,
// one 115; 4 x 1000 x 4, eight: 322, one 437; 2 x 512 x 16, one: 281, two 356;
// 8 x 128 x 4, one: 80, two 108.
double lin_cost(int64_t items, int m, int S, bool tc) {
  if (tc) {
    const double all = (double)((items * S + LIN_SMS - 1) / LIN_SMS) * (m + 8.0);
    return S > 1 ? all + (double)((items * (S - 1) + LIN_SMS - 1) / LIN_SMS) * (0.8 * m + 2.0) + 4.0 + 0.3 * S : all;
  }
  auto units = [&](int64_t parts) {
    const int64_t blocks = (4 * parts + LIN_SMS - 1) / LIN_SMS;  // of an SM
    const double rest[3] = {0.0, 1.5, 2.4};
    return (double)(blocks / 3 * 3) + rest[blocks % 3];
  };
  return S > 1 ? 1.03 * (units(items * S) + 0.5 * units(items * (S - 1))) * m + 0.8 + 0.03 * S : units(items) * m;
}
void lin_segments(int64_t items, int nc, bool tc, int* segs, int* seg_chunks) {
  const int least = tc ? 3 : 1;
  double best = 0.0;
  *segs = 1;
  *seg_chunks = nc < 1 ? 1 : nc;
  for (int want = 1; want <= LIN_SMS && want * least <= (nc > least ? nc : least); ++want) {
    const int m = (nc + want - 1) / want;
    if (m < 1) break;
    const int S = (nc + m - 1) / m;
    const double cost = lin_cost(items, m, S, tc);
    if (want == 1 || cost < best - 1e-9) {
      best = cost;
      *segs = S;
      *seg_chunks = m;
    }
  }
}

m3_status lin_plan(const m3_linattn_dims* d, m3_dtype act, LinPlan* p) {
  const m3_status st = lin_validate(d, act);
  if (st != M3_OK) return st;
  p->B = (int)d->batch; p->T = (int)d->seq_len;
  p->Hk = (int)d->k_heads; p->Hv = (int)d->v_heads;
  p->DK = (int)d->head_k; p->DV = (int)d->head_v;
  p->share = p->Hv / p->Hk;
  size_t off = STATUS_BYTES;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  // (one token by the recurrence, without a chunk's latency)
  p->tc = act == M3_BF16 && p->T > 1;
  p->nc = (p->T + LIN_C - 1) / LIN_C;
  if ((int64_t)3 * p->B * p->Hv * p->nc > 0x7FFFFFFF) return M3_ERR_DIMS;  // chunks are counted in 32 bits
  for (int i = 0; i < 2; ++i) {
    LinPlan::Walk& w = p->walk[i];
    const int64_t items = (int64_t)(i ? 3 : 1) * p->B * p->Hv;
    w.segs = 1;
    w.seg_chunks = p->nc;
    w.stream = p->tc && items > LIN_SMS;
    if (!w.stream && p->T > 1) lin_segments(items, p->nc, p->tc, &w.segs, &w.seg_chunks);
    // a block of equal shares hands on one state at most; segments have their starts and their ends
    const size_t slot = (size_t)LIN_DMAX * LIN_DMAX * 4, slots = w.segs > 1 ? (size_t)items * w.segs : 0;
    w.o_start = take((w.stream ? LIN_SMS : slots) * slot);
    w.o_end = take(slots * slot);
    w.o_flags = take(w.stream ? LIN_SMS * 4 : 0);
    if (i == 0) p->fwd_ws_bytes = off > align_up(STATUS_BYTES, 256) ? off : 0;  // (no more than a status block: none at all)
  }
  // the backward's: shares of dq and dk where key heads are shared, and a
  // copy of a state gradient that is to be overwritten
  const size_t part = p->share > 1 ? (size_t)p->B * p->T * p->Hv * p->DK * 4 : 0;
  p->o_pdq = take(part);
  p->o_pdk = take(part);
  p->o_dstate = take((size_t)p->B * p->Hv * p->DK * p->DV * 4);
  p->ws_bytes = off;
  const bool empty = p->B == 0 || p->T == 0;
  p->fwd_launches = empty ? 0 : p->walk[0].segs > 1 ? 3 : 1;
  p->bwd_launches = empty ? 0 : (p->walk[1].segs > 1 ? 3 : 1) + (p->share > 1 ? 1 : 0);
  return M3_OK;
}

LinArgs lin_args(const m3_linattn_dims* d, const LinPlan& p, const float* log_decay) {
  LinArgs a{};
  a.B = p.B; a.T = p.T; a.Hv = p.Hv;
  a.ld = log_decay;
  a.scale = d->scale != 0.0f ? d->scale : 1.0f / sqrtf((float)p.DK);
  return a;
}

int64_t or_dense(int64_t stride, int64_t width) { return stride ? stride : width; }

LinPass lin_fwd_pass(const m3_linattn_dims* d, const LinPlan& p, const void* q, const void* k, const void* v) {
  LinPass r{};
  const int64_t kw = (int64_t)p.Hk * p.DK, vw = (int64_t)p.Hv * p.DV;
  r.q = q; r.k = k; r.v = v;
  r.qs = or_dense(d->q_stride, kw); r.ks = or_dense(d->k_stride, kw); r.vs = or_dense(d->v_stride, vw);
  r.os = vw;
  r.qh = r.kh = p.share;
  r.vh = 1;
  r.DK = p.DK; r.DV = p.DV;
  return r;
}

cudaError_t lin_launch(LinArgs a, const LinPlan& p, m3_dtype act, void* workspace, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  const LinPlan::Walk& w = p.walk[a.np > 1];
  a.status = static_cast<unsigned*>(workspace);
  a.nc = p.nc;
  a.stream = w.stream; a.segs = w.segs; a.seg_chunks = w.seg_chunks;
  if (ws) {
    a.seg_start = reinterpret_cast<float*>(ws + w.o_start);
    a.seg_end = reinterpret_cast<float*>(ws + w.o_end);
    a.flags = reinterpret_cast<unsigned*>(ws + w.o_flags);
  }
  if (p.tc) return launch_lin_tc(a, s, sms);
  return act == M3_BF16 ? launch_lin_rec<__nv_bfloat16>(a, s, sms) : launch_lin_rec<float>(a, s, sms);
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

// (none needed: NULL will do, and one that is given has its status block)
m3_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0 && !ws) return M3_OK;
  if (!ws || bytes < need || bytes < STATUS_BYTES) return M3_ERR_WORKSPACE;
  return aligned(ws, 256) ? M3_OK : M3_ERR_ALIGN;
}

}  // namespace
}  // namespace m3

using namespace m3;

extern "C" {

m3_status m3scan_linattn_plan(const m3_linattn_dims* dims, m3_dtype act, m3_linattn_plan* out) {
  if (!out) return M3_ERR_NULL;
  LinPlan p;
  const m3_status st = lin_plan(dims, act, &p);
  if (st != M3_OK) return st;
  out->workspace_bytes = (int64_t)p.ws_bytes;
  out->fwd_workspace_bytes = (int64_t)p.fwd_ws_bytes;
  out->fwd_launches = p.fwd_launches;
  out->bwd_launches = p.bwd_launches;
  return M3_OK;
}

m3_status m3scan_linattn_fwd(const m3_linattn_dims* dims, m3_dtype act, const void* q, const void* k, const void* v,
                             const float* log_decay, const float* state, void* o, float* state_out,
                             void* workspace, size_t workspace_bytes, m3_stream_t stream) {
  LinPlan p;
  m3_status st = lin_plan(dims, act, &p);
  if (st != M3_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!all_aligned({q, k, v, o, state, state_out}, 16) || !all_aligned({log_decay}, 4)) return M3_ERR_ALIGN;
  if (p.B == 0 || p.T == 0) return pass_state(state, state_out, (size_t)p.B * p.Hv * p.DK * p.DV * 4, s);
  if (!q || !k || !v || !log_decay || !o) return M3_ERR_NULL;
  st = check_workspace(workspace, workspace_bytes, p.fwd_ws_bytes);
  if (st != M3_OK) return st;
  LinArgs a = lin_args(dims, p, log_decay);
  a.np = 1;
  a.p[0] = lin_fwd_pass(dims, p, q, k, v);
  a.p[0].out = o; a.p[0].s_in = state; a.p[0].s_out = state_out;
  return note(lin_launch(a, p, act, workspace, s)) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

m3_status m3scan_linattn_decode(const m3_linattn_dims* dims, m3_dtype act, const void* q, const void* k, const void* v,
                                const float* log_decay, float* state, void* o, m3_stream_t stream) {
  LinPlan p;
  const m3_status st = lin_plan(dims, act, &p);
  if (st != M3_OK) return st;
  if (!all_aligned({q, k, v, o, state}, 16) || !all_aligned({log_decay}, 4)) return M3_ERR_ALIGN;
  if (p.B == 0 || p.T == 0) return M3_OK;
  if (!q || !k || !v || !log_decay || !o || !state) return M3_ERR_NULL;
  LinArgs a = lin_args(dims, p, log_decay);
  a.np = 1;
  a.p[0] = lin_fwd_pass(dims, p, q, k, v);
  a.p[0].out = o; a.p[0].s_in = a.p[0].s_out = state;
  int sms = 0;
  if (note(sm_count(&sms)) != cudaSuccess) return M3_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = act == M3_BF16 ? launch_lin_rec<__nv_bfloat16>(a, s, sms) : launch_lin_rec<float>(a, s, sms);
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

m3_status m3scan_linattn_bwd(const m3_linattn_dims* dims, m3_dtype act, const void* q, const void* k, const void* v,
                             const float* log_decay, const float* state, const void* d_o, const float* d_state_out,
                             void* dq, void* dk, void* dv, float* d_state, void* workspace, size_t workspace_bytes,
                             m3_stream_t stream) {
  LinPlan p;
  m3_status st = lin_plan(dims, act, &p);
  if (st != M3_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!all_aligned({q, k, v, state, d_o, d_state_out, dq, dk, dv, d_state}, 16) || !all_aligned({log_decay}, 4))
    return M3_ERR_ALIGN;
  const size_t sbytes = (size_t)p.B * p.Hv * p.DK * p.DV * 4;
  if (p.B == 0 || p.T == 0) return pass_state(d_state_out, d_state, sbytes, s);
  if (!q || !k || !v || !log_decay || !d_o || !dq || !dk || !dv) return M3_ERR_NULL;
  st = check_workspace(workspace, workspace_bytes, p.ws_bytes);
  if (st != M3_OK) return st;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  if (d_state_out && d_state == d_state_out) {  // two passes start from it, at times of their own
    float* copy = reinterpret_cast<float*>(ws + p.o_dstate);
    if (note(cudaMemcpyAsync(copy, d_state_out, sbytes, cudaMemcpyDeviceToDevice, s)) != cudaSuccess) return M3_ERR_CUDA;
    d_state_out = copy;
  }
  LinArgs a = lin_args(dims, p, log_decay);
  a.np = 3;
  const LinPass f = lin_fwd_pass(dims, p, q, k, v);
  const int64_t kw = (int64_t)p.Hk * p.DK, vw = (int64_t)p.Hv * p.DV, pw = (int64_t)p.Hv * p.DK;
  float* part[2] = {reinterpret_cast<float*>(ws + p.o_pdq), reinterpret_cast<float*>(ws + p.o_pdk)};
  const bool shared = p.share > 1;
  // dk, dv: backwards in time over the same four tensors; dq: in time
  LinPass& pk = a.p[0];
  pk.q = v; pk.qs = f.vs; pk.qh = 1;
  pk.k = d_o; pk.ks = vw; pk.kh = 1;
  pk.v = q; pk.vs = f.qs; pk.vh = p.share;
  pk.DK = p.DV; pk.DV = p.DK;
  pk.rev = true; pk.st = true;
  pk.s_in = d_state_out;
  pk.out = shared ? part[1] : dk;
  pk.os = shared ? pw : or_dense(dims->dk_stride, kw);
  pk.out_f32 = shared || act == M3_F32;
  LinPass& pv = a.p[1];
  pv.q = k; pv.qs = f.ks; pv.qh = p.share;
  pv.k = q; pv.ks = f.qs; pv.kh = p.share;
  pv.v = d_o; pv.vs = vw; pv.vh = 1;
  pv.DK = p.DK; pv.DV = p.DV;
  pv.rev = true;
  pv.s_in = d_state_out; pv.s_out = d_state;
  pv.out = dv; pv.os = or_dense(dims->dv_stride, vw);
  LinPass& pq = a.p[2];
  pq.q = d_o; pq.qs = vw; pq.qh = 1;
  pq.k = v; pq.ks = f.vs; pq.kh = 1;
  pq.v = k; pq.vs = f.ks; pq.vh = p.share;
  pq.DK = p.DV; pq.DV = p.DK;
  pq.st = true;
  pq.s_in = state;
  pq.out = shared ? part[0] : dq;
  pq.os = shared ? pw : or_dense(dims->dq_stride, kw);
  pq.out_f32 = pk.out_f32;
  cudaError_t e = lin_launch(a, p, act, workspace, s);
  if (e == cudaSuccess && shared) {
    LinShare sh{};
    sh.part[0] = part[0]; sh.part[1] = part[1];
    sh.out[0] = dq; sh.out[1] = dk;
    sh.os[0] = or_dense(dims->dq_stride, kw); sh.os[1] = or_dense(dims->dk_stride, kw);
    sh.tokens = (int64_t)p.B * p.T; sh.Hk = p.Hk; sh.share = p.share; sh.D = p.DK;
    e = act == M3_BF16 ? launch_lin_share<__nv_bfloat16>(sh, s) : launch_lin_share<float>(sh, s);
  }
  return note(e) == cudaSuccess ? M3_OK : M3_ERR_CUDA;
}

}  // extern "C"
