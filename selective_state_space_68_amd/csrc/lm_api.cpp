// C-ABI host layer of the linear attention and block norm entry points: argument
// validation, aliasing checks and dispatch to the gfx950 kernels on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/ssm.h"
#include "host_common.hpp"
#include "lm_kernels.hpp"

namespace {

using ssm::aligned;
using ssm::from_hip;
using ssm::mul_ok;
using ssm::overlaps;
using ssm::probe_device;
using ssm::Span;
using ssm::span;

constexpr uint64_t kMaxBytes = uint64_t(1) << 62;
constexpr int64_t kMaxL = int64_t(1) << 30;
constexpr int64_t kMaxPairs = int64_t(1) << 20;      // batch * H of the prompt form
constexpr int64_t kMaxHeads = int64_t(1) << 16;      // (64 rows of the output span less than 2^32 bytes)
constexpr int64_t kMaxTokenStride = int64_t(1) << 23;  // ... and 64 rows of an input that moves as vectors
constexpr int64_t kMaxStepPairs = int64_t(1) << 22;  // batch * H of the step
constexpr int64_t kMaxRows = int64_t(1) << 22;

uint64_t up256(uint64_t n) { return (n + 255) / 256 * 256; }

// Bytes of a packed array of `n` factors and an element size; false on overflow.
template <typename... N>
bool bytes_of(uint64_t elem, uint64_t* out, N... n) {
  uint64_t t = elem;
  const int64_t sizes[] = {static_cast<int64_t>(n)...};
  for (const int64_t x : sizes)
    if (!mul_ok(t, static_cast<uint64_t>(x), &t)) return false;
  *out = t;
  return t <= kMaxBytes;
}

// A tensor of DIMS strided axes and a contiguous last one.
template <int DIMS>
struct View {
  int64_t stride[3] = {};
  uint64_t extent = 0;       // bytes from its first element to past its last
  bool empty = true;
};

// Fills *v from the caller's strides (or packed ones); false for a negative stride or overflow.
template <int DIMS>
bool make_view(const int64_t* strides, const int64_t (&n)[DIMS], int64_t width, uint64_t elem, View<DIMS>* v) {
  int64_t packed = width;
  v->empty = width == 0;
  for (int i = DIMS - 1; i >= 0; --i) {
    v->stride[i] = strides ? strides[i] : packed;
    if (v->stride[i] < 0 || __builtin_mul_overflow(packed, n[i], &packed)) return false;
    if (n[i] == 0) v->empty = true;
  }
  if (v->empty) return true;
  uint64_t last = static_cast<uint64_t>(width);
  for (int i = 0; i < DIMS; ++i) {
    uint64_t t;
    if (!mul_ok(static_cast<uint64_t>(v->stride[i]), static_cast<uint64_t>(n[i] - 1), &t) ||
        __builtin_add_overflow(last, t, &last))
      return false;
  }
  return mul_ok(last, elem, &v->extent) && v->extent <= kMaxBytes;
}

// Whether every row of the tensor starts at a multiple of `unit` bytes.
template <int DIMS>
bool rows_aligned(const void* p, const View<DIMS>& v, uint64_t elem, uint64_t unit) {
  if (!aligned(p, unit)) return false;
  for (int i = 0; i < DIMS; ++i)
    if (static_cast<uint64_t>(v.stride[i]) * elem % unit) return false;
  return true;
}

// Bytes in which `width` elements of every row can move (16, with the rows of a tile near enough; 4; or 0: an element).
int row_move(const void* p, const View<3>& v, int64_t width, uint64_t elem) {
  const uint64_t bytes = static_cast<uint64_t>(width) * elem;
  if (width % 8 == 0 && v.stride[1] <= kMaxTokenStride && rows_aligned(p, v, elem, 16)) return 16;
  return bytes % 4 == 0 && rows_aligned(p, v, elem, 4) ? 4 : 0;
}

int least(int a, int b) { return a < b ? a : b; }

bool any_overlap(const Span* outs, int n_out, const Span* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlaps(outs[i], ins[j])) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

bool dtype_ok(ssm_dtype dt) { return dt == SSM_F32 || dt == SSM_BF16; }
ssm::Dt dt_of(ssm_dtype dt) { return dt == SSM_BF16 ? ssm::Dt::BF16 : ssm::Dt::F32; }

// Sizes of a linear attention call (L: 1 for the step).
ssm_status check_la_sizes(int64_t batch, int64_t L, int64_t H, int64_t Hq, int64_t Hk, int64_t Hv, int64_t K, int64_t V,
                          int64_t max_pairs, ssm_dtype dt) {
  if (!dtype_ok(dt)) return SSM_ERR_UNSUPPORTED;
  if (batch < 0 || L < 0 || H < 0 || Hq < 0 || Hk < 0 || Hv < 0 || K < 0 || V < 0) return SSM_ERR_INVALID_ARG;
  if (K < 1 || V < 1 || K > SSM_LA_MAX_DIM || V > SSM_LA_MAX_DIM || L >= kMaxL) return SSM_ERR_UNSUPPORTED;
  if (H > 0 && (Hq < 1 || Hk < 1 || Hv < 1 || H % Hq || H % Hk || H % Hv)) return SSM_ERR_INVALID_ARG;
  uint64_t pairs;
  if (!mul_ok(static_cast<uint64_t>(batch), static_cast<uint64_t>(H), &pairs)) return SSM_ERR_INVALID_ARG;
  if (pairs > static_cast<uint64_t>(max_pairs) || batch > max_pairs || H > kMaxHeads)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Workspace of a call: the segments' states (`sets` of them), then float32 partial sums.
struct LaPlan {
  int nseg = 1;
  uint64_t seg_bytes = 0;             // one set
  uint64_t part[3] = {};              // dq, dk, dv of shared heads (0: not shared)
  uint64_t total = 0;
};

bool la_plan(int64_t batch, int64_t L, int64_t H, int64_t K, int64_t V, int sets, const int64_t* share, LaPlan* p) {
  if (batch == 0 || L == 0 || H == 0) return true;
  p->nseg = ssm::la_segments(batch, L, H, sets == 1 ? 1 : 3);
  if (p->nseg > 1 && !bytes_of(4, &p->seg_bytes, batch, H, p->nseg, K, V)) return false;
  p->total = up256(p->seg_bytes) * sets;
  const int64_t width[3] = {K, K, V};
  for (int i = 0; share && i < 3; ++i) {
    if (share[i] == H) continue;
    if (!bytes_of(4, &p->part[i], batch, L, H, width[i])) return false;
    p->total += up256(p->part[i]);
  }
  return p->total <= kMaxBytes;
}

struct LaTensors {
  View<3> q, k, v, d;
};

}  // namespace

extern "C" {

size_t ssm_linear_attention_workspace_size(int64_t batch, int64_t L, int64_t H, int64_t K, int64_t V, ssm_dtype dt) {
  LaPlan p;
  if (check_la_sizes(batch, L, H, H, H, H, K, V, kMaxPairs, dt) != SSM_OK) return 0;
  return la_plan(batch, L, H, K, V, 1, nullptr, &p) ? p.total : 0;
}

size_t ssm_linear_attention_bwd_workspace_size(int64_t batch, int64_t L, int64_t H, int64_t Hq, int64_t Hk, int64_t Hv,
                                               int64_t K, int64_t V, ssm_dtype dt) {
  LaPlan p;
  if (check_la_sizes(batch, L, H, Hq, Hk, Hv, K, V, kMaxPairs, dt) != SSM_OK) return 0;
  const int64_t share[3] = {Hq, Hk, Hv};
  return la_plan(batch, L, H, K, V, 2, share, &p) ? p.total : 0;
}

ssm_status ssm_linear_attention_fwd(const void* q, const void* k, const void* v, const int64_t* q_strides,
                                    const int64_t* k_strides, const int64_t* v_strides, const float* log_decay,
                                    float scale, const int32_t* lengths, const float* initial_state, void* out,
                                    float* final_state, int64_t batch, int64_t L, int64_t H, int64_t Hq, int64_t Hk,
                                    int64_t Hv, int64_t K, int64_t V, ssm_dtype dt, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  ssm_status st = check_la_sizes(batch, L, H, Hq, Hk, Hv, K, V, kMaxPairs, dt);
  if (st != SSM_OK) return st;
  const uint64_t e = dt == SSM_BF16 ? 2 : 4;
  LaTensors t;
  uint64_t out_bytes, state_bytes;
  LaPlan plan;
  if (!make_view<3>(q_strides, {batch, L, Hq}, K, e, &t.q) || !make_view<3>(k_strides, {batch, L, Hk}, K, e, &t.k) ||
      !make_view<3>(v_strides, {batch, L, Hv}, V, e, &t.v) || !bytes_of(e, &out_bytes, batch, L, H, V) ||
      !bytes_of(4, &state_bytes, batch, H, K, V) || !la_plan(batch, L, H, K, V, 1, nullptr, &plan))
    return SSM_ERR_INVALID_ARG;
  if (out_bytes && (!q || !k || !v || !out)) return SSM_ERR_INVALID_ARG;
  if (!log_decay && H > 0) return SSM_ERR_INVALID_ARG;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(out, e) || !aligned(log_decay, 4) ||
      !aligned(lengths, 4) || !aligned(initial_state, 4) || !aligned(final_state, 4) || !aligned(workspace, 16))
    return SSM_ERR_INVALID_ARG;
  if ((workspace_bytes && !workspace) || workspace_bytes < plan.total) return SSM_ERR_INVALID_ARG;
  const Span ins[] = {span(q, t.q.extent),          span(k, t.k.extent),
                      span(v, t.v.extent),          span(log_decay, 4 * static_cast<uint64_t>(H)),
                      span(lengths, 4 * static_cast<uint64_t>(batch))};
  const Span outs[] = {span(out, out_bytes), span(final_state, state_bytes), span(workspace, workspace_bytes)};
  const Span init = span(initial_state, state_bytes);
  if (any_overlap(outs, 3, ins, 5) || overlaps(outs[0], init) || overlaps(outs[2], init)) return SSM_ERR_INVALID_ARG;
  if (overlaps(outs[1], init) && final_state != initial_state) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || H == 0) return SSM_OK;
  st = probe_device();
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (L == 0)
    return final_state ? from_hip(ssm::launch_la_copy_state(final_state, initial_state, batch * H * K * V, s)) : SSM_OK;
  ssm::LaArgs a;
  a.log_decay = log_decay; a.lengths = lengths; a.batch = batch; a.L = L; a.H = static_cast<int>(H);
  a.nseg = plan.nseg; a.nroles = 1;
  ssm::LaRole& r = a.role[0];
  r.q = q; r.k = k; r.v = v; r.o = out; r.carry = initial_state; r.fin = final_state;
  for (int i = 0; i < 3; ++i) { r.qs[i] = t.q.stride[i]; r.ks[i] = t.k.stride[i]; r.vs[i] = t.v.stride[i]; }
  r.qdiv = static_cast<int>(H / Hq); r.kdiv = static_cast<int>(H / Hk); r.vdiv = static_cast<int>(H / Hv);
  r.seg = static_cast<float*>(workspace);
  r.sk = static_cast<int>(V); r.sv = 1; r.K = static_cast<int>(K); r.V = static_cast<int>(V);
  r.out_scale = scale;
  r.move = least(least(row_move(q, t.q, K, e), row_move(k, t.k, K, e)), row_move(v, t.v, V, e));
  r.o_vec = V % 4 == 0 && aligned(out, 4 * e);
  if (r.move == 16 && !aligned(out, 16)) r.move = 4;
  return from_hip(ssm::launch_la(a, dt_of(dt), s));
}

ssm_status ssm_linear_attention_bwd(const void* q, const void* k, const void* v, const void* dout,
                                    const int64_t* q_strides, const int64_t* k_strides, const int64_t* v_strides,
                                    const int64_t* dout_strides, const float* log_decay, float scale,
                                    const int32_t* lengths, const float* initial_state, const float* dfinal_state,
                                    void* dq, void* dk, void* dv, float* dinitial_state, int64_t batch, int64_t L,
                                    int64_t H, int64_t Hq, int64_t Hk, int64_t Hv, int64_t K, int64_t V, ssm_dtype dt,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  ssm_status st = check_la_sizes(batch, L, H, Hq, Hk, Hv, K, V, kMaxPairs, dt);
  if (st != SSM_OK) return st;
  const uint64_t e = dt == SSM_BF16 ? 2 : 4;
  LaTensors t;
  uint64_t qb, kb, vb, state_bytes;
  LaPlan plan;
  const int64_t share[3] = {Hq, Hk, Hv};
  if (!make_view<3>(q_strides, {batch, L, Hq}, K, e, &t.q) || !make_view<3>(k_strides, {batch, L, Hk}, K, e, &t.k) ||
      !make_view<3>(v_strides, {batch, L, Hv}, V, e, &t.v) || !make_view<3>(dout_strides, {batch, L, H}, V, e, &t.d) ||
      !bytes_of(e, &qb, batch, L, Hq, K) || !bytes_of(e, &kb, batch, L, Hk, K) || !bytes_of(e, &vb, batch, L, Hv, V) ||
      !bytes_of(4, &state_bytes, batch, H, K, V) || !la_plan(batch, L, H, K, V, 2, share, &plan))
    return SSM_ERR_INVALID_ARG;
  if (qb && (!q || !k || !v || !dout || !dq || !dk || !dv)) return SSM_ERR_INVALID_ARG;
  if (!log_decay && H > 0) return SSM_ERR_INVALID_ARG;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(dout, e) || !aligned(dq, e) || !aligned(dk, e) ||
      !aligned(dv, e) || !aligned(log_decay, 4) || !aligned(lengths, 4) || !aligned(initial_state, 4) ||
      !aligned(dfinal_state, 4) || !aligned(dinitial_state, 4) || !aligned(workspace, 16))
    return SSM_ERR_INVALID_ARG;
  if ((workspace_bytes && !workspace) || workspace_bytes < plan.total) return SSM_ERR_INVALID_ARG;
  const Span ins[] = {span(q, t.q.extent),
                      span(k, t.k.extent),
                      span(v, t.v.extent),
                      span(dout, t.d.extent),
                      span(log_decay, 4 * static_cast<uint64_t>(H)),
                      span(lengths, 4 * static_cast<uint64_t>(batch)),
                      span(initial_state, state_bytes),
                      span(dfinal_state, state_bytes)};
  const Span outs[] = {span(dq, qb), span(dk, kb), span(dv, vb), span(dinitial_state, state_bytes),
                       span(workspace, workspace_bytes)};
  if (any_overlap(outs, 5, ins, 8)) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || H == 0) return SSM_OK;
  st = probe_device();
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (L == 0)
    return dinitial_state ? from_hip(ssm::launch_la_copy_state(dinitial_state, dfinal_state, batch * H * K * V, s))
                          : SSM_OK;
  ssm::LaArgs a;
  a.log_decay = log_decay; a.lengths = lengths; a.batch = batch; a.L = L; a.H = static_cast<int>(H);
  a.nseg = plan.nseg; a.nroles = 3;
  char* ws = static_cast<char*>(workspace);
  float* seg[2] = {reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + up256(plan.seg_bytes))};
  char* at = ws + 2 * up256(plan.seg_bytes);
  void* const outp[3] = {dq, dk, dv};
  float* part[3] = {};
  for (int i = 0; i < 3; ++i) {
    if (!plan.part[i]) continue;
    part[i] = reinterpret_cast<float*>(at);
    at += up256(plan.part[i]);
  }
  struct Operand {
    const void* p;
    const View<3>* view;
    int div;
    int64_t width;
  };
  const Operand oq{q, &t.q, static_cast<int>(H / Hq), K}, ok{k, &t.k, static_cast<int>(H / Hk), K},
      ov{v, &t.v, static_cast<int>(H / Hv), V}, od{dout, &t.d, 1, V};
  const Operand ops[3][3] = {{od, ov, ok}, {ov, od, oq}, {ok, oq, od}};   // of dq, dk, dv
  for (int i = 0; i < 3; ++i) {
    ssm::LaRole& r = a.role[i];
    const Operand(&o)[3] = ops[i];
    r.q = o[0].p; r.k = o[1].p; r.v = o[2].p;
    for (int x = 0; x < 3; ++x) {
      r.qs[x] = o[0].view->stride[x]; r.ks[x] = o[1].view->stride[x]; r.vs[x] = o[2].view->stride[x];
    }
    r.qdiv = o[0].div; r.kdiv = o[1].div; r.vdiv = o[2].div;
    r.K = static_cast<int>(o[1].width); r.V = static_cast<int>(o[2].width);
    r.o = part[i] ? part[i] : outp[i];
    r.o_f32 = part[i] != nullptr;
    r.reverse = i > 0;
    r.carry = i > 0 ? dfinal_state : initial_state;
    r.fin = i == 2 ? dinitial_state : nullptr;
    r.seg = seg[i > 0];
    // the state is stored [K][V]; dq and dk see its axes exchanged
    r.sk = i == 2 ? static_cast<int>(V) : 1;
    r.sv = i == 2 ? 1 : static_cast<int>(V);
    r.in_scale = i > 0 ? scale : 1.0f;
    r.out_scale = i > 0 ? 1.0f : scale;
    r.move = 16;
    for (int x = 0; x < 3; ++x) r.move = least(r.move, row_move(o[x].p, *o[x].view, o[x].width, e));
    r.o_vec = r.V % 4 == 0 && aligned(r.o, r.o_f32 ? 16 : 4 * e);
    if (r.move == 16 && !aligned(r.o, 16)) r.move = 4;
  }
  hipError_t err = ssm::launch_la(a, dt_of(dt), s);
  const int64_t width[3] = {K, K, V};
  ssm::LaSum sums[3];
  int n = 0;
  for (int i = 0; i < 3; ++i) {
    if (!part[i]) continue;
    ssm::LaSum& x = sums[n++];
    x.part = part[i]; x.out = outp[i]; x.rows = batch * L * share[i];
    x.share = static_cast<int>(H / share[i]); x.d = static_cast<int>(width[i]);
  }
  if (err == hipSuccess && n) err = ssm::launch_la_sum_heads(sums, n, dt_of(dt), s);
  return from_hip(err);
}

ssm_status ssm_linear_attention_step(const float* state_in, float* state_out, const void* q, const void* k,
                                     const void* v, const int64_t* q_strides, const int64_t* k_strides,
                                     const int64_t* v_strides, const float* log_decay, float scale,
                                     const int32_t* slots, void* out, int64_t batch, int64_t states, int64_t H,
                                     int64_t Hq, int64_t Hk, int64_t Hv, int64_t K, int64_t V, ssm_dtype dt,
                                     void* stream) {
  ssm_status st = check_la_sizes(batch, 1, H, Hq, Hk, Hv, K, V, kMaxStepPairs, dt);
  if (st != SSM_OK) return st;
  if (states < 0 || (!slots && states < batch)) return SSM_ERR_INVALID_ARG;
  const uint64_t e = dt == SSM_BF16 ? 2 : 4;
  View<2> vq, vk, vv;
  uint64_t out_bytes, state_bytes;
  if (!make_view<2>(q_strides, {batch, Hq}, K, e, &vq) || !make_view<2>(k_strides, {batch, Hk}, K, e, &vk) ||
      !make_view<2>(v_strides, {batch, Hv}, V, e, &vv) || !bytes_of(e, &out_bytes, batch, H, V) ||
      !bytes_of(4, &state_bytes, states, H, K, V))
    return SSM_ERR_INVALID_ARG;
  if (out_bytes && (!q || !k || !v || !out || !log_decay)) return SSM_ERR_INVALID_ARG;
  if (out_bytes && state_bytes && (!state_in || !state_out)) return SSM_ERR_INVALID_ARG;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(out, e) || !aligned(state_in, 4) ||
      !aligned(state_out, 4) || !aligned(log_decay, 4) || !aligned(slots, 4))
    return SSM_ERR_INVALID_ARG;
  const Span ins[] = {span(q, vq.extent), span(k, vk.extent), span(v, vv.extent),
                      span(log_decay, 4 * static_cast<uint64_t>(H)), span(slots, 4 * static_cast<uint64_t>(batch))};
  const Span outs[] = {span(out, out_bytes), span(state_out, state_bytes)};
  const Span sin = span(state_in, state_bytes);
  if (any_overlap(outs, 2, ins, 5) || overlaps(outs[0], sin)) return SSM_ERR_INVALID_ARG;
  if (overlaps(outs[1], sin) && state_out != state_in) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || H == 0) return SSM_OK;
  st = probe_device();
  if (st != SSM_OK) return st;
  ssm::LaStepArgs a;
  a.state_in = state_in; a.state_out = state_out; a.q = q; a.k = k; a.v = v;
  for (int i = 0; i < 2; ++i) { a.qs[i] = vq.stride[i]; a.ks[i] = vk.stride[i]; a.vs[i] = vv.stride[i]; }
  a.qdiv = static_cast<int>(H / Hq); a.kdiv = static_cast<int>(H / Hk); a.vdiv = static_cast<int>(H / Hv);
  a.log_decay = log_decay; a.slots = slots; a.o = out; a.batch = batch; a.states = states;
  a.H = static_cast<int>(H); a.K = static_cast<int>(K); a.V = static_cast<int>(V); a.scale = scale;
  return from_hip(ssm::launch_la_step(a, dt_of(dt), static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

struct NormSizes {
  uint64_t act = 0, res = 0, vec = 0;   // bytes of a packed [rows][D] of each type, of a [D] float32
  View<1> x, gate;
};

ssm_status check_norm(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, int64_t rows, int64_t D,
                      int64_t groups, float eps, ssm_dtype dt, ssm_dtype rdt, NormSizes* sz) {
  if (!dtype_ok(dt) || (rdt != SSM_F32 && rdt != dt)) return SSM_ERR_UNSUPPORTED;
  if (rows < 0 || D < 0 || groups < 1 || !(eps >= 0.0f)) return SSM_ERR_INVALID_ARG;
  if (D < 1 || D > SSM_NORM_MAX_D || rows > kMaxRows) return SSM_ERR_UNSUPPORTED;
  if (D % groups) return SSM_ERR_INVALID_ARG;
  if (groups > 1 && (D / groups) % 8) return SSM_ERR_UNSUPPORTED;
  if (x_stride < D || (gate && gate_stride < D)) return SSM_ERR_INVALID_ARG;
  const uint64_t e = dt == SSM_BF16 ? 2 : 4, r = rdt == SSM_BF16 ? 2 : 4;
  const int64_t n[1] = {rows}, xs[1] = {x_stride}, gs[1] = {gate ? gate_stride : D};
  if (!make_view<1>(xs, n, D, e, &sz->x) || !make_view<1>(gs, n, D, e, &sz->gate) ||
      !bytes_of(e, &sz->act, rows, D) || !bytes_of(r, &sz->res, rows, D))
    return SSM_ERR_INVALID_ARG;
  sz->vec = static_cast<uint64_t>(D) * 4;
  if (!x && rows) return SSM_ERR_INVALID_ARG;
  if (!aligned(x, e) || !aligned(gate, e)) return SSM_ERR_INVALID_ARG;
  return SSM_OK;
}

// Whether all rows move as 8-element vectors.
bool norm_vec(const NormSizes& sz, const void* x, const void* gate, int64_t D, uint64_t e, const void* const* packed,
              int n) {
  bool ok = D % 8 == 0 && rows_aligned(x, sz.x, e, 16) && (!gate || rows_aligned(gate, sz.gate, e, 16));
  for (int i = 0; i < n; ++i) ok = ok && aligned(packed[i], 16);
  return ok;
}

}  // namespace

extern "C" {

ssm_status ssm_block_norm_fwd(const void* x, int64_t x_row_stride, const void* residual, const void* gate,
                              int64_t gate_row_stride, const float* post_weight, const float* res_scale,
                              const float* pre_weight, void* h, void* y, int64_t rows, int64_t D, int64_t groups,
                              float eps, ssm_dtype dt, ssm_dtype residual_dtype, void* stream) {
  NormSizes sz;
  ssm_status st = check_norm(x, x_row_stride, gate, gate_row_stride, rows, D, groups, eps, dt, residual_dtype, &sz);
  if (st != SSM_OK) return st;
  if (rows && ((pre_weight != nullptr) != (y != nullptr) || (!h && !y))) return SSM_ERR_INVALID_ARG;
  const uint64_t e = dt == SSM_BF16 ? 2 : 4, r = residual_dtype == SSM_BF16 ? 2 : 4;
  if (!aligned(residual, r) || !aligned(h, r) || !aligned(y, e) || !aligned(post_weight, 4) ||
      !aligned(res_scale, 4) || !aligned(pre_weight, 4))
    return SSM_ERR_INVALID_ARG;
  const Span ins[] = {span(x, sz.x.extent), span(gate, sz.gate.extent), span(post_weight, sz.vec),
                      span(res_scale, sz.vec), span(pre_weight, sz.vec)};
  const Span outs[] = {span(h, sz.res), span(y, sz.act)};
  const Span rs = span(residual, sz.res);
  if (any_overlap(outs, 2, ins, 5) || overlaps(outs[1], rs)) return SSM_ERR_INVALID_ARG;
  if (overlaps(outs[0], rs) && h != residual) return SSM_ERR_INVALID_ARG;
  if (rows == 0) return SSM_OK;
  st = probe_device();
  if (st != SSM_OK) return st;
  ssm::NormArgs a;
  a.x = x; a.gate = gate; a.residual = residual; a.w1 = post_weight; a.rs = res_scale; a.w2 = pre_weight;
  a.h = h; a.y = y; a.rows = rows; a.D = D; a.x_row = x_row_stride; a.gate_row = gate_row_stride;
  a.group = D / groups; a.eps = eps;
  const void* const packed[] = {residual, h, y, post_weight, res_scale, pre_weight};
  a.vec = norm_vec(sz, x, gate, D, e, packed, 6);
  return from_hip(ssm::launch_norm_fwd(a, dt_of(dt), dt_of(residual_dtype), static_cast<hipStream_t>(stream)));
}

size_t ssm_block_norm_bwd_workspace_size(int64_t rows, int64_t D) {
  if (rows <= 0 || D < 1 || D > SSM_NORM_MAX_D || rows > kMaxRows) return 0;
  return static_cast<size_t>(ssm::norm_bwd_parts(rows, D)) * 3 * static_cast<size_t>(D) * sizeof(float);
}

ssm_status ssm_block_norm_bwd(const void* x, int64_t x_row_stride, const void* h, const void* dy, const void* dh,
                              const void* gate, int64_t gate_row_stride, const float* post_weight,
                              const float* res_scale, const float* pre_weight, void* dx, void* dgate, void* dresidual,
                              float* dpost_weight, float* dres_scale, float* dpre_weight, int64_t rows, int64_t D,
                              int64_t groups, float eps, ssm_dtype dt, ssm_dtype residual_dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  NormSizes sz;
  ssm_status st = check_norm(x, x_row_stride, gate, gate_row_stride, rows, D, groups, eps, dt, residual_dtype, &sz);
  if (st != SSM_OK) return st;
  if (rows && ((pre_weight != nullptr) != (dy != nullptr) || (pre_weight && !h) || !dx ||
               (gate != nullptr) != (dgate != nullptr)))
    return SSM_ERR_INVALID_ARG;
  if ((post_weight != nullptr) != (dpost_weight != nullptr) || (res_scale != nullptr) != (dres_scale != nullptr) ||
      (pre_weight != nullptr) != (dpre_weight != nullptr))
    return SSM_ERR_INVALID_ARG;
  const uint64_t e = dt == SSM_BF16 ? 2 : 4, r = residual_dtype == SSM_BF16 ? 2 : 4;
  if (!aligned(h, r) || !aligned(dy, e) || !aligned(dh, r) || !aligned(dx, e) || !aligned(dgate, e) ||
      !aligned(dresidual, r) || !aligned(post_weight, 4) || !aligned(res_scale, 4) || !aligned(pre_weight, 4) ||
      !aligned(dpost_weight, 4) || !aligned(dres_scale, 4) || !aligned(dpre_weight, 4) || !aligned(workspace, 16))
    return SSM_ERR_INVALID_ARG;
  const uint64_t need = ssm_block_norm_bwd_workspace_size(rows, D);
  if ((workspace_bytes && !workspace) || workspace_bytes < need) return SSM_ERR_INVALID_ARG;
  const Span ins[] = {span(x, sz.x.extent),      span(gate, sz.gate.extent), span(h, sz.res),
                      span(dy, sz.act),          span(post_weight, sz.vec),  span(res_scale, sz.vec),
                      span(pre_weight, sz.vec)};
  const Span outs[] = {span(dx, sz.act),           span(dgate, sz.act),        span(dresidual, sz.res),
                       span(dpost_weight, sz.vec), span(dres_scale, sz.vec),   span(dpre_weight, sz.vec),
                       span(workspace, workspace_bytes)};
  if (any_overlap(outs, 7, ins, 7)) return SSM_ERR_INVALID_ARG;
  const Span dhs = span(dh, sz.res);
  for (const Span& o : outs)
    if (overlaps(o, dhs) && !(o.lo == outs[2].lo && dresidual && dresidual == dh)) return SSM_ERR_INVALID_ARG;
  st = probe_device();
  if (st != SSM_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) {
    hipError_t err = hipSuccess;
    float* const sums[] = {dpost_weight, dres_scale, dpre_weight};
    for (float* p : sums)
      if (p && err == hipSuccess) err = ssm::launch_copy_state(p, nullptr, D, s);
    return from_hip(err);
  }
  ssm::NormArgs a;
  a.x = x; a.gate = gate; a.w1 = post_weight; a.rs = res_scale; a.w2 = pre_weight;
  a.rows = rows; a.D = D; a.x_row = x_row_stride; a.gate_row = gate_row_stride; a.group = D / groups; a.eps = eps;
  a.hin = h; a.dy = dy; a.dh = dh; a.dx = dx; a.dgate = dgate; a.dres = dresidual;
  a.dw1 = dpost_weight; a.drs = dres_scale; a.dw2 = dpre_weight;
  a.part = static_cast<float*>(workspace);
  a.parts = ssm::norm_bwd_parts(rows, D);
  const void* const packed[] = {h, dy, dh, dx, dgate, dresidual, post_weight, res_scale, pre_weight};
  a.vec = norm_vec(sz, x, gate, D, e, packed, 9);
  return from_hip(ssm::launch_norm_bwd(a, dt_of(dt), dt_of(residual_dtype), s));
}

}  // extern "C"
