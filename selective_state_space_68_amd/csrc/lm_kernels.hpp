// Internal launch interface of the linear attention and block norm kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"

namespace ssm {

// One linear attention over the tokens of every (batch row, head),
//     E <- the carried state;  o_i = out_scale (sum_{j<=i} lam^(i-j) in_scale (q_i.k_j) v_j + lam^i q_i E),
// forwards or backwards in time.  The forward operator is one such role; the gradient is
// three: (q, k, v) = (do, v, k) forwards for dq, (v, do, q) and (k, q, do) backwards for
// dk and dv.  States are float32; `sk` and `sv` are the element strides of the state's two
// axes as this role sees them (its k axis, its v axis), so a role can use the state that
// another role built with the axes exchanged.
struct LaRole {
  const void *q = nullptr, *k = nullptr, *v = nullptr;   // elements of the activation type
  int64_t qs[3] = {}, ks[3] = {}, vs[3] = {};            // element strides: batch, token, head
  int qdiv = 1, kdiv = 1, vdiv = 1;                      // head h of the state uses head h / div
  void* o = nullptr;                                     // [batch][L][H][V]
  int o_f32 = 0;                                         // o is float32 (partial sums of a shared head)
  const float* carry = nullptr;                          // state before the first token, or null (zero)
  float* fin = nullptr;                                  // state after the last token, or null
  float* seg = nullptr;                                  // [batch * H][nseg][K * V]: the segments' states
  int sk = 0, sv = 0;
  int K = 0, V = 0;
  float in_scale = 1.0f, out_scale = 1.0f;
  int reverse = 0;
  int move = 0;                                          // bytes in which rows of q, k and v move: 16, 4, or 0 (an element)
  int o_vec = 0;                                         // rows of o move as 4-element vectors
};

struct LaArgs {
  LaRole role[3];
  int nroles = 1;
  const float* log_decay = nullptr;   // [H]
  const int32_t* lengths = nullptr;   // [batch] or null
  int64_t batch = 0, L = 0;
  int H = 0;
  int nseg = 1;
  int64_t seg_chunks = 0;
};

constexpr int kLaMaxDim = 128;        // largest K and V

// Segments per sequence of a call with `roles` roles.
int la_segments(int64_t batch, int64_t L, int64_t H, int roles);
hipError_t launch_la(const LaArgs& a, Dt dt, hipStream_t s);

// out[rows][d] (act) = sum over `share` of part[rows][share][d]: rows are the (batch row, token, head), d <= 128.
// `part` is 16-byte aligned.
struct LaSum {
  const float* part = nullptr;
  void* out = nullptr;
  int64_t rows = 0;
  int share = 1, d = 1;
};
hipError_t launch_la_sum_heads(const LaSum* sums, int n, Dt dt, hipStream_t s);

// dst = src, or zeros when src is null (the state of an attention over no tokens; up to 2^34 entries, of which
// launch_copy_state's thread for each takes fewer than 2^32).
hipError_t launch_la_copy_state(float* dst, const float* src, int64_t n, hipStream_t s);

struct LaStepArgs {
  const float* state_in = nullptr;    // [states][H][K][V]
  float* state_out = nullptr;
  const void *q = nullptr, *k = nullptr, *v = nullptr;
  int64_t qs[2] = {}, ks[2] = {}, vs[2] = {};            // element strides: batch, head
  int qdiv = 1, kdiv = 1, vdiv = 1;
  const float* log_decay = nullptr;
  const int32_t* slots = nullptr;     // [batch] or null
  void* o = nullptr;                  // [batch][H][V]
  int64_t batch = 0, states = 0;
  int H = 0, K = 0, V = 0;
  float scale = 1.0f;
};
hipError_t launch_la_step(const LaStepArgs& a, Dt dt, hipStream_t s);

// The gated delta rule over the tokens of every (batch row, head).
struct GdArgs {
  const void *q = nullptr, *k = nullptr, *v = nullptr;
  int64_t qs[3] = {}, ks[3] = {}, vs[3] = {};            // element strides: batch, token, head
  int qdiv = 1, kdiv = 1, vdiv = 1;                      // head h of the state uses head h / div
  const float *g = nullptr, *beta = nullptr;             // [batch][L][H]
  const int32_t* lengths = nullptr;                      // [batch] or null
  const float* carry = nullptr;                          // state before the first token, or null (zero)
  float* fin = nullptr;                                  // state after the last token, or null
  void* o = nullptr;                                     // [batch][L][H][V]
  int o_f32 = 0;                                         // (the gradient of a shared head of v) o is float32
  char *rec = nullptr, *rec_back = nullptr;              // a record for each chunk of each (batch row, head)
  float* w_out = nullptr;                                // gradient walks: [batch * H][chunks][64][w_stride]
  int w_stride = 0;                                      // V in whole blocks of 64
  float* kept = nullptr;                                 // ... the state before every `every` chunks, [batch * H][..][K * V]
  int every = 1;
  int nseg = 1, seg_chunks = 0;                          // segments of a sequence, and their chunks (set by the launch)
  float* seg = nullptr;                                  // [batch * H][nseg][K * V]: states entering the segments
  float *seg_m = nullptr, *seg_mt = nullptr;             // [batch * H][nseg][64 or 128 squared]; mt where a gradient needs it
  int64_t batch = 0, L = 0;
  int H = 0, K = 0, V = 0;
  float scale = 1.0f;
  int move = 0;                                          // bytes in which rows of q, k and v move: 16, 4, or 0 (an element)
  int o_vec = 0;                                         // rows of o move as 4-element vectors
};
// The gradients of q, k, g and beta from what the walks left.
struct GdGradArgs {
  const void *q = nullptr, *k = nullptr, *v = nullptr, *d = nullptr;   // d: the outputs' gradient, [batch][L][H][V]
  int64_t qs[3] = {}, ks[3] = {}, vs[3] = {}, ds[3] = {};
  int qdiv = 1, kdiv = 1, vdiv = 1;
  char* rec = nullptr;
  float* through = nullptr;                              // states before chunks of which a part passes through, [batch * H][chunks][..]
  const float *w = nullptr, *y = nullptr;                // w_out of the two walks
  const float *kept_e = nullptr, *kept_f = nullptr;      // kept of the two walks
  const int32_t* lengths = nullptr;
  void* dq = nullptr;                                    // [batch][L][H][K]; dq_f32: float32 (partial sums of a shared head)
  float* dk_part = nullptr;                              // dk's forward part, [batch * H][chunks][64 or 128 columns][64]
  void* dk = nullptr;                                    // [batch][L][H][K]; dk_f32: float32, as dq
  float *dg = nullptr, *dbeta = nullptr;                 // [batch][L][H]
  int64_t batch = 0, L = 0;
  int H = 0, K = 0, V = 0, every = 1;
  float scale = 1.0f;
  int dq_f32 = 0, dk_f32 = 0;
  int carried = 0;                                       // there is an initial state
  int move = 0;                                          // bytes in which rows of q, k, v and d move (16, 4, 0: an element); 16: those of dq and dk as 4 elements
};
int gd_every(int64_t batch, int64_t L, int64_t H, int64_t K, int64_t V, Dt dt);
hipError_t launch_gd_qk(const GdGradArgs& a, Dt dt, hipStream_t s);

struct GdStepArgs {
  const float* state_in = nullptr;    // [states][H][K][V]
  float* state_out = nullptr;
  const void *q = nullptr, *k = nullptr, *v = nullptr;
  int64_t qs[2] = {}, ks[2] = {}, vs[2] = {};            // element strides: batch, head
  int qdiv = 1, kdiv = 1, vdiv = 1;
  const float *g = nullptr, *beta = nullptr;             // [batch][H]
  const int32_t* slots = nullptr;     // [batch] or null
  void* o = nullptr;                  // [batch][H][V]
  int64_t batch = 0, states = 0;
  int H = 0, K = 0, V = 0;
  float scale = 1.0f;
};
hipError_t launch_gd_step(const GdStepArgs& a, Dt dt, hipStream_t s);

struct GdRecords {
  int64_t out, save, back;                               // bytes of a chunk's record: forward pass, the gradient's walks
};
GdRecords gd_records(Dt dt);
int gd_segments(int64_t batch, int64_t L, int64_t H);
hipError_t launch_gd(const GdArgs& a, Dt dt, hipStream_t s);
// The two walks of the gradient: forwards (v, carry: the inputs'), then backwards (v: the outputs' gradient, carry: the
// final state's, o: dv, fin: the initial state's).
hipError_t launch_gd_walks(const GdArgs& forwards, const GdArgs& backwards, Dt dt, hipStream_t s);

// Norms of queries and keys with the rotation.
struct QkArgs {
  const void *q = nullptr, *k = nullptr;
  int64_t qs[3] = {}, ks[3] = {};                        // element strides: batch, token, head
  const void *dqo = nullptr, *dko = nullptr;             // gradients of the outputs
  int64_t dqs[3] = {}, dks[3] = {};
  const float *qw = nullptr, *kw = nullptr;              // [K] or null
  const float* inv_freq = nullptr;                       // [rotary / 2]
  const int32_t* positions = nullptr;                    // [batch][L] or null (0..L-1)
  void *qo = nullptr, *ko = nullptr;                     // packed outputs, backwards dq and dk
  float *dqw = nullptr, *dkw = nullptr;                  // [K] or null
  float* part = nullptr;                                 // [2][workgroups][K]
  int64_t batch = 0, L = 0;
  int Hq = 0, Hk = 0, K = 0, rotary = 0, interleaved = 0;
  float inv_count = 1.0f, eps = 0.0f;                    // 1 / K, or 1 for the norm by the sum
  int vec = 0;                                           // rows move as pieces of 4 elements
  int split = 1;
};
int qk_norm_parts();                                     // most workgroups that sum the weights' gradients
hipError_t launch_qk_norm(const QkArgs& a, Dt dt, hipStream_t s);
hipError_t launch_qk_norm_bwd(const QkArgs& a, Dt dt, hipStream_t s);

struct NormArgs {
  const void *x = nullptr, *gate = nullptr, *residual = nullptr;
  const float *w1 = nullptr, *rs = nullptr, *w2 = nullptr;   // post weight, residual scale, pre weight: [D] or null
  void *h = nullptr, *y = nullptr;                            // forward outputs, or null
  int64_t rows = 0, D = 0, x_row = 0, gate_row = 0;           // row strides of x and gate in elements
  int64_t group = 0;                                          // columns of a group of the first norm
  float eps = 0.0f;
  int vec = 0;                                                // every row moves as 8-element vectors
  // backward
  const void *hin = nullptr, *dy = nullptr, *dh = nullptr;
  void *dx = nullptr, *dgate = nullptr, *dres = nullptr;
  float *dw1 = nullptr, *drs = nullptr, *dw2 = nullptr;
  float* part = nullptr;                                      // [parts][3][D] column sums of row blocks
  int parts = 0;
};
hipError_t launch_norm_fwd(const NormArgs& a, Dt dt, Dt rdt, hipStream_t s);
// Row blocks of the backward pass: each forms its own column sums.
int norm_bwd_parts(int64_t rows, int64_t D);
hipError_t launch_norm_bwd(const NormArgs& a, Dt dt, Dt rdt, hipStream_t s);

}  // namespace ssm
