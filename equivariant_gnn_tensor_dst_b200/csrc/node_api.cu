// C ABI of the node-feature operators (include/tpconv_node.h): plans, argument checks and
// launches.
#include <cmath>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/tpconv_node.h"
#include "irreps.h"
#include "node.h"
#include "prof.h"

using namespace tpc;

struct tpconv_node_plan {
  NodeDesc desc{};
  int dtype = TPCONV_DTYPE_F32;
  // workspace of the last row count asked for (host bookkeeping: a training loop asks for the same)
  mutable std::mutex mu;
  mutable int64_t ws_rows = -1;
  mutable size_t ws_bytes = 0;
};

namespace {

size_t elem_bytes(const tpconv_node_plan* P) { return P->dtype == TPCONV_DTYPE_F32 ? 4 : 2; }

// The arrays of one call, checked together: required ones present, 16-byte alignment, no
// output overlapping another array.
struct Arrays {
  struct Span {
    uintptr_t p;
    size_t bytes;
    bool out;
  } a[16];
  int n = 0;
  bool missing = false, misaligned = false;

  void add(const void* p, size_t bytes, bool required, bool out) {
    if (!p) {
      missing = missing || required;
      return;
    }
    const uintptr_t v = reinterpret_cast<uintptr_t>(p);
    misaligned = misaligned || (v & 15u) != 0;
    if (bytes) a[n++] = Span{v, bytes, out};
  }
  // in_place: exact equality of an output with an input is allowed (element-wise operators)
  tpconv_status check(bool in_place = false) const {
    if (missing) return TPCONV_ERR_INVALID_ARG;
    if (misaligned) return TPCONV_ERR_MISALIGNED;
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j) {
        if (!a[i].out && !a[j].out) continue;
        if (in_place && a[i].out != a[j].out && a[i].p == a[j].p && a[i].bytes == a[j].bytes) continue;
        if (a[i].p < a[j].p + a[j].bytes && a[j].p < a[i].p + a[i].bytes) return TPCONV_ERR_INVALID_ARG;
      }
    return TPCONV_OK;
  }
};

bool rows_ok(const tpconv_node_plan* P, int64_t N) { return P && N >= 0 && N < 0x80000000LL; }

tpconv_status make_drop(const tpconv_dropout_spec* spec, Drop& d) {
  if (!spec || !(spec->p >= 0.0 && spec->p <= 1.0)) return TPCONV_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(spec->step) & 7u) != 0) return TPCONV_ERR_MISALIGNED;
  for (uint32_t i = 0; i < 10; ++i) {  // each round advances the key by fixed odd increments
    d.key[i][0] = (uint32_t)spec->seed + i * 0x9E3779B9u;
    d.key[i][1] = (uint32_t)(spec->seed >> 32) + i * 0xBB67AE85u;
  }
  d.offset = spec->offset;
  d.step = reinterpret_cast<const long long*>(spec->step);
  const double t = std::floor(spec->p * 4294967296.0 + 0.5);
  d.mode = t <= 0.0 ? 0 : t >= 4294967296.0 ? 2 : 1;
  d.threshold = d.mode == 1 ? (uint32_t)t : 0;
  d.scale = spec->p < 1.0 ? (float)(1.0 / (1.0 - spec->p)) : 0.f;
  return TPCONV_OK;
}

size_t sums_bytes(const tpconv_node_plan* P, int64_t N) {
  std::lock_guard<std::mutex> g(P->mu);
  if (P->ws_rows != N) {
    P->ws_bytes = sizeof(float) * norm_partial_floats(P->desc, N, (int)elem_bytes(P));
    P->ws_rows = N;
  }
  return P->ws_bytes;
}

// Bytes of the workspace that a pass writes, for the overlap check (one that is too small is
// reported as that).
size_t ws_span(const tpconv_node_plan* P, int64_t N, size_t ws_bytes) {
  const size_t need = sums_bytes(P, N);
  return ws_bytes < need ? ws_bytes : need;
}

// Workspace of the sums over rows; NULL *partial when no sum is wanted.
tpconv_status sums_workspace(const tpconv_node_plan* P, int64_t N, bool wanted, void* ws, size_t ws_bytes,
                             float** partial) {
  *partial = nullptr;
  if (!wanted || N == 0) return TPCONV_OK;
  const size_t need = sums_bytes(P, N);
  if (ws_bytes < need) return TPCONV_ERR_WORKSPACE_TOO_SMALL;
  if (need == 0) return TPCONV_OK;  // few rows: the sums go to the gradients themselves
  if (!ws) return TPCONV_ERR_INVALID_ARG;
  *partial = static_cast<float*>(ws);
  return TPCONV_OK;
}

// N = 0: the sums over rows are zero
tpconv_status zero_sums(const tpconv_node_plan* P, float* grad_weight, float* grad_bias, cudaStream_t s) {
  if (grad_weight && cudaMemsetAsync(grad_weight, 0, sizeof(float) * P->desc.channels, s) != cudaSuccess)
    return TPCONV_ERR_CUDA;
  if (grad_bias && P->desc.biases &&
      cudaMemsetAsync(grad_bias, 0, sizeof(float) * P->desc.biases, s) != cudaSuccess)
    return TPCONV_ERR_CUDA;
  return TPCONV_OK;
}

tpconv_status run(const tpconv_node_plan* P, NormPass pass, int64_t N, const NormArgs& A, const Drop* drop,
                  cudaStream_t s) {
  ProfScope scope(PC_NODE, 0, s);
  return launch_norm(pass, P->dtype, P->desc, N, A, drop, s) == cudaSuccess ? TPCONV_OK : TPCONV_ERR_CUDA;
}

}  // namespace

extern "C" {

tpconv_status tpconv_node_plan_create(tpconv_node_plan_t* out, const char* irreps, int32_t dtype, float eps) {
  if (!out || !irreps) return TPCONV_ERR_INVALID_ARG;
  if (dtype != TPCONV_DTYPE_F32 && dtype != TPCONV_DTYPE_BF16 && dtype != TPCONV_DTYPE_F16)
    return TPCONV_ERR_UNSUPPORTED;
  if (!(eps > 0.f) || !std::isnormal(eps)) return TPCONV_ERR_INVALID_ARG;
  try {
    std::vector<Block> blocks;
    const tpconv_status st = parse_irreps(irreps, blocks);
    if (st != TPCONV_OK) return st;
    tpconv_node_plan* P = new tpconv_node_plan();
    NodeDesc& D = P->desc;
    for (const Block& b : blocks) {
      NodeBlock& B = D.b[D.n_blocks++];
      B.off = b.offset;
      B.C = b.mul;
      B.d = 2 * b.l + 1;
      B.S = B.C * B.d;
      B.chan0 = D.channels;
      B.grp0 = D.groups;
      const bool centred = b.l == 0 && b.parity == 1;
      B.bias0 = centred ? D.biases : -1;
      D.dim += B.S;
      D.channels += B.C;
      D.groups += (B.C + 3) / 4;
      if (centred) D.biases += B.C;
    }
    D.eps = eps;
    P->dtype = dtype;
    *out = P;
    return TPCONV_OK;
  } catch (...) {
    return TPCONV_ERR_INVALID_ARG;
  }
}

tpconv_status tpconv_node_plan_destroy(tpconv_node_plan_t P) {
  delete P;
  return TPCONV_OK;
}

tpconv_status tpconv_node_plan_info(tpconv_node_plan_t P, int64_t* dim, int64_t* channels, int64_t* biases,
                                    int64_t* blocks) {
  if (!P) return TPCONV_ERR_INVALID_ARG;
  if (dim) *dim = P->desc.dim;
  if (channels) *channels = P->desc.channels;
  if (biases) *biases = P->desc.biases;
  if (blocks) *blocks = P->desc.n_blocks;
  return TPCONV_OK;
}

tpconv_status tpconv_node_plan_set_layout(tpconv_node_plan_t P, int32_t layout) {
  if (!P) return TPCONV_ERR_INVALID_ARG;
  if (layout != TPCONV_LAYOUT_IR_MUL && layout != TPCONV_LAYOUT_MUL_IR) return TPCONV_ERR_UNSUPPORTED;
  P->desc.mul_ir = layout == TPCONV_LAYOUT_MUL_IR;
  return TPCONV_OK;
}

tpconv_status tpconv_node_workspace_bytes(tpconv_node_plan_t P, int64_t N, size_t* bytes) {
  if (!bytes || !rows_ok(P, N)) return TPCONV_ERR_INVALID_ARG;
  *bytes = sums_bytes(P, N);
  return TPCONV_OK;
}

tpconv_status tpconv_norm_forward(tpconv_node_plan_t P, int64_t N, const void* x, const float* weight,
                                  const float* bias, void* y, struct CUstream_st* stream) {
  if (!rows_ok(P, N)) return TPCONV_ERR_INVALID_ARG;
  if (N == 0) return TPCONV_OK;
  const size_t rows = elem_bytes(P) * N * P->desc.dim;
  Arrays a;
  a.add(x, rows, true, false);
  a.add(weight, sizeof(float) * P->desc.channels, false, false);
  a.add(bias, sizeof(float) * P->desc.biases, false, false);
  a.add(y, rows, true, true);
  const tpconv_status st = a.check();
  if (st != TPCONV_OK) return st;
  NormArgs A{};
  A.x = x;
  A.weight = weight;
  A.bias = bias;
  A.y = y;
  return run(P, NORM_FORWARD, N, A, nullptr, (cudaStream_t)stream);
}

tpconv_status tpconv_norm_backward(tpconv_node_plan_t P, int64_t N, const void* x, const float* weight,
                                   const void* grad_y, void* grad_x, float* grad_weight, float* grad_bias, void* ws,
                                   size_t ws_bytes, struct CUstream_st* stream) {
  if (!rows_ok(P, N)) return TPCONV_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t rows = elem_bytes(P) * N * P->desc.dim;
  Arrays a;
  a.add(x, rows, N > 0, false);
  a.add(weight, sizeof(float) * P->desc.channels, false, false);
  a.add(grad_y, rows, N > 0, false);
  a.add(grad_x, rows, false, true);
  a.add(grad_weight, sizeof(float) * P->desc.channels, false, true);
  a.add(grad_bias, sizeof(float) * P->desc.biases, false, true);
  const bool sums = grad_weight || (grad_bias && P->desc.biases);
  a.add(sums ? ws : nullptr, ws_span(P, N, ws_bytes), false, true);
  tpconv_status st = a.check();
  if (st != TPCONV_OK) return st;
  NormArgs A{};
  st = sums_workspace(P, N, sums, ws, ws_bytes, &A.partial);
  if (st != TPCONV_OK) return st;
  if (N == 0) return zero_sums(P, grad_weight, grad_bias, s);
  if (!grad_x && !sums) return TPCONV_OK;
  A.x = x;
  A.weight = weight;
  A.grad_y = grad_y;
  A.grad_x = grad_x;
  A.grad_weight = grad_weight;
  A.grad_bias = grad_bias;
  return run(P, NORM_BACKWARD, N, A, nullptr, s);
}

tpconv_status tpconv_norm_double_backward(tpconv_node_plan_t P, int64_t N, const void* x, const float* weight,
                                          const void* grad_y, const void* gg_x, const float* gg_weight,
                                          const float* gg_bias, void* grad_x, float* grad_weight, void* grad_grad_y,
                                          void* ws, size_t ws_bytes, struct CUstream_st* stream) {
  if (!rows_ok(P, N)) return TPCONV_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t rows = elem_bytes(P) * N * P->desc.dim;
  Arrays a;
  a.add(x, rows, N > 0, false);
  a.add(weight, sizeof(float) * P->desc.channels, false, false);
  a.add(grad_y, rows, N > 0, false);
  a.add(gg_x, rows, false, false);
  a.add(gg_weight, sizeof(float) * P->desc.channels, false, false);
  a.add(gg_bias, sizeof(float) * P->desc.biases, false, false);
  a.add(grad_x, rows, false, true);
  a.add(grad_weight, sizeof(float) * P->desc.channels, false, true);
  a.add(grad_grad_y, rows, false, true);
  a.add(grad_weight ? ws : nullptr, ws_span(P, N, ws_bytes), false, true);
  tpconv_status st = a.check();
  if (st != TPCONV_OK) return st;
  NormArgs A{};
  st = sums_workspace(P, N, grad_weight != nullptr, ws, ws_bytes, &A.partial);
  if (st != TPCONV_OK) return st;
  if (N == 0) return zero_sums(P, grad_weight, nullptr, s);
  if (!grad_x && !grad_weight && !grad_grad_y) return TPCONV_OK;
  A.x = x;
  A.weight = weight;
  A.grad_y = grad_y;
  A.gg_x = gg_x;
  A.gg_weight = gg_weight;
  A.gg_bias = gg_bias;
  A.grad_x = grad_x;
  A.grad_weight = grad_weight;
  A.grad_grad_y = grad_grad_y;
  return run(P, NORM_DOUBLE_BACKWARD, N, A, nullptr, s);
}

tpconv_status tpconv_dropout_forward(tpconv_node_plan_t P, int64_t N, const void* x, const void* residual,
                                     const tpconv_dropout_spec* dropout, void* out, struct CUstream_st* stream) {
  if (!rows_ok(P, N)) return TPCONV_ERR_INVALID_ARG;
  Drop drop{};
  tpconv_status st = make_drop(dropout, drop);
  if (st != TPCONV_OK) return st;
  if (N == 0) return TPCONV_OK;
  const size_t rows = elem_bytes(P) * N * P->desc.dim;
  Arrays a;
  a.add(x, rows, true, false);
  a.add(residual, rows, false, false);
  a.add(out, rows, true, true);
  st = a.check(true);
  if (st != TPCONV_OK) return st;
  ProfScope scope(PC_NODE, 0, (cudaStream_t)stream);
  return launch_dropout(P->dtype, P->desc, N, x, residual, drop, out, (cudaStream_t)stream) == cudaSuccess
             ? TPCONV_OK
             : TPCONV_ERR_CUDA;
}

tpconv_status tpconv_dropout_backward(tpconv_node_plan_t P, int64_t N, const void* grad_out,
                                      const tpconv_dropout_spec* dropout, void* grad_x, struct CUstream_st* stream) {
  return tpconv_dropout_forward(P, N, grad_out, nullptr, dropout, grad_x, stream);
}

tpconv_status tpconv_dropout_norm_forward(tpconv_node_plan_t P, int64_t N, const void* x, const void* residual,
                                          const tpconv_dropout_spec* dropout, const float* weight, const float* bias,
                                          void* z, void* y, struct CUstream_st* stream) {
  if (!rows_ok(P, N)) return TPCONV_ERR_INVALID_ARG;
  Drop drop{};
  tpconv_status st = make_drop(dropout, drop);
  if (st != TPCONV_OK) return st;
  if (N == 0) return TPCONV_OK;
  const size_t rows = elem_bytes(P) * N * P->desc.dim;
  Arrays a;
  a.add(x, rows, true, false);
  a.add(residual, rows, false, false);
  a.add(weight, sizeof(float) * P->desc.channels, false, false);
  a.add(bias, sizeof(float) * P->desc.biases, false, false);
  a.add(z, rows, true, true);
  a.add(y, rows, true, true);
  st = a.check();
  if (st != TPCONV_OK) return st;
  NormArgs A{};
  A.x = x;
  A.residual = residual;
  A.weight = weight;
  A.bias = bias;
  A.z = z;
  A.y = y;
  return run(P, NORM_FORWARD, N, A, &drop, (cudaStream_t)stream);
}

tpconv_status tpconv_dropout_norm_backward(tpconv_node_plan_t P, int64_t N, const void* z, const float* weight,
                                           const void* grad_y, const void* grad_z,
                                           const tpconv_dropout_spec* dropout, void* grad_x, void* grad_residual,
                                           float* grad_weight, float* grad_bias, void* ws, size_t ws_bytes,
                                           struct CUstream_st* stream) {
  if (!rows_ok(P, N)) return TPCONV_ERR_INVALID_ARG;
  Drop drop{};
  tpconv_status st = make_drop(dropout, drop);
  if (st != TPCONV_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const size_t rows = elem_bytes(P) * N * P->desc.dim;
  Arrays a;
  a.add(z, rows, N > 0, false);
  a.add(weight, sizeof(float) * P->desc.channels, false, false);
  a.add(grad_y, rows, N > 0, false);
  a.add(grad_z, rows, false, false);
  a.add(grad_x, rows, false, true);
  a.add(grad_residual, rows, false, true);
  a.add(grad_weight, sizeof(float) * P->desc.channels, false, true);
  a.add(grad_bias, sizeof(float) * P->desc.biases, false, true);
  const bool sums = grad_weight || (grad_bias && P->desc.biases);
  a.add(sums ? ws : nullptr, ws_span(P, N, ws_bytes), false, true);
  st = a.check();
  if (st != TPCONV_OK) return st;
  NormArgs A{};
  st = sums_workspace(P, N, sums, ws, ws_bytes, &A.partial);
  if (st != TPCONV_OK) return st;
  if (N == 0) return zero_sums(P, grad_weight, grad_bias, s);
  if (!grad_x && !grad_residual && !sums) return TPCONV_OK;
  A.x = z;
  A.weight = weight;
  A.grad_y = grad_y;
  A.grad_z = grad_z;
  A.grad_x = grad_x;
  A.grad_residual = grad_residual;
  A.grad_weight = grad_weight;
  A.grad_bias = grad_bias;
  return run(P, NORM_BACKWARD, N, A, &drop, s);
}

}  // extern "C"
