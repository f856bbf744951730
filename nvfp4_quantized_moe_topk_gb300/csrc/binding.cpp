// binding.cpp -- Python module with the argument checks of the operators
// around the layer: torch tensors in, the C ABI's argument structs out.
//
// These operators run for a few microseconds on the smallest batches, less
// than ctypes and a dozen tensors' attribute look-ups in Python take (8 to 17
// us a call); here a tensor's type, device, shape and strides are read in
// place.  Every refusal is raised as the error class that set_error was given,
// before anything is enqueued.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/moe_nvfp4.h"

namespace {

PyObject* g_error = nullptr;  // MoeError(status, where, why)

// Thrown after the Python error has been set.
struct Raised {};

[[noreturn]] void raise(int status, const char* where, const std::string& why) {
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "iss", status, where, why.c_str()) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, why.c_str());
  }
  throw Raised();
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

// One call's arguments: where it is, the device of its first tensor.
struct Call {
  const char* where;
  int device = -1;

  [[noreturn]] void refuse(const std::string& why) const { raise(MOE_ERR_INVALID_ARG, where, why); }

  const at::Tensor* tensor(PyObject* o, const char* name) const {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " is not a tensor");
    return &THPVariable_Unpack(o);
  }
  // The call's leading tensor: its device has to be the current one, where the kernels are launched.
  void lead(const at::Tensor& t) {
    device = t.get_device();
    if (device < 0 || device != c10::cuda::current_device())
      refuse("the tensors are not on the current CUDA device");
  }
  void type(const at::Tensor& t, const char* name, at::ScalarType want) const {
    if (t.scalar_type() != want)
      refuse(std::string(name) + " is " + c10::toString(t.scalar_type()) + ", not " + c10::toString(want));
    if (t.get_device() != device) refuse(std::string(name) + " is not on the call's CUDA device");
  }
  // MOE_DTYPE_ of a tensor that may be bf16 or fp32.
  int32_t dtype(const at::Tensor& t, const char* name) const {
    if (t.scalar_type() == at::kBFloat16) return MOE_DTYPE_BF16;
    if (t.scalar_type() != at::kFloat)
      refuse(std::string(name) + " is " + c10::toString(t.scalar_type()) + "; bfloat16 or float32 is supported");
    return MOE_DTYPE_F32;
  }
  void* array(const at::Tensor* t, const char* name, at::ScalarType want, at::IntArrayRef shape) const {
    if (!t) return nullptr;
    type(*t, name, want);
    if (t->sizes() != shape) refuse(std::string(name) + " is " + shape_of(t->sizes()) + ", not " + shape_of(shape));
    if (!t->is_contiguous()) refuse(std::string(name) + " is not contiguous");
    return t->data_ptr();
  }
  void* array(PyObject* o, const char* name, at::ScalarType want, at::IntArrayRef shape) const {
    return array(tensor(o, name), name, want, shape);
  }
  moe_rows rows(const at::Tensor* t, const char* name, at::ScalarType want, int64_t n, int64_t cols) const {
    if (!t) return {nullptr, 0};
    type(*t, name, want);
    if (t->dim() != 2 || t->size(0) != n || t->size(1) != cols)
      refuse(std::string(name) + " is " + shape_of(t->sizes()) + ", not " + shape_of({n, cols}));
    if (t->is_contiguous()) return {t->data_ptr(), 0};
    if ((cols > 1 && t->stride(1) != 1) || (n > 1 && t->stride(0) < cols))
      refuse(std::string(name) + " has strides " + shape_of(t->strides()) +
             ": rows must be contiguous and must not overlap");
    return {t->data_ptr(), n > 1 ? t->stride(0) : 0};
  }
  moe_rows rows(PyObject* o, const char* name, at::ScalarType want, int64_t n, int64_t cols) const {
    return rows(tensor(o, name), name, want, n, cols);
  }
  void workspace(PyObject* o, void** data, size_t* bytes) const {
    const at::Tensor* t = tensor(o, "workspace");
    *data = array(t, "workspace", at::kByte, t ? t->sizes() : at::IntArrayRef());
    *bytes = t ? (size_t)t->numel() : 0;
  }
  moe_stream_t stream(PyObject* o) const {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    PyObject* h = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!h) throw Raised();
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised();
    return p;
  }
  int32_t i32(int64_t v, const char* name) const {
    if (v > INT32_MAX) raise(MOE_ERR_UNSUPPORTED, where, std::string(name) + " does not fit 32 bits");
    return (int32_t)v;
  }
  PyObject* done(moe_status st) const {
    if (st != MOE_OK) raise(st, where, moe_nvfp4_status_string(st));
    Py_RETURN_NONE;
  }
};

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return (float)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

// Runs `body` with n arguments expected; C++ errors become Python ones.
template <typename Body>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, Body&& body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

at::ScalarType scalar_type(int32_t dtype) { return dtype == MOE_DTYPE_BF16 ? at::kBFloat16 : at::kFloat; }

// A gate [hidden] of type par, [n, 1] fp32 or [n, hidden] of type act.
int32_t gate_rows(const Call& c, const at::Tensor* t, const char* name, int64_t n, int64_t hidden, at::ScalarType act,
                  at::ScalarType par, moe_rows* out) {
  *out = {nullptr, 0};
  if (!t) return MOE_GATE_NONE;
  if (t->dim() == 1) {
    out->data = c.array(t, name, par, {hidden});
    return MOE_GATE_CHANNEL;
  }
  if (t->dim() == 2 && t->size(1) == 1) {
    out->data = c.array(t, name, at::kFloat, {n, 1});
    return MOE_GATE_TOKEN;
  }
  *out = c.rows(t, name, act, n, hidden);
  return MOE_GATE_FULL;
}

// What both norm calls share: args[0..]: branch, gate, post_weight, pre_weight, rstd_post, rstd_pre.
moe_block_norm_args norm_args(const Call& c, int64_t n, int64_t hidden, int32_t res, PyObject* branch, PyObject* gate,
                              PyObject* post, PyObject* pre, PyObject* rstd_post, PyObject* rstd_pre,
                              PyObject* const* scalars) {
  moe_block_norm_args a = {};
  a.n = c.i32(n, "n");
  a.hidden = c.i32(hidden, "hidden");
  a.residual_dtype = res;
  const at::Tensor *tb = c.tensor(branch, "branch"), *tg = c.tensor(gate, "gate"), *tp = c.tensor(post, "post_weight"),
                   *tq = c.tensor(pre, "pre_weight");
  a.branch_dtype = tb ? c.dtype(*tb, "branch") : res;
  const at::Tensor* par = tp ? tp : tq ? tq : tg && tg->dim() == 1 ? tg : nullptr;
  a.param_dtype = par ? c.dtype(*par, "the weights") : MOE_DTYPE_F32;
  const at::ScalarType act_t = scalar_type(a.branch_dtype), par_t = scalar_type(a.param_dtype);
  a.gate_kind = gate_rows(c, tg, "gate", n, hidden, act_t, par_t, &a.gate);
  a.eps = number(scalars[0]);
  a.residual_scale = number(scalars[1]);
  a.branch_scale = number(scalars[2]);
  a.weight_offset = number(scalars[3]);
  a.gate_sigmoid = a.gate_kind != MOE_GATE_NONE && truth(scalars[4]);
  a.branch = c.rows(tb, "branch", act_t, n, hidden);
  a.post_weight = c.array(tp, "post_weight", par_t, {hidden});
  a.pre_weight = c.array(tq, "pre_weight", par_t, {hidden});
  a.rstd_post = static_cast<float*>(c.array(rstd_post, "rstd_post", at::kFloat, {n}));
  a.rstd_pre = static_cast<float*>(c.array(rstd_pre, "rstd_pre", at::kFloat, {n}));
  return a;
}

// residual, branch, gate, post_weight, pre_weight, residual_out, x_out, rstd_post, rstd_pre, eps, residual_scale,
// branch_scale, weight_offset, gate_sigmoid, stream
PyObject* block_norm(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 15, [&] {
    Call c{"moe_block_norm"};
    const at::Tensor* r = c.tensor(p[0], "residual");
    if (!r || r->dim() != 2) c.refuse("residual is not an [n, hidden] tensor");
    c.lead(*r);
    const int64_t n = r->size(0), hidden = r->size(1);
    const int32_t res = c.dtype(*r, "residual");
    moe_block_norm_args a = norm_args(c, n, hidden, res, p[1], p[2], p[3], p[4], p[7], p[8], p + 9);
    a.residual = c.rows(r, "residual", scalar_type(res), n, hidden);
    a.residual_out = c.rows(p[5], "residual_out", scalar_type(res), n, hidden);
    a.x_out = c.rows(p[6], "x_out", at::kBFloat16, n, hidden);
    return c.done(moe_block_norm(&a, c.stream(p[14])));
  });
}

// d_residual_out, d_x, residual_out, branch, gate, post_weight, pre_weight, rstd_post, rstd_pre, d_residual, d_branch,
// d_gate, d_post_weight, d_pre_weight, eps, residual_scale, branch_scale, weight_offset, gate_sigmoid, workspace, stream
PyObject* block_norm_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 21, [&] {
    Call c{"moe_block_norm_backward"};
    const at::Tensor *dr = c.tensor(p[0], "d_residual_out"), *u = c.tensor(p[2], "residual_out");
    const at::Tensor* lead = dr ? dr : u ? u : c.tensor(p[3], "branch");
    if (!lead || lead->dim() != 2) c.refuse("no [n, hidden] gradient is given");
    c.lead(*lead);
    const int64_t n = lead->size(0), hidden = lead->size(1);
    const int32_t res = c.dtype(*lead, "the residual");
    moe_block_norm_args a = norm_args(c, n, hidden, res, p[3], p[4], p[5], p[6], p[7], p[8], p + 14);
    const at::ScalarType res_t = scalar_type(res), act_t = scalar_type(a.branch_dtype);
    a.residual_out = c.rows(u, "residual_out", res_t, n, hidden);
    moe_block_norm_grads d = {};
    const at::Tensor* dg = c.tensor(p[11], "d_gate");
    const int32_t kind = gate_rows(c, dg, "d_gate", n, hidden, act_t, at::kFloat, &d.d_gate);
    if (dg && kind != a.gate_kind) c.refuse("d_gate is " + shape_of(dg->sizes()) + ", the gate another shape");
    d.d_residual_out = c.rows(dr, "d_residual_out", res_t, n, hidden);
    d.d_x = c.rows(p[1], "d_x", at::kBFloat16, n, hidden);
    d.d_residual = c.rows(p[9], "d_residual", res_t, n, hidden);
    d.d_branch = c.rows(p[10], "d_branch", act_t, n, hidden);
    d.d_post_weight = static_cast<float*>(c.array(p[12], "d_post_weight", at::kFloat, {hidden}));
    d.d_pre_weight = static_cast<float*>(c.array(p[13], "d_pre_weight", at::kFloat, {hidden}));
    void* ws;
    size_t bytes;
    c.workspace(p[19], &ws, &bytes);
    return c.done(moe_block_norm_backward(&a, &d, ws, bytes, c.stream(p[20])));
  });
}

// The arguments that both router calls share; S is read from seq_offsets.
moe_router_args router_args(Call& c, PyObject* logits, PyObject* bias, PyObject* ids, PyObject* counts, PyObject* tokens,
                            PyObject* coef, PyObject* mask, PyObject* seq) {
  const at::Tensor *z = c.tensor(logits, "logits"), *t = c.tensor(ids, "topk_ids"), *m = c.tensor(mask, "mask"),
                   *s = c.tensor(seq, "seq_offsets");
  if (!z || z->dim() != 2 || !t || t->dim() != 2) c.refuse("logits are not [n, n_experts] or topk_ids not [n, top_k]");
  c.lead(*z);
  const int64_t n = z->size(0), E = z->size(1), k = t->size(1);
  int64_t S = 1;
  if (s) {
    S = s->dim() == 1 ? s->size(0) - 1 : 0;
    if (S < 1) c.refuse("seq_offsets holds no sequence");
  }
  moe_router_args a = {};
  a.n = c.i32(n, "n");
  a.n_experts = c.i32(E, "n_experts");
  a.top_k = c.i32(k, "top_k");
  a.n_seqs = c.i32(S, "n_seqs");
  a.coef = number(coef);
  a.logits = static_cast<float*>(c.array(z, "logits", at::kFloat, {n, E}));
  a.bias = static_cast<float*>(c.array(bias, "bias", at::kFloat, {E}));
  a.topk_ids = static_cast<int32_t*>(c.array(t, "topk_ids", at::kInt, {n, k}));
  const at::ScalarType bytes = m && m->scalar_type() == at::kBool ? at::kBool : at::kByte;
  a.token_mask = static_cast<uint8_t*>(c.array(m, "mask", bytes, {n}));
  a.seq_offsets = static_cast<int32_t*>(c.array(s, "seq_offsets", at::kInt, {S + 1}));
  a.counts = static_cast<int32_t*>(c.array(counts, "counts", at::kInt, {S, E}));
  a.tokens = static_cast<int32_t*>(c.array(tokens, "tokens", at::kInt, {S + 1}));
  return a;
}

// logits, bias, topk_ids, loss, counts, prob_sums, tokens, coef, mask, seq_offsets, workspace, stream
PyObject* balance_loss(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 12, [&] {
    Call c{"moe_balance_loss"};
    const moe_router_args a = router_args(c, p[0], p[1], p[2], p[4], p[6], p[7], p[8], p[9]);
    float* sums = static_cast<float*>(c.array(p[5], "prob_sums", at::kFloat, {a.n_seqs, a.n_experts}));
    float* loss = static_cast<float*>(c.array(p[3], "loss", at::kFloat, {1}));
    void* ws;
    size_t bytes;
    c.workspace(p[10], &ws, &bytes);
    return c.done(moe_balance_loss(&a, sums, loss, ws, bytes, c.stream(p[11])));
  });
}

// logits, bias, topk_ids, topk_weights, d_weights, counts, tokens, d_logits, d_bias, d_loss, coef, mask, seq_offsets,
// workspace, stream
PyObject* router_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 15, [&] {
    Call c{"moe_router_backward"};
    const moe_router_args a = router_args(c, p[0], p[1], p[2], p[5], p[6], p[10], p[11], p[12]);
    const at::ScalarType f = at::kFloat;
    auto* w = static_cast<const float*>(c.array(p[3], "topk_weights", f, {a.n, a.top_k}));
    auto* dw = static_cast<const float*>(c.array(p[4], "d_weights", f, {a.n, a.top_k}));
    auto* dl = static_cast<const float*>(c.array(p[9], "d_loss", f, {1}));
    auto* dz = static_cast<float*>(c.array(p[7], "d_logits", f, {a.n, a.n_experts}));
    auto* db = static_cast<float*>(c.array(p[8], "d_bias", f, {a.n_experts}));
    void* ws;
    size_t bytes;
    c.workspace(p[13], &ws, &bytes);
    return c.done(moe_router_backward(&a, w, dw, dl, dz, db, ws, bytes, c.stream(p[14])));
  });
}

// x, adapter_ids, a, b, y, out, scale, ranks, workspace, stream
PyObject* lora_apply(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 10, [&] {
    Call c{"moe_lora_apply"};
    const at::Tensor *x = c.tensor(p[0], "x"), *A = c.tensor(p[2], "a"), *B = c.tensor(p[3], "b"),
                     *y = c.tensor(p[4], "y"), *out = c.tensor(p[5], "out");
    if (!x || x->dim() != 2 || !A || A->dim() != 3 || !B || B->dim() != 3 || !out)
      c.refuse("x is not [n, in], a not [L, R, in], b not [L, out, R], or out is missing");
    c.lead(*x);
    const int64_t n = x->size(0), in = x->size(1), L = A->size(0), R = A->size(1), o = B->size(1);
    moe_lora_args a = {};
    a.n = c.i32(n, "n");
    a.in_features = c.i32(in, "in");
    a.out_features = c.i32(o, "out");
    a.n_adapters = c.i32(L, "L");
    a.max_rank = c.i32(R, "R");
    a.y_dtype = y ? c.dtype(*y, "y") : MOE_DTYPE_BF16;
    a.out_dtype = c.dtype(*out, "out");
    const at::ScalarType bf = at::kBFloat16;
    a.a = static_cast<uint16_t*>(c.array(A, "a", bf, {L, R, in}));
    a.b = static_cast<uint16_t*>(c.array(B, "b", bf, {L, o, R}));
    a.scale = static_cast<float*>(c.array(p[6], "scale", at::kFloat, {L}));
    a.ranks = static_cast<int32_t*>(c.array(p[7], "ranks", at::kInt, {L}));
    a.adapter_ids = static_cast<int32_t*>(c.array(p[1], "adapter_ids", at::kInt, {n}));
    if (n > 0 && !a.adapter_ids) c.refuse("adapter_ids is missing");
    a.x = c.rows(x, "x", bf, n, in);
    a.y = c.rows(y, "y", scalar_type(a.y_dtype), n, o);
    a.out = c.rows(out, "out", scalar_type(a.out_dtype), n, o);
    void* ws;
    size_t bytes;
    c.workspace(p[8], &ws, &bytes);
    return c.done(moe_lora_apply(&a, ws, bytes, c.stream(p[9])));
  });
}

// n heads of [n, heads, dim] as rows: heads contiguous, tokens at any stride.
moe_rows heads(const Call& c, const at::Tensor* t, const char* name, at::ScalarType want, int64_t n, int64_t count,
               int64_t dim) {
  if (!t) return {nullptr, 0};
  c.type(*t, name, want);
  if (t->dim() != 3 || t->size(0) != n || t->size(1) != count || t->size(2) != dim)
    c.refuse(std::string(name) + " is " + shape_of(t->sizes()) + ", not " + shape_of({n, count, dim}));
  if (t->is_contiguous()) return {t->data_ptr(), 0};
  if ((dim > 1 && t->stride(2) != 1) || (count > 1 && t->stride(1) != dim) || (n > 1 && t->stride(0) < count * dim))
    c.refuse(std::string(name) + " has strides " + shape_of(t->strides()) +
             ": a token's heads must be contiguous and must not overlap");
  return {t->data_ptr(), n > 1 ? t->stride(0) : 0};
}

// What both calls share.  q, k: the inputs, or the tensors that stand for their shapes.  scalars: eps, weight_offset,
// rotary_scale, sections, sections_interleaved, pairs_interleaved.
moe_qk_args qk_args(Call& c, const at::Tensor* q, const at::Tensor* k, PyObject* positions, PyObject* inv_freq,
                    PyObject* q_weight, PyObject* k_weight, PyObject* const* scalars) {
  const at::Tensor* lead = q ? q : k;
  if (!lead || (q && q->dim() != 3) || (k && k->dim() != 3)) c.refuse("q and k are not [n, heads, head_dim] tensors");
  c.lead(*lead);
  moe_qk_args a = {};
  a.n = c.i32(lead->size(0), "n");
  a.head_dim = c.i32(lead->size(2), "head_dim");
  a.q_heads = q ? c.i32(q->size(1), "q_heads") : 0;
  a.k_heads = k ? c.i32(k->size(1), "k_heads") : 0;
  a.dtype = c.dtype(*lead, q ? "q" : "k");
  const at::Tensor *pos = c.tensor(positions, "positions"), *freq = c.tensor(inv_freq, "inv_freq"),
                   *qw = c.tensor(q_weight, "q_weight"), *kw = c.tensor(k_weight, "k_weight");
  if ((pos != nullptr) != (freq != nullptr)) c.refuse("positions and inv_freq go together");
  a.n_axes = 1;
  if (pos) {
    if (freq->dim() != 1) c.refuse("inv_freq is not [rotary_dim / 2]");
    a.rotary_dim = c.i32(2 * freq->size(0), "rotary_dim");
    a.inv_freq = static_cast<float*>(c.array(freq, "inv_freq", at::kFloat, freq->sizes()));
    if (pos->dim() == 2) a.n_axes = c.i32(pos->size(0), "axes");
    if (pos->dim() == 2)
      a.positions = static_cast<int32_t*>(c.array(pos, "positions", at::kInt, {a.n_axes, a.n}));
    else
      a.positions = static_cast<int32_t*>(c.array(pos, "positions", at::kInt, {a.n}));
  }
  if (scalars[3] != Py_None) {
    PyObject* seq = PySequence_Fast(scalars[3], "sections is not a sequence");
    if (!seq) throw Raised();
    const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
    bool fits = len == a.n_axes && len <= MOE_MAX_AXES;
    for (Py_ssize_t i = 0; fits && i < len; ++i) {
      const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
      if (v == -1 && PyErr_Occurred()) {
        Py_DECREF(seq);
        throw Raised();
      }
      fits = v >= 0 && v <= INT32_MAX;
      a.sections[i] = (int32_t)v;
    }
    Py_DECREF(seq);
    if (!fits) c.refuse("sections does not hold one number of pairs for each axis of positions");
    if (pos && len == 1 && a.sections[0] != a.rotary_dim / 2) c.refuse("sections does not add up to the pairs");
  } else if (a.n_axes > 1) {
    c.refuse("several axes of positions need sections");
  }
  const at::Tensor* par = qw ? qw : kw;
  a.param_dtype = par ? c.dtype(*par, "the weights") : MOE_DTYPE_F32;
  a.q_weight = c.array(qw, "q_weight", scalar_type(a.param_dtype), {a.head_dim});
  a.k_weight = c.array(kw, "k_weight", scalar_type(a.param_dtype), {a.head_dim});
  a.eps = number(scalars[0]);
  a.weight_offset = number(scalars[1]);
  a.rotary_scale = number(scalars[2]);
  a.sections_interleaved = truth(scalars[4]);
  a.pairs_interleaved = truth(scalars[5]);
  const at::ScalarType t = scalar_type(a.dtype);
  a.q = heads(c, q, "q", t, a.n, a.q_heads, a.head_dim);
  a.k = heads(c, k, "k", t, a.n, a.k_heads, a.head_dim);
  return a;
}

// q, k, q_out, k_out, positions, inv_freq, q_weight, k_weight, eps, weight_offset, rotary_scale, sections,
// sections_interleaved, pairs_interleaved, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 15, [&] {
    Call c{"moe_qk_norm_rope"};
    moe_qk_args a = qk_args(c, c.tensor(p[0], "q"), c.tensor(p[1], "k"), p[4], p[5], p[6], p[7], p + 8);
    const at::ScalarType t = scalar_type(a.dtype);
    a.q_out = heads(c, c.tensor(p[2], "q_out"), "q_out", t, a.n, a.q_heads, a.head_dim);
    a.k_out = heads(c, c.tensor(p[3], "k_out"), "k_out", t, a.n, a.k_heads, a.head_dim);
    return c.done(moe_qk_norm_rope(&a, c.stream(p[14])));
  });
}

// d_q_out, d_k_out, q, k, d_q, d_k, positions, inv_freq, q_weight, k_weight, d_q_weight, d_k_weight, eps,
// weight_offset, rotary_scale, sections, sections_interleaved, pairs_interleaved, workspace, stream
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 20, [&] {
    Call c{"moe_qk_norm_rope_backward"};
    const at::Tensor *dq = c.tensor(p[0], "d_q_out"), *dk = c.tensor(p[1], "d_k_out"), *q = c.tensor(p[2], "q"),
                     *k = c.tensor(p[3], "k");
    moe_qk_args a = qk_args(c, q ? q : dq, k ? k : dk, p[6], p[7], p[8], p[9], p + 12);
    if (!q) a.q.data = nullptr;
    if (!k) a.k.data = nullptr;
    const at::ScalarType t = scalar_type(a.dtype);
    moe_qk_grads d = {};
    d.d_q_out = heads(c, dq, "d_q_out", t, a.n, a.q_heads, a.head_dim);
    d.d_k_out = heads(c, dk, "d_k_out", t, a.n, a.k_heads, a.head_dim);
    d.d_q = heads(c, c.tensor(p[4], "d_q"), "d_q", t, a.n, a.q_heads, a.head_dim);
    d.d_k = heads(c, c.tensor(p[5], "d_k"), "d_k", t, a.n, a.k_heads, a.head_dim);
    d.d_q_weight = static_cast<float*>(c.array(p[10], "d_q_weight", at::kFloat, {a.head_dim}));
    d.d_k_weight = static_cast<float*>(c.array(p[11], "d_k_weight", at::kFloat, {a.head_dim}));
    void* ws;
    size_t bytes;
    c.workspace(p[18], &ws, &bytes);
    return c.done(moe_qk_norm_rope_backward(&a, &d, ws, bytes, c.stream(p[19])));
  });
}

// What both projection calls share: sizes, weight, x, z and the activation.
moe_linear_args linear_args(Call& c, const at::Tensor* lead, const at::Tensor* x, const at::Tensor* w,
                            const at::Tensor* z, PyObject* activation) {
  if (!lead || lead->dim() != 2 || !w || w->dim() != 2) c.refuse("no [n, features] tensor, or weight is not [out, in]");
  c.lead(*lead);
  moe_linear_args a = {};
  a.n = c.i32(lead->size(0), "n");
  a.in_features = c.i32(w->size(1), "in");
  a.out_features = c.i32(w->size(0), "out");
  const long act = PyLong_AsLong(activation);
  if (act == -1 && PyErr_Occurred()) throw Raised();
  a.activation = (int32_t)act;
  a.weight = static_cast<uint16_t*>(c.array(w, "weight", at::kBFloat16, w->sizes()));
  a.x = c.rows(x, "x", at::kBFloat16, a.n, a.in_features);
  a.z_dtype = z ? c.dtype(*z, "z") : MOE_DTYPE_BF16;
  a.z = c.rows(z, "z", scalar_type(a.z_dtype), a.n, a.out_features);
  return a;
}

// x, weight, out, bias, residual, z_out, activation, residual_scale, stream
PyObject* linear(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 9, [&] {
    Call c{"moe_linear"};
    const at::Tensor *x = c.tensor(p[0], "x"), *out = c.tensor(p[2], "out"), *bias = c.tensor(p[3], "bias"),
                     *res = c.tensor(p[4], "residual");
    moe_linear_args a = linear_args(c, x, x, c.tensor(p[1], "weight"), c.tensor(p[5], "z_out"), p[6]);
    if (!out) c.refuse("out is missing");
    a.out_dtype = c.dtype(*out, "out");
    a.out = c.rows(out, "out", scalar_type(a.out_dtype), a.n, a.out_features);
    a.bias_dtype = bias ? c.dtype(*bias, "bias") : MOE_DTYPE_F32;
    a.bias = c.array(bias, "bias", scalar_type(a.bias_dtype), {a.out_features});
    a.residual_dtype = res ? c.dtype(*res, "residual") : MOE_DTYPE_BF16;
    a.residual = c.rows(res, "residual", scalar_type(a.residual_dtype), a.n, a.out_features);
    a.residual_scale = number(p[7]);
    return c.done(moe_linear(&a, c.stream(p[8])));
  });
}

// d_out, x, weight, z, d_x, d_weight, d_bias, activation, workspace, stream
PyObject* linear_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 10, [&] {
    Call c{"moe_linear_backward"};
    const at::Tensor *dy = c.tensor(p[0], "d_out"), *x = c.tensor(p[1], "x"), *w = c.tensor(p[2], "weight"),
                     *z = c.tensor(p[3], "z"), *dx = c.tensor(p[4], "d_x"), *dw = c.tensor(p[5], "d_weight");
    moe_linear_args a = linear_args(c, dy, x, w, z, p[7]);
    moe_linear_grads d = {};
    d.d_out_dtype = c.dtype(*dy, "d_out");
    d.d_x_dtype = dx ? c.dtype(*dx, "d_x") : MOE_DTYPE_BF16;
    d.d_weight_dtype = dw ? c.dtype(*dw, "d_weight") : MOE_DTYPE_BF16;
    d.d_out = c.rows(dy, "d_out", scalar_type(d.d_out_dtype), a.n, a.out_features);
    d.d_x = c.rows(dx, "d_x", scalar_type(d.d_x_dtype), a.n, a.in_features);
    d.d_weight = c.array(dw, "d_weight", scalar_type(d.d_weight_dtype), {a.out_features, a.in_features});
    d.d_bias = static_cast<float*>(c.array(p[6], "d_bias", at::kFloat, {a.out_features}));
    void* ws;
    size_t bytes;
    c.workspace(p[8], &ws, &bytes);
    return c.done(moe_linear_backward(&a, &d, ws, bytes, c.stream(p[9])));
  });
}

// handle, hidden, n_experts, top_k, x, router_weight, dst, residual, router_bias, shared_experts, topk_ids, topk_weights,
// logits, stream
PyObject* layer_forward(PyObject*, PyObject* const* p, Py_ssize_t count) {
  return guarded(count, 14, [&] {
    Call c{"moe_nvfp4_layer_forward"};
    int64_t v[5] = {};
    PyObject* const ints[5] = {p[0], p[1], p[2], p[3], p[9]};
    for (int i = 0; i < 5; ++i) {
      if (i == 0 && ints[i] == Py_None) c.refuse("the layer is closed");
      v[i] = PyLong_AsLongLong(ints[i]);
      if (v[i] == -1 && PyErr_Occurred()) throw Raised();
    }
    const int64_t H = v[1], S = v[4], E = v[2] - S, k = v[3] - S;
    if (S < 0 || k < 1 || E < k) c.refuse("shared_experts leaves no routed experts to pick from");
    const at::Tensor *x = c.tensor(p[4], "x"), *w = c.tensor(p[5], "router_weight");
    if (!x || x->dim() != 2 || !w) c.refuse("x is not [n, hidden], or router_weight is missing");
    c.lead(*x);
    const int64_t n = x->size(0);
    moe_layer_args a = {};
    a.n_tokens = c.i32(n, "n");
    a.shared_experts = (int32_t)S;
    a.router_dtype = c.dtype(*w, "router_weight");
    a.x = static_cast<uint16_t*>(c.array(x, "x", at::kBFloat16, {n, H}));
    a.router_weight = c.array(w, "router_weight", scalar_type(a.router_dtype), {E, H});
    a.dst = static_cast<uint16_t*>(c.array(p[6], "dst", at::kBFloat16, {n, H}));
    a.residual = static_cast<uint16_t*>(c.array(p[7], "residual", at::kBFloat16, {n, H}));
    a.router_bias = static_cast<float*>(c.array(p[8], "router_bias", at::kFloat, {E}));
    a.topk_ids = static_cast<int32_t*>(c.array(p[10], "topk_ids", at::kInt, {n, k}));
    a.topk_weights = static_cast<float*>(c.array(p[11], "topk_weights", at::kFloat, {n, k}));
    a.logits = static_cast<float*>(c.array(p[12], "logits", at::kFloat, {n, E}));
    return c.done(moe_nvfp4_layer_forward(reinterpret_cast<moe_nvfp4_t>(v[0]), &a, c.stream(p[13])));
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

#define FAST(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {FAST(block_norm),
                          FAST(block_norm_backward),
                          FAST(balance_loss),
                          FAST(router_backward),
                          FAST(lora_apply),
                          FAST(linear),
                          FAST(linear_backward),
                          FAST(layer_forward),
                          FAST(qk_norm_rope),
                          FAST(qk_norm_rope_backward),
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "moe_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_moe_binding() { return PyModule_Create(&kModule); }
