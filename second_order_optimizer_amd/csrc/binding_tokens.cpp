// Calls of include/kfac_tokens.h and include/kfac_orthogonal.h on torch tensors
// (the _tokens extension), in the manner of binding.cpp: each function takes the
// address of an operator's plan, mirrored by tokens.py and orthogonal.py, and
// tensors or None, runs on the device's current stream and returns the outputs.
#include "binding.h"
#include "overlap.h"

#include "../../include/kfac_orthogonal.h"
#include "../../include/kfac_tokens.h"

#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/variable.h>

namespace {

struct SamplePlan {
  Plan base;
  kfac_sample_t s;
};
struct EmbeddingPlan {
  Plan base;
  kfac_embedding_t e;
};
struct OrthogonalPlan {
  Plan base;
  kfac_orthogonal_matrix_t m;
  kfac_orthogonal_t how;
};
struct StepPlan {
  Plan base;
  kfac_layer_t* layers;        // kept by the operator, pointers set per call
  PyObject* weights;           // list of the tensors that a step writes: weights, momenta, biases, bias momenta
                               // (of the layers that have them)
  int64_t n;
  kfac_orthogonal_t how;
  kfac_hparams_t hp;
};

struct Entries {
  decltype(&kfac_sample_tokens) sample;
  decltype(&kfac_embedding_lookup) lookup;
  decltype(&kfac_embedding_grad) grad;
  decltype(&kfac_orthogonalize) orthogonalize;
  decltype(&kfac_step_orthogonal) step;
};
Entries entries{};

// (plan, logits, u, temperature, top_k, top_p, min_p) -> (token, logp, kept)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const SamplePlan* plan = plan_of<SamplePlan>(a, n, 7);
    Call c(plan->base);
    kfac_sample_t s = plan->s;
    s.logits = c.matrix(c.tensor(a[1], "logits"), "logits", s.rows, s.vocab, &s.ld);
    s.u = static_cast<const float*>(c.vector(a[2], "u", s.rows, at::kFloat));
    s.row_temperature = c.floats(a[3], "temperature", s.rows);
    if (a[4] != Py_None) s.row_top_k = static_cast<const int32_t*>(c.vector(a[4], "top_k", s.rows, at::kInt));
    s.row_top_p = c.floats(a[5], "top_p", s.rows);
    s.row_min_p = c.floats(a[6], "min_p", s.rows);
    void* stream = c.enter();
    at::Tensor token = c.make(s.rows, at::kLong), logp = c.make(s.rows), kept = c.make(s.rows, at::kInt);
    s.token = token.data_ptr<int64_t>();
    s.logp = logp.data_ptr<float>();
    s.kept = kept.data_ptr<int32_t>();
    done(entries.sample(&s, plan->base.ws, plan->base.ws_bytes, stream), "kfac_sample_tokens");
    return tuple_of({token, logp, kept});
  });
}

// The memory of a tensor that has passed its checks: adjacent columns.
kfac::Lines lines_of(const at::Tensor& t) {
  const int64_t el = t.element_size(), d = t.dim();
  return kfac::lines_of(t.data_ptr(), t.numel() ? t.size(d - 1) * el : 0, d > 1 ? t.size(d - 2) : 1, d > 1 ? t.stride(d - 2) * el : 0,
                        d > 2 ? t.size(0) : 1, d > 2 ? t.stride(0) * el : 0);
}

// (plan, table, ids, out) -> y, or None (and nothing done) where the call belongs into autograd's graph
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const EmbeddingPlan* plan = plan_of<EmbeddingPlan>(a, n, 4);
    Call c(plan->base);
    kfac_embedding_t e = plan->e;
    const at::Tensor& table = c.differentiable(a[1], "table");
    e.table = c.matrix_of(table, "table", e.table_dtype, e.vocab, e.width, &e.table_ld);
    e.ids = c.indices(a[2], "ids", e.tokens, -1, &e.id_type);
    if (c10::GradMode::is_enabled() && table.requires_grad()) {
      if (a[3] != Py_None) c.refuse("out cannot be given where table requires grad");
      Py_RETURN_NONE;
    }
    at::Tensor y;
    if (a[3] != Py_None) {
      y = c.differentiable(a[3], "out");
      c.matrix(y, "out", e.tokens, e.width, &e.y_ld);
      const kfac::Lines to = lines_of(y);
      if (kfac::overlap(to, lines_of(table)) || kfac::overlap(to, lines_of(c.tensor(a[2], "ids"))))
        c.refuse("out must not share memory with table or ids");
    }
    const bool given = y.defined();
    void* stream = c.enter();
    if (!given) y = c.make_rows(e.tokens, e.width, e.y_ld = e.width, &e.y_ld);
    e.y = y.data_ptr();
    done(entries.lookup(&e, plan->base.ws, plan->base.ws_bytes, stream), "kfac_embedding_lookup");
    if (given) written(y);
    return THPVariable_Wrap(std::move(y));
  });
}

// (tensor) -> whether a living graph adds up its gradient on the default stream.  A leaf's gradients are added where
// the first of its living graphs was made, whatever operators they are of.
PyObject* gathers_on_default(PyObject*, PyObject* t) {
  return guarded([&]() -> PyObject* {
    if (!THPVariable_Check(t)) throw Refused{KFAC_ERR_ARG, "not a tensor"};
    const auto node = torch::autograd::impl::try_get_grad_accumulator(THPVariable_Unpack(t));
    const auto stream = node ? node->stream() : std::nullopt;
    return PyBool_FromLong(stream && stream->id() == 0);
  });
}

// (plan, dy, ids, grad, accumulate) -> (grad, counts)
PyObject* embedding_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const EmbeddingPlan* plan = plan_of<EmbeddingPlan>(a, n, 5);
    Call c(plan->base);
    kfac_embedding_t e = plan->e;
    e.y = c.matrix(c.differentiable(a[1], "dy"), "dy", e.tokens, e.width, &e.y_ld);
    e.ids = c.indices(a[2], "ids", e.tokens, -1, &e.id_type);
    at::Tensor grad;
    if (a[3] != Py_None) {
      grad = c.differentiable(a[3], "grad");
      e.table = c.matrix_of(grad, "grad", e.table_dtype, e.vocab, e.width, &e.table_ld);
      const kfac::Lines to = lines_of(grad);
      if (kfac::overlap(to, lines_of(c.tensor(a[1], "dy"))) || kfac::overlap(to, lines_of(c.tensor(a[2], "ids"))))
        c.refuse("grad must not share memory with dy or ids");
    }
    const bool given = grad.defined();
    const int accumulate = PyObject_IsTrue(a[4]);
    if (accumulate < 0) return nullptr;
    e.accumulate = accumulate;
    if (e.accumulate && !given) c.refuse("accumulate needs grad");
    void* stream = c.enter();
    at::Tensor counts = c.make(e.vocab, at::kInt);
    if (!given) {
      grad = c.make_matrix(e.vocab, e.width, e.table_dtype);
      e.table = grad.data_ptr();
      e.table_ld = e.width;
    }
    e.counts = counts.data_ptr<int32_t>();
    done(entries.grad(&e, plan->base.ws, plan->base.ws_bytes, stream), "kfac_embedding_grad");
    if (given) written(grad);
    return tuple_of({grad, counts});
  });
}

// [batch, rows, cols] of the operator's dtype (or [rows, cols] for a batch of one) with adjacent columns
void* stack_of(const Call& c, const at::Tensor& t, const char* name, const kfac_orthogonal_matrix_t& m, int64_t* ld, int64_t* stride) {
  if (t.dim() == 2 && m.batch == 1) {
    void* p = c.matrix(t, name, m.rows, m.cols, ld);
    *stride = 0;
    return p;
  }
  if (t.scalar_type() != c.dtype())
    c.refuse(std::string(name) + " must be " + (m.dtype == KFAC_BF16 ? "bfloat16" : "float32"), KFAC_ERR_DTYPE);
  if (t.dim() != 3 || t.size(0) != m.batch || t.size(1) != m.rows || t.size(2) != m.cols || !c.placed(t))
    c.refuse(std::string(name) + " must be [" + std::to_string(m.batch) + ", " + std::to_string(m.rows) + ", " +
             std::to_string(m.cols) + "] on " + c.place());
  *ld = m.rows < 2 ? m.cols : t.stride(1);
  const int64_t span = (m.rows - 1) * *ld + m.cols;
  *stride = m.batch < 2 ? span : t.stride(0);
  if ((t.stride(2) != 1 && m.cols > 1) || *ld < m.cols || *stride < span)
    c.refuse(std::string(name) + " must have adjacent columns, and rows and matrices that do not overlap");
  return t.data_ptr();
}

// (plan, x, out) -> y
PyObject* orthogonalize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const OrthogonalPlan* plan = plan_of<OrthogonalPlan>(a, n, 3);
    Call c(plan->base);
    kfac_orthogonal_matrix_t m = plan->m;
    const at::Tensor& x = c.tensor(a[1], "x");
    m.x = stack_of(c, x, "x", m, &m.ld, &m.stride);
    at::Tensor y;
    if (a[2] != Py_None) {
      y = c.tensor(a[2], "out");
      m.y = stack_of(c, y, "out", m, &m.y_ld, &m.y_stride);
      const bool same = m.y == m.x && m.y_ld == m.ld && (m.batch < 2 || m.y_stride == m.stride);
      if (!same && kfac::overlap(lines_of(y), lines_of(x))) c.refuse("out must be x itself, or share no memory with it");
    }
    const bool given = y.defined();
    void* stream = c.enter();
    if (!given) {
      y = c.make_like(x.sizes(), m.dtype);
      m.y = y.data_ptr();
      m.y_ld = m.cols;
      m.y_stride = static_cast<int64_t>(m.rows) * m.cols;
    }
    done(entries.orthogonalize(&m, &plan->how, plan->base.ws, plan->base.ws_bytes, stream), "kfac_orthogonalize");
    if (given) written(y);
    return THPVariable_Wrap(std::move(y));
  });
}

// (plan, gradients, bias gradients or None, lr, momentum, weight_decay) -> None
PyObject* orthogonal_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const StepPlan* plan = plan_of<StepPlan>(a, n, 6);
    Call c(plan->base);
    kfac_hparams_t hp = plan->hp;
    float* to[3] = {&hp.lr, &hp.momentum, &hp.weight_decay};
    for (int i = 0; i < 3; ++i) *to[i] = static_cast<float>(PyFloat_AsDouble(a[3 + i]));
    if (PyErr_Occurred()) return nullptr;
    // The tensors are the operator's own, but a program may have given them other memory (w.data = v): what they
    // hold now is what is written.
    Py_ssize_t next = 0;
    auto kept = [&] { return PyList_GET_ITEM(plan->weights, next++); };
    auto square = [&](const kfac_layer_t& L, const char* name) {
      int64_t ld;
      float* p = static_cast<float*>(c.matrix(THPVariable_Unpack(kept()), name, L.d_out, L.d_in, &ld));
      if (ld != L.d_in) c.refuse(std::string(name) + " must be contiguous");
      return p;
    };
    for (int64_t i = 0; i < plan->n; ++i) plan->layers[i].w = square(plan->layers[i], "a weight");
    for (int64_t i = 0; i < plan->n; ++i) plan->layers[i].mom_w = square(plan->layers[i], "a momentum");
    for (int64_t i = 0; i < plan->n; ++i)
      if (plan->layers[i].has_bias) plan->layers[i].b = c.floats(kept(), "a bias", plan->layers[i].d_out);
    for (int64_t i = 0; i < plan->n; ++i)
      if (plan->layers[i].has_bias) plan->layers[i].mom_b = c.floats(kept(), "a bias momentum", plan->layers[i].d_out);
    for (int which = 0; which < 2; ++which) {
      const char* name = which ? "bias_grads" : "grads";
      PyObject* list = a[1 + which];
      if (which == 1 && list == Py_None) {
        for (int64_t i = 0; i < plan->n; ++i)
          if (plan->layers[i].has_bias) c.refuse("bias_grads is missing");
        continue;
      }
      if (!(PyList_Check(list) || PyTuple_Check(list)) || PySequence_Fast_GET_SIZE(list) != plan->n)
        c.refuse(std::string(name) + " must be a list of " + std::to_string(plan->n) + " tensors");
      for (int64_t i = 0; i < plan->n; ++i) {
        kfac_layer_t& L = plan->layers[i];
        PyObject* o = PySequence_Fast_GET_ITEM(list, i);
        if (which == 0) {
          const at::Tensor& g = c.tensor(o, name);
          int64_t ld;
          L.grad_w = static_cast<const float*>(c.matrix(g, name, L.d_out, L.d_in, &ld));
          if (ld != L.d_in) c.refuse("grads must be contiguous");
        } else if (L.has_bias) {
          L.grad_b = static_cast<const float*>(c.vector(o, name, L.d_out, at::kFloat));
        } else if (o != Py_None) {
          c.refuse("bias_grads must be None for a layer without bias");
        }
      }
    }
    if (kfac::step_shares_memory(plan->layers, plan->n))
      c.refuse("weights, momenta and biases must not share memory, and no gradient may share theirs");
    void* stream = c.enter();
    done(entries.step(plan->layers, static_cast<int32_t>(plan->n), &hp, &plan->how, plan->base.ws, plan->base.ws_bytes, stream),
         "kfac_step_orthogonal");
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(plan->weights); ++i) written(THPVariable_Unpack(PyList_GET_ITEM(plan->weights, i)));
    Py_RETURN_NONE;
  });
}

// bind(error class, five entry points): once, before any call.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes the error class and five addresses");
    return nullptr;
  }
  void* at[5];
  for (int i = 0; i < 5; ++i) at[i] = PyLong_AsVoidPtr(a[1 + i]);
  if (PyErr_Occurred()) return nullptr;
  Py_INCREF(a[0]);
  Py_XDECREF(error_class);
  error_class = a[0];
  entries = Entries{reinterpret_cast<decltype(entries.sample)>(at[0]), reinterpret_cast<decltype(entries.lookup)>(at[1]),
                    reinterpret_cast<decltype(entries.grad)>(at[2]), reinterpret_cast<decltype(entries.orthogonalize)>(at[3]),
                    reinterpret_cast<decltype(entries.step)>(at[4])};
  Py_RETURN_NONE;
}

// Sizes of the plans, for their mirrors.
PyObject* plan_sizes(PyObject*, PyObject*) {
  return Py_BuildValue("(nnnn)", static_cast<Py_ssize_t>(sizeof(SamplePlan)), static_cast<Py_ssize_t>(sizeof(EmbeddingPlan)),
                       static_cast<Py_ssize_t>(sizeof(OrthogonalPlan)), static_cast<Py_ssize_t>(sizeof(StepPlan)));
}

PyMethodDef methods[] = {{"bind", method(bind), METH_FASTCALL, nullptr},
                         {"plan_sizes", plan_sizes, METH_NOARGS, nullptr},
                         {"sample", method(sample), METH_FASTCALL, nullptr},
                         {"embedding", method(embedding), METH_FASTCALL, nullptr},
                         {"gathers_on_default", gathers_on_default, METH_O, nullptr},
                         {"embedding_grad", method(embedding_grad), METH_FASTCALL, nullptr},
                         {"orthogonalize", method(orthogonalize), METH_FASTCALL, nullptr},
                         {"orthogonal_step", method(orthogonal_step), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tokens", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tokens() { return PyModule_Create(&module); }
