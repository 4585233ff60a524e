// Calls of include/kfac_objectives.h on torch tensors: the checks of a call's
// tensors, its outputs and the C call, in one native step.  The smallest calls
// (one row of dropout, the tokens of one decoding step) take a few
// microseconds on the GPU; the same marshalling in Python took 5 us (one input
// matrix) to 12 us (seven tensors) a call.
//
// Each function takes the address of an operator's plan (the structures below,
// mirrored by second_order_optimizer_amd/objectives.py) and tensors or None,
// runs on the device's current stream and returns the outputs.  A tensor that
// does not fit raises KfacError through the class given to bind(), before
// anything is allocated or enqueued.
#include "binding.h"

namespace {

struct TokenPlan {
  Plan base;
  kfac_token_rows_t t;
};
struct PolicyPlan {
  Plan base;
  kfac_token_rows_t t;
  kfac_policy_t p;
};
struct PreferencePlan {
  Plan base;
  kfac_token_rows_t t;
  kfac_preference_t p;
};
struct BalancePlan {
  Plan base;
  kfac_balance_t b;
};
struct DropoutPlan {
  Plan base;
  kfac_dropout_t d;
};

// The library's entry points, by the addresses bind() was given.
struct Entries {
  decltype(&kfac_token_logp) token_logp;
  decltype(&kfac_policy_loss) policy_loss;
  decltype(&kfac_preference_loss) preference_loss;
  decltype(&kfac_balance_loss) balance_loss;
  decltype(&kfac_dropout) dropout;
};
Entries entries{};
void take_rows(const Call& c, kfac_token_rows_t& t, PyObject* logits, PyObject* labels) {
  t.logits = c.matrix(c.tensor(logits, "logits"), "logits", t.rows, t.vocab, &t.ld);
  t.labels = c.indices(labels, "labels", t.rows, -1, &t.label_type);
}

// The caller's gradient tensor, checked, or none.
at::Tensor given_grad(const Call& c, PyObject* o, int64_t rows, int64_t cols, int64_t* ld) {
  if (o == Py_None) return at::Tensor();
  const at::Tensor& t = c.tensor(o, "grad");
  c.matrix(t, "grad", rows, cols, ld);
  return t;
}

// (plan, logits, labels) -> logp
PyObject* token_logp(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const TokenPlan* plan = plan_of<TokenPlan>(a, n, 3);
    Call c(plan->base);
    kfac_token_rows_t t = plan->t;
    take_rows(c, t, a[1], a[2]);
    void* stream = c.enter();
    at::Tensor logp = c.make(t.rows);
    t.logp = logp.data_ptr<float>();
    done(entries.token_logp(&t, plan->base.ws, plan->base.ws_bytes, stream), "kfac_token_logp");
    return THPVariable_Wrap(std::move(logp));
  });
}

// (plan, logits, labels, advantage, weight, old_logp, ref_logp, grad) -> (stats, logp, grad)
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const PolicyPlan* plan = plan_of<PolicyPlan>(a, n, 8);
    Call c(plan->base);
    kfac_token_rows_t t = plan->t;
    kfac_policy_t p = plan->p;
    take_rows(c, t, a[1], a[2]);
    p.advantage = static_cast<const float*>(c.vector(a[3], "advantage", t.rows, at::kFloat));
    p.weight = c.floats(a[4], "weight", t.rows);
    p.old_logp = c.floats(a[5], "old_logp", t.rows);
    p.ref_logp = c.floats(a[6], "ref_logp", t.rows);
    if (a[6] == Py_None && p.kl_coef > 0.f) c.refuse("kl_coef > 0 needs ref_logp");
    at::Tensor grad = given_grad(c, a[7], t.rows, t.vocab, &t.grad_ld);
    const bool given = grad.defined();
    void* stream = c.enter();
    at::Tensor stats = c.make(4), logp = c.make(t.rows);
    if (!given) grad = c.make_rows(t.rows, t.vocab, t.ld, &t.grad_ld);
    t.logp = logp.data_ptr<float>();
    t.grad = grad.data_ptr();
    p.stats = stats.data_ptr<float>();
    done(entries.policy_loss(&t, &p, plan->base.ws, plan->base.ws_bytes, stream), "kfac_policy_loss");
    if (given) written(grad);
    return tuple_of({stats, logp, grad});
  });
}

// (plan, logits, labels, offsets, ref_logp, pair_weight, grad) -> (stats, seq, logp, grad)
PyObject* preference_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const PreferencePlan* plan = plan_of<PreferencePlan>(a, n, 7);
    Call c(plan->base);
    kfac_token_rows_t t = plan->t;
    kfac_preference_t p = plan->p;
    const int64_t seqs = 2 * static_cast<int64_t>(p.pairs);
    take_rows(c, t, a[1], a[2]);
    p.offsets = static_cast<const int32_t*>(c.vector(a[3], "offsets", seqs + 1, at::kInt));
    p.ref_logp = c.floats(a[4], "ref_logp", t.rows);
    p.pair_weight = c.floats(a[5], "pair_weight", p.pairs);
    at::Tensor grad = given_grad(c, a[6], t.rows, t.vocab, &t.grad_ld);
    const bool given = grad.defined();
    void* stream = c.enter();
    at::Tensor stats = c.make(4), seq = c.make(seqs), logp = c.make(t.rows);
    if (!given) grad = c.make_rows(t.rows, t.vocab, t.ld, &t.grad_ld);
    t.logp = logp.data_ptr<float>();
    t.grad = grad.data_ptr();
    p.seq = seq.data_ptr<float>();
    p.stats = stats.data_ptr<float>();
    done(entries.preference_loss(&t, &p, plan->base.ws, plan->base.ws_bytes, stream), "kfac_preference_loss");
    if (given) written(grad);
    return tuple_of({stats, seq, logp, grad});
  });
}

// (plan, logits, chosen, mask, grad) -> (stats, counts, prob, grad)
PyObject* balance_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const BalancePlan* plan = plan_of<BalancePlan>(a, n, 5);
    Call c(plan->base);
    kfac_balance_t b = plan->b;
    b.logits = c.matrix(c.tensor(a[1], "logits"), "logits", b.tokens, b.experts, &b.ld);
    b.chosen = c.indices(a[2], "chosen", b.tokens, b.top_k, &b.index_type);
    b.mask = a[3] == Py_None ? nullptr : static_cast<const uint8_t*>(c.vector(a[3], "mask", b.tokens, at::kBool));
    at::Tensor grad = given_grad(c, a[4], b.tokens, b.experts, &b.grad_ld);
    const bool given = grad.defined();
    void* stream = c.enter();
    at::Tensor stats = c.make(4), counts = c.make(b.experts, at::kInt), prob = c.make(b.experts);
    if (!given) grad = c.make_rows(b.tokens, b.experts, b.ld, &b.grad_ld);
    b.stats = stats.data_ptr<float>();
    b.counts = counts.data_ptr<int32_t>();
    b.prob = prob.data_ptr<float>();
    b.grad = grad.data_ptr();
    done(entries.balance_loss(&b, plan->base.ws, plan->base.ws_bytes, stream), "kfac_balance_loss");
    if (given) written(grad);
    return tuple_of({stats, counts, prob, grad});
  });
}

// (plan, x, seed, offset, residual, out, offset_tensor) -> y, or None (and nothing
// done) where the call belongs into autograd's graph
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const DropoutPlan* plan = plan_of<DropoutPlan>(a, n, 7);
    Call c(plan->base);
    kfac_dropout_t d = plan->d;
    const at::Tensor& x = c.differentiable(a[1], "x");
    if (a[4] != Py_None) c.differentiable(a[4], "residual");
    if (c10::GradMode::is_enabled() &&
        (x.requires_grad() || (a[4] != Py_None && c.tensor(a[4], "residual").requires_grad()))) {
      if (a[5] != Py_None) c.refuse("out cannot be given where x or residual requires grad");
      Py_RETURN_NONE;
    }
    d.x = c.matrix(x, "x", d.rows, d.cols, &d.ld);
    d.seed = PyLong_AsUnsignedLongLongMask(a[2]);
    d.offset = PyLong_AsUnsignedLongLongMask(a[3]);
    if (PyErr_Occurred()) return nullptr;
    if (a[4] != Py_None) d.residual = c.matrix(c.tensor(a[4], "residual"), "residual", d.rows, d.cols, &d.residual_ld);
    at::Tensor y;
    if (a[5] != Py_None) {
      y = c.differentiable(a[5], "out");
      c.matrix(y, "out", d.rows, d.cols, &d.y_ld);
    }
    if (a[6] != Py_None) d.offset_dev = static_cast<const int64_t*>(c.vector(a[6], "offset_tensor", 1, at::kLong));
    const bool given = y.defined();
    void* stream = c.enter();
    if (!given) y = c.make_rows(d.rows, d.cols, d.y_ld = d.cols, &d.y_ld);
    d.y = y.data_ptr();
    done(entries.dropout(&d, stream), "kfac_dropout");
    if (given) written(y);
    return THPVariable_Wrap(std::move(y));
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
  entries = Entries{reinterpret_cast<decltype(entries.token_logp)>(at[0]),
                    reinterpret_cast<decltype(entries.policy_loss)>(at[1]),
                    reinterpret_cast<decltype(entries.preference_loss)>(at[2]),
                    reinterpret_cast<decltype(entries.balance_loss)>(at[3]),
                    reinterpret_cast<decltype(entries.dropout)>(at[4])};
  Py_RETURN_NONE;
}

// Sizes of the plans, for their mirrors.
PyObject* plan_sizes(PyObject*, PyObject*) {
  return Py_BuildValue("(nnnnn)", static_cast<Py_ssize_t>(sizeof(TokenPlan)), static_cast<Py_ssize_t>(sizeof(PolicyPlan)),
                       static_cast<Py_ssize_t>(sizeof(PreferencePlan)), static_cast<Py_ssize_t>(sizeof(BalancePlan)),
                       static_cast<Py_ssize_t>(sizeof(DropoutPlan)));
}

PyMethodDef methods[] = {{"bind", method(bind), METH_FASTCALL, nullptr},
                         {"plan_sizes", plan_sizes, METH_NOARGS, nullptr},
                         {"token_logp", method(token_logp), METH_FASTCALL, nullptr},
                         {"policy_loss", method(policy_loss), METH_FASTCALL, nullptr},
                         {"preference_loss", method(preference_loss), METH_FASTCALL, nullptr},
                         {"balance_loss", method(balance_loss), METH_FASTCALL, nullptr},
                         {"dropout", method(dropout), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_objectives", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__objectives() { return PyModule_Create(&module); }
