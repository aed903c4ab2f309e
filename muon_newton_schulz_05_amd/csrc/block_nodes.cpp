// block_nodes.cpp -- the operators of include/muon_block.h on torch tensors, and their autograd nodes.
//
// Outputs and workspaces come from torch's caching allocator, launches go to the current stream of the tensors' device.
// The nodes are C++ so that a backward pass runs without the interpreter: on a
// small training step (777 x 1001 float32, forward and backward) nodes in Python took 100 us of the
// host.  Shapes and types are checked by the caller (block.py, mx.py); what is checked
// here is what a wrong value would turn into an access outside a tensor.
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/extension.h>

#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>

#include <algorithm>
#include <optional>

#include "../../include/muon_block.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::Function;
using torch::autograd::variable_list;
typedef std::optional<Tensor> OptTensor;

void check(int rc, const char* what) {
  TORCH_CHECK(rc == MUON_OK, what, " failed (", rc, "): ", muon_last_error());
}
void* stream_of(const Tensor& t) {
  return c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.get_device()).stream();
}
int32_t dtype_of(const Tensor& t) { return t.scalar_type() == at::kBFloat16 ? MUON_BF16 : MUON_F32; }

// A transform's wrapper (functionalization's, a fake tensor) has no memory: a view's place in it would be an address.
void check_memory(const Tensor& t) {
  TORCH_CHECK(t.numel() == 0 || t.storage().data(),
              "a tensor has no memory: these operators cannot run under tracers and transforms");
}
// t as [rows, cols] with contiguous rows.
Tensor flat(const Tensor& t, int64_t cols) {
  check_memory(t);
  Tensor r = t;
  if (t.dim() != 2) {
    int64_t rows = 1;
    for (int64_t d = 0; d + 1 < t.dim(); ++d) rows *= t.size(d);
    r = t.reshape({rows, cols});
  }
  return r.size(1) <= 1 || r.stride(1) == 1 ? r : r.contiguous();
}
int64_t ld(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(t.size(1), 1); }
Tensor whole(const OptTensor& t) { return t && t->defined() ? t->contiguous() : Tensor(); }
const void* at_of(const Tensor& t) {
  if (!t.defined()) return nullptr;
  check_memory(t);
  return t.const_data_ptr();
}
void* out_of(const Tensor& t) {
  if (!t.defined()) return nullptr;
  check_memory(t);
  return t.mutable_data_ptr();
}
Tensor space(uint64_t bytes, const Tensor& like) {
  return bytes ? at::empty({(int64_t)bytes}, like.options().dtype(at::kByte)) : Tensor();
}

// A gradient that is asked for its own gradient: the second differentiation raises.
variable_list once(variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  for (Tensor& g : grads) {
    if (!g.defined()) continue;
    variable_list one{g.detach().requires_grad_()};
    auto node = std::make_shared<torch::autograd::DelayedError>("this operator is differentiable once", 1);
    g = (*node)(std::move(one))[0];
  }
  return grads;
}

// ------------------------------------------------------------------ norms

struct Normed {
  Tensor y, s, stats, w;
  Tensor x, r;  // what the gradient reads: as given, or the copies, where their rows are not contiguous
};
Normed norm_run(const Tensor& x, const OptTensor& weight, const OptTensor& bias, const OptTensor& residual, double eps,
                int64_t kind, bool keep) {
  const c10::DeviceGuard guard(x.device());
  const int64_t cols = x.size(-1);
  const Tensor x2 = flat(x, cols), b = whole(bias);
  const Tensor r2 = residual ? flat(*residual, cols) : Tensor();
  Normed o;
  o.w = whole(weight);
  o.y = at::empty(x.sizes(), x.options());
  if (residual) o.s = at::empty(x.sizes(), x.options());
  if (keep) o.stats = at::empty({x2.size(0), 2}, x.options().dtype(at::kFloat));
  const muon_norm_desc_t d{dtype_of(x), (int32_t)kind, x2.size(0), cols, ld(x2), residual ? ld(r2) : 0, 0, 0, eps};
  check(muon_norm_forward(&d, at_of(x2), at_of(r2), at_of(o.w), at_of(b), out_of(o.y), out_of(o.s),
                          static_cast<float*>(out_of(o.stats)), stream_of(x)),
        "muon_norm_forward");
  o.x = x2.is_alias_of(x) ? x : x2;
  if (residual) o.r = r2.is_alias_of(*residual) ? *residual : r2;
  return o;
}
// dx like x, dw, db; undefined where not needed.
variable_list norm_grad(const Tensor& dy, const Tensor& x, const Tensor& residual, const Tensor& w, const Tensor& stats, const Tensor& ds,
                        int64_t kind, bool need_x, bool need_w, bool need_b) {
  const c10::DeviceGuard guard(x.device());
  const int64_t cols = x.size(-1);
  const Tensor rows = flat(x, cols), g = flat(dy, cols), d2 = ds.defined() ? flat(ds, cols) : Tensor();
  const Tensor r2 = residual.defined() ? flat(residual, cols) : Tensor();
  Tensor dx, dw, db;
  if (need_x) dx = at::empty(x.sizes(), rows.options());
  if (need_w) dw = at::empty({cols}, rows.options());
  if (need_b) db = at::empty({cols}, rows.options());
  const muon_norm_desc_t d{dtype_of(rows), (int32_t)kind, rows.size(0), cols, ld(rows), residual.defined() ? ld(r2) : 0, ld(g),
                           ds.defined() ? ld(d2) : 0, 0.0};
  uint64_t bytes = 0;
  if (need_w || need_b) check(muon_norm_workspace(&d, &bytes), "muon_norm_workspace");
  const Tensor ws = space(bytes, rows);
  check(muon_norm_backward(&d, at_of(g), at_of(rows), at_of(r2), at_of(w), static_cast<const float*>(at_of(stats)), at_of(d2),
                           out_of(dx), out_of(dw), out_of(db), out_of(ws), bytes, stream_of(rows)),
        "muon_norm_backward");
  return {dx, dw, db};
}

struct NormNode : public Function<NormNode> {
  static variable_list forward(AutogradContext* ctx, const Tensor& x, const OptTensor& weight, const OptTensor& bias,
                               const OptTensor& residual, double eps, int64_t kind) {
    const Normed o = norm_run(x, weight, bias, residual, eps, kind, true);
    ctx->save_for_backward({o.x, o.r, o.w, o.stats});
    const bool reshaped = o.x.dim() != x.dim();
    if (reshaped) ctx->saved_data["shape"] = x.sizes().vec();
    ctx->saved_data["given"] = int64_t((weight ? 1 : 0) | (bias ? 2 : 0) | (residual ? 4 : 0) | (reshaped ? 8 : 0)) | kind << 8;
    ctx->set_materialize_grads(false);
    if (residual) return {o.y, o.s};
    return {o.y};
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    // The edges are those of the tensors that were given.
    const int64_t given = ctx->saved_data["given"].toInt();
    int edge = 1;
    const bool need_x = ctx->needs_input_grad(0);
    const bool need_w = (given & 1) && ctx->needs_input_grad(edge++);
    const bool need_b = (given & 2) && ctx->needs_input_grad(edge++);
    const bool need_r = (given & 4) && ctx->needs_input_grad(edge);
    const Tensor& dy = grads[0];
    const Tensor ds = grads.size() > 1 ? grads[1] : Tensor();
    Tensor dx, dw, db;
    if (!dy.defined()) {  // only s was used
      dx = ds;
    } else {
      const variable_list saved = ctx->get_saved_variables();
      const variable_list g = norm_grad(dy, saved[0], saved[1], saved[2], saved[3], ds, given >> 8, need_x || need_r, need_w, need_b);
      dx = g[0];
      if (dx.defined() && (given & 8)) dx = dx.view(ctx->saved_data["shape"].toIntVector());
      dw = g[1];
      db = g[2];
    }
    return once({need_x ? dx : Tensor(), dw, db, need_r ? dx : Tensor(), Tensor(), Tensor()});
  }
};

variable_list norm(const Tensor& x, const OptTensor& weight, const OptTensor& bias, const OptTensor& residual, double eps,
                   int64_t kind, bool track) {
  if (track) return NormNode::apply(x, weight, bias, residual, eps, kind);
  const Normed o = norm_run(x, weight, bias, residual, eps, kind, false);
  if (residual) return {o.y, o.s};
  return {o.y};
}
// y, s (undefined without a residual), stats.
std::tuple<Tensor, OptTensor, Tensor> norm_forward(const Tensor& x, const OptTensor& weight, const OptTensor& bias,
                                                   const OptTensor& residual, double eps, int64_t kind) {
  const at::NoGradGuard no_grad;
  const Normed o = norm_run(x, weight, bias, residual, eps, kind, true);
  return {o.y, residual ? OptTensor(o.s) : OptTensor(), o.stats};
}
std::vector<OptTensor> norm_backward(const Tensor& dy, const Tensor& x, const OptTensor& residual, const OptTensor& weight,
                                     const Tensor& stats, const OptTensor& ds, int64_t kind, bool need_x, bool need_w, bool need_b) {
  const at::NoGradGuard no_grad;
  const variable_list g = norm_grad(dy, x, residual ? *residual : Tensor(), whole(weight), stats, ds ? *ds : Tensor(), kind,
                                    need_x, need_w, need_b);
  std::vector<OptTensor> out;
  for (const Tensor& t : g) out.push_back(t.defined() ? OptTensor(t) : OptTensor());
  return out;
}

// ------------------------------------------------------------------ gate

struct Gated {
  Tensor weights, ids, z, mask;
};
muon_gate_desc_t gate_desc(const Tensor& z, int64_t top, int64_t normalize) {
  return muon_gate_desc_t{dtype_of(z), (int32_t)z.size(1), (int32_t)top, (int32_t)normalize, z.size(0), ld(z)};
}
Gated gate_run(const Tensor& logits, int64_t top, int64_t normalize, const OptTensor& mask) {
  const c10::DeviceGuard guard(logits.device());
  Gated o;
  o.z = flat(logits, logits.size(1));
  o.mask = whole(mask);
  o.weights = at::empty({o.z.size(0), top}, logits.options().dtype(at::kFloat));
  o.ids = at::empty({o.z.size(0), top}, logits.options().dtype(at::kInt));
  const muon_gate_desc_t d = gate_desc(o.z, top, normalize);
  check(muon_gate_forward(&d, at_of(o.z), static_cast<const uint8_t*>(at_of(o.mask)), static_cast<float*>(out_of(o.weights)),
                          static_cast<int32_t*>(out_of(o.ids)), stream_of(o.z)),
        "muon_gate_forward");
  return o;
}
// z: the logits, or (normalised weights need no more of them) nothing.
Tensor gate_grad(const Tensor& dweights, const Tensor& z, at::ScalarType dtype, int64_t experts, const Tensor& weights,
                 const Tensor& ids, int64_t normalize, const Tensor& mask) {
  const c10::DeviceGuard guard(weights.device());
  const Tensor dw = dweights.contiguous(), dz = at::empty({ids.size(0), experts}, weights.options().dtype(dtype));
  muon_gate_desc_t d = gate_desc(dz, ids.size(1), normalize);
  if (z.defined()) d.ldz = ld(z);
  check(muon_gate_backward(&d, at_of(z), static_cast<const uint8_t*>(at_of(mask)), static_cast<const float*>(at_of(weights)),
                           static_cast<const int32_t*>(at_of(ids)), static_cast<const float*>(at_of(dw)), out_of(dz),
                           stream_of(weights)),
        "muon_gate_backward");
  return dz;
}

struct GateNode : public Function<GateNode> {
  static variable_list forward(AutogradContext* ctx, const Tensor& logits, int64_t top, int64_t normalize,
                               const OptTensor& mask) {
    const Gated o = gate_run(logits, top, normalize, mask);
    ctx->save_for_backward({normalize ? Tensor() : o.z, o.weights, o.ids, o.mask});
    ctx->saved_data["kind"] = normalize | (int64_t)logits.scalar_type() << 1 | logits.size(1) << 16;
    ctx->mark_non_differentiable({o.ids});
    ctx->set_materialize_grads(false);
    return {o.weights, o.ids};
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    variable_list out(4);
    if (grads[0].defined()) {
      const variable_list s = ctx->get_saved_variables();
      const int64_t kind = ctx->saved_data["kind"].toInt();
      out[0] = gate_grad(grads[0], s[0], static_cast<at::ScalarType>(kind >> 1 & 0x7fff), kind >> 16, s[1], s[2], kind & 1, s[3]);
    }
    return once(std::move(out));
  }
};

std::tuple<Tensor, Tensor> gate(const Tensor& logits, int64_t top, int64_t normalize, const OptTensor& mask, bool track) {
  if (track) {
    const variable_list o = GateNode::apply(logits, top, normalize, mask);
    return {o[0], o[1]};
  }
  const at::NoGradGuard no_grad;
  const Gated o = gate_run(logits, top, normalize, mask);
  return {o.weights, o.ids};
}
Tensor gate_backward(const Tensor& dweights, const Tensor& logits, const Tensor& weights, const Tensor& ids,
                     int64_t normalize, const OptTensor& mask) {
  const at::NoGradGuard no_grad;
  return gate_grad(dweights, normalize ? Tensor() : flat(logits, logits.size(1)), logits.scalar_type(), logits.size(1), weights,
                   ids, normalize, whole(mask));
}

// ------------------------------------------------------------------ balance loss

struct Balanced {
  Tensor loss, counts, shares, z, mask;
};
Balanced balance_run(const Tensor& logits, const Tensor& expert_ids, const OptTensor& mask) {
  const c10::DeviceGuard guard(logits.device());
  Balanced o;
  o.z = flat(logits, logits.size(1));
  o.mask = whole(mask);
  const Tensor ids = expert_ids.contiguous();
  const int64_t e = o.z.size(1);
  o.loss = at::empty({}, logits.options().dtype(at::kFloat));
  o.counts = at::empty({e}, logits.options().dtype(at::kInt));
  o.shares = at::empty({e + 1}, logits.options().dtype(at::kFloat));
  const muon_gate_desc_t d = gate_desc(o.z, ids.size(1), 0);
  uint64_t bytes = 0;
  check(muon_balance_workspace(&d, &bytes), "muon_balance_workspace");
  const Tensor ws = space(bytes, logits);
  check(muon_balance_forward(&d, at_of(o.z), at_of(ids), (int32_t)ids.element_size(),
                             static_cast<const uint8_t*>(at_of(o.mask)), static_cast<float*>(out_of(o.loss)),
                             static_cast<int32_t*>(out_of(o.counts)), static_cast<float*>(out_of(o.shares)), out_of(ws),
                             bytes, stream_of(o.z)),
        "muon_balance_forward");
  return o;
}
Tensor balance_grad(const Tensor& dloss, const Tensor& z, int64_t top, const Tensor& shares, const Tensor& mask) {
  const c10::DeviceGuard guard(z.device());
  const Tensor dz = at::empty(z.sizes(), z.options());
  const muon_gate_desc_t d = gate_desc(z, top, 0);
  check(muon_balance_backward(&d, at_of(z), static_cast<const uint8_t*>(at_of(mask)), static_cast<const float*>(at_of(shares)),
                              static_cast<const float*>(at_of(dloss)), out_of(dz), stream_of(z)),
        "muon_balance_backward");
  return dz;
}

struct BalanceNode : public Function<BalanceNode> {
  static variable_list forward(AutogradContext* ctx, const Tensor& logits, const Tensor& ids, const OptTensor& mask) {
    const Balanced o = balance_run(logits, ids, mask);
    ctx->save_for_backward({o.z, o.shares, o.mask});
    ctx->saved_data["top"] = ids.size(1);
    ctx->mark_non_differentiable({o.counts});
    ctx->set_materialize_grads(false);
    return {o.loss, o.counts};
  }
  static variable_list backward(AutogradContext* ctx, const variable_list& grads) {
    variable_list out(3);
    if (grads[0].defined()) {
      const variable_list s = ctx->get_saved_variables();
      out[0] = balance_grad(grads[0], s[0], ctx->saved_data["top"].toInt(), s[1], s[2]);
    }
    return once(std::move(out));
  }
};

std::tuple<Tensor, Tensor> balance(const Tensor& logits, const Tensor& ids, const OptTensor& mask, bool track) {
  if (track) {
    const variable_list o = BalanceNode::apply(logits, ids, mask);
    return {o[0], o[1]};
  }
  const at::NoGradGuard no_grad;
  const Balanced o = balance_run(logits, ids, mask);
  return {o.loss, o.counts};
}
std::tuple<Tensor, Tensor, Tensor> balance_forward(const Tensor& logits, const Tensor& ids, const OptTensor& mask) {
  const at::NoGradGuard no_grad;
  const Balanced o = balance_run(logits, ids, mask);
  return {o.loss, o.counts, o.shares};
}
Tensor balance_backward(const Tensor& dloss, const Tensor& logits, int64_t top, const Tensor& shares, const OptTensor& mask) {
  const at::NoGradGuard no_grad;
  return balance_grad(dloss, flat(logits, logits.size(1)), top, shares, whole(mask));
}

// ------------------------------------------------------------------ four bits

std::tuple<Tensor, Tensor> mx_quantize(const Tensor& weight) {
  const at::NoGradGuard no_grad;
  const c10::DeviceGuard guard(weight.device());
  const int64_t k = weight.size(-2), n = weight.size(-1), groups = weight.dim() == 3 ? weight.size(0) : 0;
  auto layout = [&](const Tensor& w) {
    // Strides that reach nothing: torch calls such a view contiguous, and a copy would keep them.
    if (w.numel() == 0 || (k == 1 && n == 1)) return 0;
    if (w.stride(-1) == 1 && (k <= 1 || w.stride(-2) >= n)) return 0;
    return w.stride(-2) == 1 && (n <= 1 || w.stride(-1) >= k) ? 1 : -1;
  };
  const Tensor w = layout(weight) < 0 ? weight.contiguous() : weight;
  const int32_t order = layout(w);
  const int64_t ldw = order == 0 ? (k > 1 ? w.stride(-2) : std::max<int64_t>(n, 1)) : (n > 1 ? w.stride(-1) : std::max<int64_t>(k, 1));
  std::vector<int64_t> vs, ss;
  if (groups) vs.push_back(groups), ss.push_back(groups);
  for (int64_t v : {(k + 127) / 128, n, (int64_t)64}) vs.push_back(v);
  for (int64_t v : {(k + 511) / 512, n, (int64_t)16}) ss.push_back(v);
  const Tensor values = at::empty(vs, w.options().dtype(at::kByte)), scales = at::empty(ss, w.options().dtype(at::kByte));
  const muon_mx_desc_t d{dtype_of(w), 0, (int32_t)groups, order, 0, k, n, 0, ldw, groups ? w.stride(0) : 0, 0};
  check(muon_mx_quantize(&d, at_of(w), static_cast<uint8_t*>(out_of(values)), static_cast<uint8_t*>(out_of(scales)), stream_of(w)),
        "muon_mx_quantize");
  return {values, scales};
}
Tensor mx_dequantize(const Tensor& values, const Tensor& scales, int64_t k, bool bf16) {
  const at::NoGradGuard no_grad;
  const c10::DeviceGuard guard(values.device());
  const int64_t n = values.size(-2), groups = values.dim() == 4 ? values.size(0) : 0;
  const auto options = values.options().dtype(bf16 ? at::kBFloat16 : at::kFloat);
  const Tensor out = groups ? at::empty({groups, n, k}, options) : at::empty({n, k}, options);
  const muon_mx_desc_t d{dtype_of(out), 0, (int32_t)groups, 0, 0, k, n, 0, n, 0, 0};
  check(muon_mx_dequantize(&d, static_cast<const uint8_t*>(at_of(values)), static_cast<const uint8_t*>(at_of(scales)), out_of(out),
                           stream_of(values)),
        "muon_mx_dequantize");
  return out.transpose(-1, -2);
}
Tensor mx_linear(const Tensor& x, const Tensor& values, const Tensor& scales, int64_t k, const OptTensor& bias,
                 const OptTensor& residual, const OptTensor& offsets, int64_t act) {
  const at::NoGradGuard no_grad;
  const c10::DeviceGuard guard(x.device());
  const int64_t n = values.size(-2);
  const Tensor x2 = flat(x, k), b = whole(bias), r2 = residual ? flat(*residual, n) : Tensor();
  std::vector<int64_t> shape = x.sizes().vec();
  shape.back() = n;
  const Tensor y = at::empty(shape, x.options());
  const muon_mx_desc_t d{dtype_of(x), (int32_t)act, offsets ? (int32_t)values.size(0) : 0, 0, x2.size(0), k, n, ld(x2), 0, 0,
                         residual ? ld(r2) : 0};
  uint64_t bytes = 0;
  check(muon_mx_linear_workspace(&d, &bytes), "muon_mx_linear_workspace");
  const Tensor ws = space(bytes, x);
  check(muon_mx_linear(&d, offsets ? static_cast<const int32_t*>(at_of(*offsets)) : nullptr, at_of(x2),
                       static_cast<const uint8_t*>(at_of(values)), static_cast<const uint8_t*>(at_of(scales)), at_of(b), at_of(r2),
                       out_of(y), out_of(ws), bytes, stream_of(x)),
        "muon_mx_linear");
  return y;
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  m.def("norm", &norm);
  m.def("norm_forward", &norm_forward);
  m.def("norm_backward", &norm_backward);
  m.def("gate", &gate);
  m.def("gate_backward", &gate_backward);
  m.def("balance", &balance);
  m.def("balance_forward", &balance_forward);
  m.def("balance_backward", &balance_backward);
  m.def("mx_quantize", &mx_quantize);
  m.def("mx_dequantize", &mx_dequantize);
  m.def("mx_linear", &mx_linear);
}
