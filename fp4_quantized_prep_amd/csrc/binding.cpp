// Python binding of the attention layer's entry points (include/iqprep.h): the
// checks of tensors and the marshalling of their addresses, in C++ because a
// decode step's kernels take less time than the same checks do in Python
// (measured on MI355X: a 16-token qk_norm_rope call issues every 17.8 us from
// Python with ctypes). Nothing is computed here.
//
// Outputs that are not passed in come from the pool of the current stream of
// the tensors' device, which is also the stream of the launch.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <string>
#include <tuple>
#include <utility>

#include "iqprep.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

py::object* g_raise = nullptr;   // (status, where): raises the package's error

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

std::string str(int64_t v) { return std::to_string(v); }

[[noreturn]] void value_error(const std::string& what) { throw py::value_error(what); }

c10::Device gpu_of(const Tensor& t, const char* name) {
  if (!t.defined()) throw py::type_error(std::string(name) + " must be a torch.Tensor");
  if (!t.is_cuda()) value_error(std::string(name) + " must be on a GPU, got " + t.device().str());
  return t.device();
}

void require(const Tensor& t, const char* name, at::ScalarType dtype, c10::Device dev, int64_t ndim) {
  if (!t.defined()) throw py::type_error(std::string(name) + " must be a torch.Tensor");
  if (t.scalar_type() != dtype)
    throw py::type_error(std::string(name) + " must have dtype " + toString(dtype) + ", got " + toString(t.scalar_type()));
  if (t.device() != dev) value_error(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
  if (t.dim() != ndim) value_error(std::string(name) + " must be " + str(ndim) + "-D, got shape " + shape_of(t));
}

// E4M3 codes: uint8 or float8_e4m3fn
void require_codes(const Tensor& t, const char* name, c10::Device dev, int64_t ndim) {
  require(t, name, t.defined() && t.scalar_type() == at::kFloat8_e4m3fn ? at::kFloat8_e4m3fn : at::kByte, dev, ndim);
}

// One C call with dev current and dev's current stream as its last argument.
template <class F, class... A>
void run(F fn, const char* where, c10::Device dev, A... args) {
  const c10::OptionalDeviceGuard guard(dev);
  const int st = fn(args..., c10::hip::getCurrentHIPStream(dev.index()).stream());
  if (st != IQP_OK) {
    (*g_raise)(st, where);
    throw std::runtime_error(where);
  }
}

Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
}

Tensor fp8_gemm(const Tensor& a, const Tensor& a_scales, const Tensor& w, const Tensor& w_scales, const OptTensor& out_,
                const OptTensor& workspace_) {
  const c10::Device dev = gpu_of(a, "a");
  require_codes(a, "a", dev, 2);
  require(a_scales, "a_scales", at::kInt, dev, 2);
  require_codes(w, "w", dev, 2);
  require(w_scales, "w_scales", at::kByte, dev, 2);
  const int64_t M = a.size(0), K = a.size(1), N = w.size(0), kb = K / 128, nw = (kb + 3) / 4;
  if (w.size(1) != K) value_error("w must be [N, " + str(K) + "], got " + shape_of(w));
  if (a_scales.size(0) != M || a_scales.size(1) != nw)
    value_error("a_scales must be [" + str(M) + ", " + str(nw) + "] (one packed word per 512 columns), got " + shape_of(a_scales));
  if (w_scales.size(0) != (N + 127) / 128 || w_scales.size(1) != kb)
    value_error("w_scales must be [" + str((N + 127) / 128) + ", " + str(kb) + "], got " + shape_of(w_scales));
  Tensor out = out_ ? *out_ : empty({M, N}, at::kBFloat16, dev);
  require(out, "out", at::kBFloat16, dev, 2);
  if (out.size(0) != M || out.size(1) != N) value_error("out must be [" + str(M) + ", " + str(N) + "], got " + shape_of(out));
  if (M && N && (a.stride(1) != 1 || w.stride(1) != 1 || (N > 1 && out.stride(1) != 1) || (kb > 1 && w_scales.stride(1) != 1)))
    value_error("a, w, w_scales and out need contiguous rows");
  // the stride of a single row means nothing: torch gives any
  const auto pitch = [](const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); };
  int64_t sm = a_scales.stride(0), sw = a_scales.stride(1);
  if (M == 1) sm = sw == 1 ? nw : 1;
  if (nw == 1) {
    if (sm == 1) sw = M;
    else sw = 1;
  }
  Tensor ws;
  if (workspace_) {
    ws = *workspace_;
    require(ws, "workspace", at::kByte, dev, 1);
    if (!ws.is_contiguous()) value_error("workspace must be contiguous");
  } else if (const int64_t need = fp8_gemm_workspace_bytes(M, N, K)) {
    ws = empty({need}, at::kByte, dev);
  }
  run(fp8_gemm_1x128_128x128, "fp8_gemm_1x128_128x128", dev, a.const_data_ptr(), pitch(a), (const int32_t*)a_scales.const_data_ptr(),
      sm, sw, w.const_data_ptr(), pitch(w), (const uint8_t*)w_scales.const_data_ptr(), pitch(w_scales), M, N, K,
      out.mutable_data_ptr(), M > 1 ? out.stride(0) : (N + 7) / 8 * 8, ws.defined() ? ws.mutable_data_ptr() : nullptr,
      ws.defined() ? (int64_t)ws.numel() : (int64_t)0);
  return out;
}

// Rows of heads, [M, H, D] or [M, H * D], contiguous within a row
struct Rows {
  int64_t heads, ld;
};

Rows rows_of(const Tensor& t, const char* name, c10::Device dev, int64_t D, int64_t heads = -1, int64_t rows = -1) {
  if (!t.defined()) throw py::type_error(std::string(name) + " must be a torch.Tensor");
  if (t.scalar_type() != at::kBFloat16)
    throw py::type_error(std::string(name) + " must have dtype BFloat16, got " + toString(t.scalar_type()));
  if (t.device() != dev) value_error(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
  int64_t h = -1;
  bool packed = false;
  if (t.dim() == 3 && t.size(2) == D) {
    h = t.size(1);
    packed = t.stride(2) == 1 && (h == 1 || t.stride(1) == D);
  } else if (t.dim() == 2 && D > 0 && t.size(1) % D == 0) {
    h = t.size(1) / D;
    packed = t.stride(1) == 1;
  }
  if (h < 0 || (!packed && t.numel() > 0) || (heads >= 0 && h != heads))
    value_error(std::string(name) + " must be [rows, heads, " + str(D) + "] or [rows, heads * " + str(D) + "] with contiguous rows" +
                (heads >= 0 ? " of " + str(heads) + " heads" : std::string()) + ", got shape " + shape_of(t));
  if (rows >= 0 && t.size(0) != rows) value_error(std::string(name) + " needs " + str(rows) + " rows, got " + str(t.size(0)));
  return {h, t.size(0) > 1 ? t.stride(0) : h * D};
}

std::tuple<Tensor, Tensor> norm_rope(const Tensor& q, const Tensor& k, const Tensor& q_weight, const Tensor& k_weight,
                                     const Tensor& positions, const Tensor& cos_sin, double eps, int64_t D,
                                     const std::string& layout, const OptTensor& q_out_, const OptTensor& k_out_) {
  const c10::Device dev = gpu_of(q, "q");
  if (layout != "half_split" && layout != "interleaved") value_error("rope_layout must be 'half_split' or 'interleaved'");
  const Rows rq = rows_of(q, "q", dev, D);
  const int64_t M = q.size(0);
  const Rows rk = rows_of(k, "k", dev, D, -1, M);
  require(positions, "positions", at::kLong, dev, 1);
  require(cos_sin, "cos_sin", at::kFloat, dev, 2);
  require(q_weight, "q_weight", at::kBFloat16, dev, 1);
  require(k_weight, "k_weight", at::kBFloat16, dev, 1);
  if (positions.size(0) != M) value_error("q, k and positions need one row per token");
  if (q_weight.size(0) != D || k_weight.size(0) != D) value_error("q_weight and k_weight need " + str(D) + " values");
  if (!positions.is_contiguous() || !cos_sin.is_contiguous() || !q_weight.is_contiguous() || !k_weight.is_contiguous())
    value_error("positions, cos_sin and the weights must be contiguous");
  Tensor q_out = q_out_ ? *q_out_ : empty(q.sizes(), at::kBFloat16, dev);
  Tensor k_out = k_out_ ? *k_out_ : empty(k.sizes(), at::kBFloat16, dev);
  const Rows ro = rows_of(q_out, "q_out", dev, D, rq.heads, M), rp = rows_of(k_out, "k_out", dev, D, rk.heads, M);
  run(qk_norm_rope, "qk_norm_rope", dev, q.const_data_ptr(), rq.ld, k.const_data_ptr(), rk.ld, M, (int32_t)rq.heads,
      (int32_t)rk.heads, (int32_t)D, (int32_t)cos_sin.size(1), q_weight.const_data_ptr(), k_weight.const_data_ptr(), (float)eps,
      (const int64_t*)positions.const_data_ptr(), (const float*)cos_sin.const_data_ptr(), cos_sin.size(0), q_out.mutable_data_ptr(),
      ro.ld, k_out.mutable_data_ptr(), rp.ld, layout == "interleaved" ? IQP_ROPE_INTERLEAVED : 0);
  return {q_out, k_out};
}

struct Cache {
  int64_t blocks, heads, block, D;
};

Cache cache_of(const Tensor& k, const Tensor& v, const Tensor& ks, const Tensor& vs, c10::Device dev) {
  require(k, "cache.k", at::kByte, dev, 4);
  require(v, "cache.v", at::kByte, dev, 4);
  require(ks, "cache.k_scales", at::kByte, dev, 2);
  require(vs, "cache.v_scales", at::kByte, dev, 2);
  const Cache c = {k.size(0), k.size(1), k.size(2), k.size(3)};
  if (v.size(0) != c.blocks || v.size(1) != c.heads || v.size(2) != c.D || v.size(3) != c.block)
    value_error("cache.v must be [" + str(c.blocks) + ", " + str(c.heads) + ", " + str(c.D) + ", " + str(c.block) + "], got " + shape_of(v));
  if (ks.size(0) != c.blocks || ks.size(1) != c.heads || vs.size(0) != c.blocks || vs.size(1) != c.heads)
    value_error("the cache's scales must be [" + str(c.blocks) + ", " + str(c.heads) + "]");
  if (!k.is_contiguous() || !v.is_contiguous() || !ks.is_contiguous() || !vs.is_contiguous())
    value_error("the cache's tensors must be contiguous");
  return c;
}

struct Batch {
  const int32_t* table;
  int64_t ld;
  int32_t width;
  const int32_t *lens, *cu;
  int32_t S;
};

Batch batch_of(const Tensor& table, const Tensor& lens, const Tensor& cu, c10::Device dev) {
  require(table, "block_table", at::kInt, dev, 2);
  require(lens, "seq_lens", at::kInt, dev, 1);
  require(cu, "cu_rows", at::kInt, dev, 1);
  const int64_t S = table.size(0), width = table.size(1);
  if (lens.size(0) != S || cu.size(0) != S + 1) value_error("seq_lens must hold " + str(S) + " entries and cu_rows " + str(S + 1));
  if (!lens.is_contiguous() || !cu.is_contiguous() || (S && width > 1 && table.stride(1) != 1))
    value_error("seq_lens and cu_rows must be contiguous, block_table's rows too");
  if (S > 0x7FFFFFFF || width > 0x7FFFFFFF) value_error("block_table is too large");
  return {(const int32_t*)table.const_data_ptr(), S > 1 ? table.stride(0) : width, (int32_t)width,
          (const int32_t*)lens.const_data_ptr(), (const int32_t*)cu.const_data_ptr(), (int32_t)S};
}

uint8_t* bytes(const Tensor& t) { return (uint8_t*)t.mutable_data_ptr(); }

void kv_append(const Tensor& k, const Tensor& v, const Tensor& kc, const Tensor& vc, const Tensor& ks, const Tensor& vs,
               const Tensor& table, const Tensor& lens, const Tensor& cu) {
  const c10::Device dev = gpu_of(k, "k");
  const Cache c = cache_of(kc, vc, ks, vs, dev);
  const Rows rk = rows_of(k, "k", dev, c.D, c.heads);
  const int64_t T = k.size(0);
  const Rows rv = rows_of(v, "v", dev, c.D, c.heads, T);
  const Batch b = batch_of(table, lens, cu, dev);
  run(kv_cache_append_fp8, "kv_cache_append_fp8", dev, k.const_data_ptr(), rk.ld, v.const_data_ptr(), rv.ld, T, (int32_t)c.heads,
      (int32_t)c.D, (void*)bytes(kc), (void*)bytes(vc), bytes(ks), bytes(vs), c.blocks, (int32_t)c.block, b.table, b.ld, b.width,
      b.lens, b.cu, b.S);
}

std::tuple<Tensor, Tensor> kv_read(const Tensor& kc, const Tensor& vc, const Tensor& ks, const Tensor& vs, const Tensor& table,
                                   const Tensor& lens, const Tensor& cu, int64_t rows, const OptTensor& k_out_,
                                   const OptTensor& v_out_) {
  const c10::Device dev = gpu_of(kc, "cache.k");
  const Cache c = cache_of(kc, vc, ks, vs, dev);
  if (rows < 0) value_error("rows must not be negative");
  Tensor k = k_out_ ? *k_out_ : empty({rows, c.heads, c.D}, at::kBFloat16, dev);
  Tensor v = v_out_ ? *v_out_ : empty({rows, c.heads, c.D}, at::kBFloat16, dev);
  const Rows rk = rows_of(k, "k_out", dev, c.D, c.heads, rows), rv = rows_of(v, "v_out", dev, c.D, c.heads, rows);
  const Batch b = batch_of(table, lens, cu, dev);
  run(kv_cache_read_fp8, "kv_cache_read_fp8", dev, kc.const_data_ptr(), vc.const_data_ptr(), (const uint8_t*)bytes(ks),
      (const uint8_t*)bytes(vs), c.blocks, (int32_t)c.block, (int32_t)c.heads, (int32_t)c.D, b.table, b.ld, b.width, b.lens, b.cu, b.S,
      k.mutable_data_ptr(), rk.ld, v.mutable_data_ptr(), rv.ld, rows);
  return {k, v};
}

Tensor attention(const Tensor& q, const Tensor& kc, const Tensor& vc, const Tensor& ks, const Tensor& vs, const Tensor& table,
                 const Tensor& lens, const Tensor& cu, std::optional<double> scale, int64_t window, const OptTensor& out_,
                 const OptTensor& workspace_) {
  const c10::Device dev = gpu_of(q, "q");
  const Cache c = cache_of(kc, vc, ks, vs, dev);
  const Rows rq = rows_of(q, "q", dev, c.D);
  if (c.heads == 0 || rq.heads % c.heads)
    value_error("q needs a multiple of the cache's " + str(c.heads) + " heads, got " + str(rq.heads));
  if (window < 0 || window > 0x7FFFFFFF) value_error("window must be 0 (none) or a number of tokens");
  const int64_t T = q.size(0);
  Tensor out = out_ ? *out_ : empty(q.sizes(), at::kBFloat16, dev);
  const Rows ro = rows_of(out, "out", dev, c.D, rq.heads, T);
  Tensor ws = workspace_ ? *workspace_ : empty({attention_fp8_kv_workspace_bytes((int32_t)c.D)}, at::kByte, dev);
  require(ws, "workspace", at::kByte, dev, 1);
  if (!ws.is_contiguous()) value_error("workspace must be contiguous");
  const Batch b = batch_of(table, lens, cu, dev);
  run(attention_fp8_kv, "attention_fp8_kv", dev, q.const_data_ptr(), rq.ld, T, (int32_t)rq.heads, (int32_t)c.heads, (int32_t)c.D,
      kc.const_data_ptr(), vc.const_data_ptr(), (const uint8_t*)bytes(ks), (const uint8_t*)bytes(vs), c.blocks, (int32_t)c.block,
      b.table, b.ld, b.width, b.lens, b.cu, b.S, (float)(scale ? *scale : 1.0 / std::sqrt((double)c.D)), (int32_t)window,
      out.mutable_data_ptr(), ro.ld, ws.mutable_data_ptr(), (int64_t)ws.numel());
  return out;
}

// A tensor that has to be contiguous, of these sizes
const Tensor& exact(const Tensor& t, const char* name, at::ScalarType dtype, c10::Device dev, at::IntArrayRef sizes) {
  require(t, name, dtype, dev, (int64_t)sizes.size());
  if (t.sizes() != sizes) {
    std::string want = "(";
    for (size_t i = 0; i < sizes.size(); ++i) want += (i ? ", " : "") + str(sizes[i]);
    value_error(std::string(name) + " must be of shape " + want + "), got " + shape_of(t));
  }
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t;
}

// The operators of experts and adapters have no backward pass: a gradient asked of
// their operands would be lost without a word.
void require_no_grad(const Tensor& t, const char* name) {
  if (c10::GradMode::is_enabled() && t.requires_grad())
    value_error(std::string(name) + " requires a gradient, and this call has no backward pass: detach it, or call under torch.no_grad()");
}

// Tells autograd that a tensor of the caller's was written to (those of inference
// mode have no version to count).
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

std::tuple<Tensor, Tensor> route(const Tensor& logits, int64_t top_k, const OptTensor& bias, int64_t scoring, bool renormalize,
                                 double scale, const OptTensor& weights_, const OptTensor& experts_) {
  const c10::Device dev = gpu_of(logits, "logits");
  const bool half = logits.scalar_type() == at::kBFloat16;
  require(logits, "logits", half ? at::kBFloat16 : at::kFloat, dev, 2);
  const int64_t M = logits.size(0), E = logits.size(1);
  if (top_k < 1 || top_k > E) value_error("top_k must be 1 to " + str(E) + ", got " + str(top_k));
  if (E > 0x7FFFFFFF) value_error("logits has too many columns");
  if (M && E > 1 && logits.stride(1) != 1) value_error("logits needs contiguous rows");
  if (bias) exact(*bias, "bias", at::kFloat, dev, {E});
  require_no_grad(logits, "logits");
  if (bias) require_no_grad(*bias, "bias");
  Tensor weights = weights_ ? *weights_ : empty({M, top_k}, at::kFloat, dev);
  Tensor experts = experts_ ? *experts_ : empty({M, top_k}, at::kInt, dev);
  exact(weights, "weights", at::kFloat, dev, {M, top_k});
  exact(experts, "experts", at::kInt, dev, {M, top_k});
  require_no_grad(weights, "weights");
  run(moe_route, "moe_route", dev, logits.const_data_ptr(), M > 1 ? logits.stride(0) : E, (int32_t)half,
      bias ? (const float*)bias->const_data_ptr() : nullptr, M, (int32_t)E, (int32_t)top_k, (int32_t)scoring, (int32_t)renormalize,
      (float)scale, (float*)weights.mutable_data_ptr(), (int32_t*)experts.mutable_data_ptr());
  written(weights);
  written(experts);
  return {weights, experts};
}

std::tuple<Tensor, Tensor, Tensor> group(const Tensor& index, int64_t G, const OptTensor& offsets_, const OptTensor& rows_,
                                         const OptTensor& slots_, const OptTensor& workspace_) {
  const c10::Device dev = gpu_of(index, "index");
  if (index.dim() != 1 && index.dim() != 2) value_error("index must be [M] or [M, k], got shape " + shape_of(index));
  exact(index, "index", at::kInt, dev, index.sizes());
  if (G < 1 || G > 1024) value_error("n_groups must be 1 to 1024, got " + str(G));
  const int64_t R = index.numel();
  Tensor offsets = offsets_ ? *offsets_ : empty({G + 1}, at::kInt, dev);
  Tensor rows = rows_ ? *rows_ : empty({R}, at::kInt, dev);
  Tensor slots = slots_ ? *slots_ : empty(index.sizes(), at::kInt, dev);
  exact(offsets, "offsets", at::kInt, dev, {G + 1});
  exact(rows, "rows", at::kInt, dev, {R});
  exact(slots, "slots", at::kInt, dev, index.sizes());
  const int64_t need = group_rows_workspace_bytes(R, (int32_t)G);
  Tensor ws;
  if (workspace_) {
    ws = *workspace_;
    require(ws, "workspace", at::kByte, dev, 1);
    if (!ws.is_contiguous()) value_error("workspace must be contiguous");
  } else if (need) {
    ws = empty({need}, at::kByte, dev);
  }
  run(group_rows, "group_rows", dev, (const int32_t*)index.const_data_ptr(), R, (int32_t)G, (int32_t*)offsets.mutable_data_ptr(),
      (int32_t*)rows.mutable_data_ptr(), (int32_t*)slots.mutable_data_ptr(), ws.defined() ? ws.mutable_data_ptr() : nullptr,
      ws.defined() ? (int64_t)ws.numel() : (int64_t)0);
  written(offsets);
  written(rows);
  written(slots);
  return {offsets, rows, slots};
}

// What group_rows gave, as its readers need it
struct Groups {
  const int32_t *offsets, *rows;
  int64_t R, top;      // places; entries of a token
  int32_t G;
};

Groups groups_of(const Tensor& offsets, const Tensor& rows, const Tensor& slots, c10::Device dev) {
  require(offsets, "groups.offsets", at::kInt, dev, 1);
  require(rows, "groups.rows", at::kInt, dev, 1);
  if (!slots.defined()) throw py::type_error("groups.slots must be a torch.Tensor");
  if (slots.dim() != 1 && slots.dim() != 2) value_error("groups.slots must be [M] or [M, k], got shape " + shape_of(slots));
  require(slots, "groups.slots", at::kInt, dev, slots.dim());
  if (!offsets.is_contiguous() || !rows.is_contiguous() || !slots.is_contiguous()) value_error("the groups' tensors must be contiguous");
  const int64_t G = offsets.size(0) - 1, R = rows.size(0);
  if (G < 1 || G > 1024) value_error("groups.offsets must hold 2 to 1025 entries, got " + str(G + 1));
  if (slots.numel() != R) value_error("groups.rows and groups.slots must hold as many entries, got " + str(R) + " and " + str(slots.numel()));
  return {(const int32_t*)offsets.const_data_ptr(), (const int32_t*)rows.const_data_ptr(), R, slots.dim() == 2 ? slots.size(1) : 1, (int32_t)G};
}

// Scale words [rows, words]: their strides as the C calls take them
std::pair<int64_t, int64_t> word_strides(const Tensor& t) {
  const int64_t M = t.size(0), nw = t.size(1);
  int64_t sm = t.stride(0), sw = t.stride(1);
  if (M == 1) sm = sw == 1 ? nw : 1;
  if (nw == 1) {
    if (sm == 1) sw = M;
    else sw = 1;
  }
  return {sm, sw};
}

// The operands that both grouped products take
struct Grouped {
  c10::Device dev;
  Groups g;
  int64_t M, K, N, lda, sm, sw, ldwg, ldw, ld_wsg, ld_ws;
  int32_t top;
};

Grouped grouped_of(const Tensor& a, const Tensor& a_scales, const Tensor& w, const Tensor& w_scales, const Tensor& offsets,
                   const Tensor& rows, const Tensor& slots, bool gather) {
  const c10::Device dev = gpu_of(a, "a");
  require_codes(a, "a", dev, 2);
  require(a_scales, "a_scales", at::kInt, dev, 2);
  require_codes(w, "w", dev, 3);
  require(w_scales, "w_scales", at::kByte, dev, 3);
  const Groups g = groups_of(offsets, rows, slots, dev);
  const int64_t M = a.size(0), K = a.size(1), N = w.size(1), kb = K / 128, nw = (kb + 3) / 4;
  const int64_t want = gather ? (g.top ? g.R / g.top : 0) : g.R;
  if (M != want)
    value_error(std::string("a must have ") + str(want) + (gather ? " rows, one a token" : " rows, one a place") + ", got " + str(M));
  if (w.size(0) != g.G || w.size(2) != K) value_error("w must be [" + str(g.G) + ", N, " + str(K) + "], got " + shape_of(w));
  if (a_scales.size(0) != M || a_scales.size(1) != nw)
    value_error("a_scales must be [" + str(M) + ", " + str(nw) + "] (one packed word per 512 columns), got " + shape_of(a_scales));
  if (w_scales.size(0) != g.G || w_scales.size(1) != (N + 127) / 128 || w_scales.size(2) != kb)
    value_error("w_scales must be [" + str(g.G) + ", " + str((N + 127) / 128) + ", " + str(kb) + "], got " + shape_of(w_scales));
  if (M && N && (a.stride(1) != 1 || w.stride(2) != 1 || (kb > 1 && w_scales.stride(2) != 1)))
    value_error("a, w and w_scales need contiguous rows");
  const auto [sm, sw] = word_strides(a_scales);
  // the stride of a single row or group means nothing: torch gives any
  const int64_t ldw = N > 1 ? w.stride(1) : K, ld_ws = w_scales.size(1) > 1 ? w_scales.stride(1) : kb;
  return {dev, g, M, K, N, M > 1 ? a.stride(0) : K, sm, sw, g.G > 1 ? w.stride(0) : N * ldw, ldw,
          g.G > 1 ? w_scales.stride(0) : w_scales.size(1) * ld_ws, ld_ws, gather ? (int32_t)g.top : 0};
}

Tensor grouped_gemm(const Tensor& a, const Tensor& a_scales, const Tensor& w, const Tensor& w_scales, const Tensor& offsets,
                    const Tensor& rows, const Tensor& slots, bool gather, const OptTensor& out_) {
  const Grouped p = grouped_of(a, a_scales, w, w_scales, offsets, rows, slots, gather);
  const int64_t R = p.g.R;
  Tensor out = out_ ? *out_ : empty({R, p.N}, at::kBFloat16, p.dev);
  require(out, "out", at::kBFloat16, p.dev, 2);
  if (out.size(0) != R || out.size(1) != p.N) value_error("out must be [" + str(R) + ", " + str(p.N) + "], got " + shape_of(out));
  if (R && p.N > 1 && out.stride(1) != 1) value_error("out needs contiguous rows");
  require_no_grad(out, "out");
  run(fp8_grouped_gemm_1x128_128x128, "fp8_grouped_gemm_1x128_128x128", p.dev, a.const_data_ptr(), p.lda,
      (const int32_t*)a_scales.const_data_ptr(), p.sm, p.sw, p.M, w.const_data_ptr(), p.ldwg, p.ldw,
      (const uint8_t*)w_scales.const_data_ptr(), p.ld_wsg, p.ld_ws, p.g.offsets, p.g.rows, R, p.g.G, p.top, p.N, p.K,
      out.mutable_data_ptr(), R > 1 ? out.stride(0) : (p.N + 7) / 8 * 8);
  written(out);
  return out;
}

std::tuple<Tensor, Tensor> grouped_swiglu(const Tensor& a, const Tensor& a_scales, const Tensor& w, const Tensor& w_scales,
                                          const Tensor& offsets, const Tensor& rows, const Tensor& slots, bool gather,
                                          const OptTensor& q_, const OptTensor& q_scales_) {
  const Grouped p = grouped_of(a, a_scales, w, w_scales, offsets, rows, slots, gather);
  if (p.N % 2) value_error("w must have gate rows and as many up rows, got " + str(p.N));
  const int64_t R = p.g.R, I = p.N / 2, nw = (I / 128 + 3) / 4;
  Tensor q = q_ ? *q_ : empty({R, I}, at::kByte, p.dev);
  Tensor words = q_scales_ ? *q_scales_ : empty({R, nw}, at::kInt, p.dev);
  require_codes(q, "q", p.dev, 2);
  require(words, "q_scales", at::kInt, p.dev, 2);
  if (q.size(0) != R || q.size(1) != I) value_error("q must be [" + str(R) + ", " + str(I) + "], got " + shape_of(q));
  if (words.size(0) != R || words.size(1) != nw) value_error("q_scales must be [" + str(R) + ", " + str(nw) + "], got " + shape_of(words));
  if (R && I > 1 && q.stride(1) != 1) value_error("q needs contiguous rows");
  const auto [sm, sw] = word_strides(words);
  run(fp8_grouped_swiglu_1x128, "fp8_grouped_swiglu_1x128", p.dev, a.const_data_ptr(), p.lda,
      (const int32_t*)a_scales.const_data_ptr(), p.sm, p.sw, p.M, w.const_data_ptr(), p.ldwg, p.ldw,
      (const uint8_t*)w_scales.const_data_ptr(), p.ld_wsg, p.ld_ws, p.g.offsets, p.g.rows, R, p.g.G, p.top, I, p.K,
      q.mutable_data_ptr(), R > 1 ? q.stride(0) : I, (int32_t*)words.mutable_data_ptr(), sm, sw);
  written(q);
  written(words);
  return {q, words};
}

// bf16 [rows, cols] with contiguous rows; its row stride
int64_t matrix(const Tensor& t, const char* name, c10::Device dev, int64_t rows, int64_t cols) {
  require(t, name, at::kBFloat16, dev, 2);
  if (t.size(0) != rows || t.size(1) != cols)
    value_error(std::string(name) + " must be [" + str(rows) + ", " + str(cols) + "], got " + shape_of(t));
  if (rows && cols > 1 && t.stride(1) != 1) value_error(std::string(name) + " needs contiguous rows");
  return rows > 1 ? t.stride(0) : (cols + 7) / 8 * 8;
}

Tensor combine(const Tensor& y, const Tensor& offsets, const Tensor& rows, const Tensor& slots, const Tensor& weights,
               const OptTensor& shared, const OptTensor& out_) {
  const c10::Device dev = gpu_of(y, "y");
  const Groups g = groups_of(offsets, rows, slots, dev);
  require(y, "y", at::kBFloat16, dev, 2);
  const int64_t R = g.R, d = y.size(1), M = slots.size(0), top = g.top;
  const int64_t ldy = matrix(y, "y", dev, R, d);
  require(weights, "weights", at::kFloat, dev, slots.dim());
  exact(weights, "weights", at::kFloat, dev, slots.sizes());
  const int64_t lds = shared ? matrix(*shared, "shared", dev, M, d) : 0;
  Tensor out = out_ ? *out_ : empty({M, d}, at::kBFloat16, dev);
  const int64_t ldo = matrix(out, "out", dev, M, d);
  require_no_grad(y, "y");
  require_no_grad(weights, "weights");
  if (shared) require_no_grad(*shared, "shared");
  require_no_grad(out, "out");
  run(moe_combine, "moe_combine", dev, y.const_data_ptr(), ldy, R, (const int32_t*)slots.const_data_ptr(),
      (const float*)weights.const_data_ptr(), M, (int32_t)top, d, shared ? shared->const_data_ptr() : nullptr, lds,
      out.mutable_data_ptr(), ldo);
  written(out);
  return out;
}

Tensor lora(const Tensor& out, const Tensor& x, const Tensor& a, const Tensor& b, const Tensor& offsets, const Tensor& rows,
            const Tensor& slots, const OptTensor& scales, const OptTensor& workspace_) {
  const c10::Device dev = gpu_of(x, "x");
  const Groups g = groups_of(offsets, rows, slots, dev);
  require(x, "x", at::kBFloat16, dev, 2);
  require(out, "out", at::kBFloat16, dev, 2);
  const int64_t M = x.size(0), K = x.size(1), N = out.size(1);
  if (g.top != 1 || g.R != M) value_error("the groups must hold one adapter for each of the " + str(M) + " tokens");
  require(a, "lora_a", at::kBFloat16, dev, 3);
  const int64_t rank = a.size(1);
  exact(a, "lora_a", at::kBFloat16, dev, {g.G, rank, K});
  exact(b, "lora_b", at::kBFloat16, dev, {g.G, N, rank});
  if (scales) exact(*scales, "scales", at::kFloat, dev, {g.G});
  const int64_t ldx = matrix(x, "x", dev, M, K), ldo = matrix(out, "out", dev, M, N);
  if (rank > 0x7FFFFFFF) value_error("lora_a has too many rows");
  require_no_grad(out, "out");
  require_no_grad(x, "x");
  require_no_grad(a, "lora_a");
  require_no_grad(b, "lora_b");
  if (scales) require_no_grad(*scales, "scales");
  Tensor ws;
  if (workspace_) {
    ws = *workspace_;
    require(ws, "workspace", at::kByte, dev, 1);
    if (!ws.is_contiguous()) value_error("workspace must be contiguous");
  } else if (const int64_t need = lora_add_workspace_bytes(M, g.G, (int32_t)rank, K)) {
    ws = empty({need}, at::kByte, dev);
  }
  run(lora_add, "lora_add", dev, x.const_data_ptr(), ldx, M, K, a.const_data_ptr(), b.const_data_ptr(),
      scales ? (const float*)scales->const_data_ptr() : nullptr, (int32_t)rank, g.offsets, g.rows, g.G, N, (void*)out.mutable_data_ptr(), ldo,
      ws.defined() ? ws.mutable_data_ptr() : nullptr, ws.defined() ? (int64_t)ws.numel() : (int64_t)0);
  written(out);
  return out;
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
  m.def("set_error", [](py::object f) {
    delete g_raise;
    g_raise = new py::object(std::move(f));
  });
  m.def("fp8_gemm", &fp8_gemm);
  m.def("norm_rope", &norm_rope);
  m.def("kv_append", &kv_append);
  m.def("kv_read", &kv_read);
  m.def("attention", &attention);
  m.def("route", &route);
  m.def("group", &group);
  m.def("grouped_gemm", &grouped_gemm);
  m.def("grouped_swiglu", &grouped_swiglu);
  m.def("combine", &combine);
  m.def("lora", &lora);
}
