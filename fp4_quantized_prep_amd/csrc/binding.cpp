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
#include <c10/hip/HIPStream.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <string>
#include <tuple>

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
}
