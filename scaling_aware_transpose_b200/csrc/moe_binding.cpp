// moe_binding.cpp — the allocating helpers of moe.py: argument checks, outputs and
// workspaces from torch's allocator on the current stream, and the C-ABI call, in one native
// function each.  From Python these steps took 10 to 25 us a call, several times what the
// smallest calls run on the GPU.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>
#include <torch/version.h>

#include <optional>
#include <tuple>

#include "fp8q.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

constexpr auto kU8 = at::kByte;
constexpr auto kI32 = at::kInt;
constexpr auto kF32 = at::kFloat;
constexpr auto kBF16 = at::kBFloat16;

void check(fp8q_status rc, const char* where) {
  if (rc == FP8Q_OK) return;
  const py::object type = py::module_::import("scaling_aware_transpose_b200").attr("Fp8qError");
  const py::object error = type(static_cast<int>(rc), where);
  PyErr_SetObject(type.ptr(), error.ptr());
  throw py::error_already_set();
}

// The current device and its current stream, once per call.
struct Here {
  c10::DeviceIndex dev = c10::cuda::current_device();
  fp8q_stream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, dev), std::nullopt));
  }
};

// Small results of one call in one allocation (each takes the allocator about 1 us, more than
// the kernels of the smallest calls spare), every part on 256 bytes: add() the parts, then make()
// the tensors in the same order.
class Together {
 public:
  explicit Together(const Here& h) : h_(h) {}
  void add(int64_t bytes) { total_ += round_up(bytes); }
  Tensor make(at::IntArrayRef shape, at::ScalarType type) {
    if (!block_.defined()) block_ = h_.empty({total_}, kU8);
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(block_.storage()),
                                                        c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                        c10::scalarTypeToTypeMeta(type));
    c10::TensorImpl* impl = t.unsafeGetTensorImpl();
    const int64_t size = (int64_t)c10::elementSize(type);
    impl->set_storage_offset(used_ / size);
    impl->set_sizes_contiguous(shape);
    used_ += round_up(t.numel() * size);
    return t;
  }

 private:
  static int64_t round_up(int64_t bytes) { return (bytes + 255) / 256 * 256; }
  const Here& h_;
  Tensor block_;
  int64_t total_ = 0, used_ = 0;
};

// Address of a contiguous tensor of the type on the current device.
template <typename T = void>
T* in(const Tensor& t, const char* name, at::ScalarType type, const Here& h) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == h.dev, name,
                    ": libfp8q takes tensors on the current CUDA device, got one on ", t.device().str());
  TORCH_CHECK_VALUE(t.scalar_type() == type, name, ": expected ", at::toString(type), ", got ",
                    at::toString(t.scalar_type()));
  TORCH_CHECK_VALUE(t.is_contiguous(), name, ": libfp8q takes contiguous tensors");
  return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* in(const OptTensor& t, const char* name, at::ScalarType type, const Here& h) {
  return t ? in<T>(*t, name, type, h) : nullptr;
}
template <typename T = void>
T* out(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* out(const OptTensor& t) {
  return t ? out<T>(*t) : nullptr;
}
void shape(const Tensor& t, const char* name, at::IntArrayRef want) {
  TORCH_CHECK_VALUE(t.sizes() == want, name, ": shape ", t.sizes(), ", expected ", want);
}
void shape(const OptTensor& t, const char* name, at::IntArrayRef want) {
  if (t) shape(*t, name, want);
}
void matrix(const Tensor& t, const char* name) { TORCH_CHECK_VALUE(t.dim() == 2, name, ": two dimensions"); }

uint32_t router_flags(const Tensor& logits, bool sigmoid, bool renorm) {
  matrix(logits, "logits");
  const auto type = logits.scalar_type();
  TORCH_CHECK_VALUE(type == kF32 || type == kBF16, "logits: fp32 or BF16, got ", at::toString(type));
  return (sigmoid ? FP8Q_ROUTER_SIGMOID : 0u) | (renorm ? FP8Q_ROUTER_RENORM : 0u) |
         (type == kBF16 ? FP8Q_ROUTER_BF16 : 0u);
}
const uint8_t* mask_in(const OptTensor& m, int64_t tokens, const Here& h) {
  shape(m, "token_mask", {tokens});
  return m ? in<uint8_t>(*m, "token_mask", m->scalar_type() == at::kBool ? at::kBool : kU8, h) : nullptr;
}

std::tuple<Tensor, Tensor, OptTensor, OptTensor, OptTensor> router_topk(const Tensor& logits, int64_t topk, bool sigmoid,
                                                                        bool renorm, const OptTensor& bias,
                                                                        const OptTensor& mask, double scale,
                                                                        bool balance, double loss_coef) {
  const Here h;
  const uint32_t flags = router_flags(logits, sigmoid, renorm);
  const int64_t T = logits.size(0), E = logits.size(1);
  TORCH_CHECK_VALUE(E <= INT32_MAX && topk >= -1 && topk <= INT32_MAX, "router_topk: sizes beyond int32");
  const void* l = in(logits, "logits", logits.scalar_type(), h);
  shape(bias, "bias", {E});
  const float* b = in<const float>(bias, "bias", kF32, h);
  const uint8_t* m = mask_in(mask, T, h);
  const int64_t k = topk > 0 && topk <= E ? topk : 0;  // (anything else is refused below)
  Tensor idx = h.empty({T, k}, kI32), w = h.empty({T, k}, kF32);
  OptTensor counts, sums, loss;
  Tensor ws;
  size_t need = 0;
  if (balance) {
    need = fp8q_router_workspace_bytes(T, (int32_t)E);
    const bool few = need <= 256;  // a larger workspace is freed at the end
    Together stats(h);
    stats.add(4 * E);
    stats.add(4 * E);
    stats.add(4);
    if (few) stats.add(256);
    counts = stats.make({E}, kI32);
    sums = stats.make({E}, kF32);
    loss = stats.make({1}, kF32);
    ws = few ? stats.make({256}, kU8) : h.empty({(int64_t)need + 16}, kU8);
  }
  check(fp8q_router_topk(l, T, (int32_t)E, flags, b, m, (int32_t)topk, (float)scale, (float)loss_coef, out<int32_t>(idx),
                         out<float>(w), out<int32_t>(counts), out<float>(sums), out<float>(loss),
                         balance ? ws.data_ptr() : nullptr, need, h.stream),
        "fp8q_router_topk");
  return {idx, w, counts, sums, loss};
}

Tensor router_topk_bwd(const Tensor& logits, const Tensor& topk_idx, const OptTensor& grad_weights,
                       const OptTensor& row_id_map, const OptTensor& counts, const OptTensor& grad_loss, bool sigmoid,
                       bool renorm, const OptTensor& mask, double scale, double loss_coef) {
  const Here h;
  const uint32_t flags = router_flags(logits, sigmoid, renorm);
  matrix(topk_idx, "topk_idx");
  const int64_t T = logits.size(0), E = logits.size(1), K = topk_idx.size(1);
  TORCH_CHECK_VALUE(E <= INT32_MAX && K <= INT32_MAX, "router_topk_bwd: sizes beyond int32");
  shape(topk_idx, "topk_idx", {T, K});
  int64_t rows = 0;
  if (row_id_map) {
    TORCH_CHECK_VALUE(row_id_map->numel() == T * K && grad_weights,
                      "row_id_map: one entry per (token, slot) pair, with grad_weights in row order");
    rows = grad_weights->numel();
  } else {
    shape(grad_weights, "grad_weights", {T, K});
  }
  shape(counts, "counts", {E});
  TORCH_CHECK_VALUE(!grad_loss || grad_loss->numel() == 1, "grad_loss: one element");
  const void* l = in(logits, "logits", logits.scalar_type(), h);
  Tensor grad = h.empty({T, E}, logits.scalar_type());
  check(fp8q_router_topk_bwd(l, T, (int32_t)E, flags, mask_in(mask, T, h), (int32_t)K, (float)scale,
                             in<int32_t>(topk_idx, "topk_idx", kI32, h), in<float>(grad_weights, "grad_weights", kF32, h),
                             in<int32_t>(row_id_map, "row_id_map", kI32, h), rows, in<int32_t>(counts, "counts", kI32, h),
                             (float)loss_coef, in<float>(grad_loss, "grad_loss", kF32, h), out(grad), h.stream),
        "fp8q_router_topk_bwd");
  return grad;
}

Tensor permute_row_weights(const Tensor& weights, const Tensor& row_id_map, int64_t rows) {
  const Here h;
  TORCH_CHECK_VALUE(weights.numel() == row_id_map.numel(),
                    "weights and row_id_map: one entry per (token, slot) pair each");
  TORCH_CHECK_VALUE(rows >= 0, "rows: not negative");
  const float* w = in<float>(weights, "weights", kF32, h);
  const int32_t* r = in<int32_t>(row_id_map, "row_id_map", kI32, h);
  Tensor o = h.empty({rows}, kF32);
  check(fp8q_permute_row_weights(w, r, weights.numel(), rows, out<float>(o), h.stream), "fp8q_permute_row_weights");
  return o;
}

// Codes [rows, cols] and scales [rows, cols/128] of a row-wise pair; the scales of a call's pairs
// lie together.
std::pair<Tensor, Tensor> pair_of(int64_t rows, int64_t cols, const Here& h, Together& scales) {
  return {h.empty({rows, cols}, kU8), scales.make({rows, cols / 128}, kU8)};
}

std::tuple<Tensor, Tensor, Tensor, Tensor, Tensor, Tensor> swiglu_quant_stash(const Tensor& gate, const Tensor& up,
                                                                              const OptTensor& row_weights) {
  const Here h;
  matrix(gate, "gate");
  const int64_t rows = gate.size(0), cols = gate.size(1);
  shape(up, "up", {rows, cols});
  shape(row_weights, "row_weights", {rows});
  const void *g = in(gate, "gate", kBF16, h), *u = in(up, "up", kBF16, h);
  const float* w = in<float>(row_weights, "row_weights", kF32, h);
  Together scales(h);
  for (int i = 0; i < 3; ++i) scales.add(rows * (cols / 128));
  auto [q, sf] = pair_of(rows, cols, h, scales);
  auto [gq, gsf] = pair_of(rows, cols, h, scales);
  auto [uq, usf] = pair_of(rows, cols, h, scales);
  check(fp8q_swiglu_quant_stash(g, u, w, rows, cols, out<uint8_t>(q), out<uint8_t>(sf), out<uint8_t>(gq),
                                out<uint8_t>(gsf), out<uint8_t>(uq), out<uint8_t>(usf), h.stream),
        "fp8q_swiglu_quant_stash");
  return {q, sf, gq, gsf, uq, usf};
}

struct BwdArgs {
  int64_t rows, cols;
  const uint8_t *gq, *gsf, *uq, *usf;
  const float* w;
  const void* dy;
  BwdArgs(const Tensor& gq_, const Tensor& gsf_, const Tensor& uq_, const Tensor& usf_, const Tensor& dy_,
          const OptTensor& w_, const Here& h) {
    matrix(gq_, "gq");
    rows = gq_.size(0);
    cols = gq_.size(1);
    shape(uq_, "uq", {rows, cols});
    shape(dy_, "dy", {rows, cols});
    shape(gsf_, "gsf", {rows, cols / 128});
    shape(usf_, "usf", {rows, cols / 128});
    shape(w_, "row_weights", {rows});
    gq = in<uint8_t>(gq_, "gq", kU8, h);
    gsf = in<uint8_t>(gsf_, "gsf", kU8, h);
    uq = in<uint8_t>(uq_, "uq", kU8, h);
    usf = in<uint8_t>(usf_, "usf", kU8, h);
    w = in<float>(w_, "row_weights", kF32, h);
    dy = in(dy_, "dy", kBF16, h);
  }
};

std::tuple<Tensor, Tensor, OptTensor> swiglu_bwd(const Tensor& gq, const Tensor& gsf, const Tensor& uq, const Tensor& usf,
                                                 const Tensor& dy, const OptTensor& row_weights) {
  const Here h;
  const BwdArgs a(gq, gsf, uq, usf, dy, row_weights, h);
  Tensor dg = h.empty({a.rows, a.cols}, kBF16), du = h.empty({a.rows, a.cols}, kBF16);
  OptTensor dw;
  if (row_weights) dw = h.empty({a.rows}, kF32);
  check(fp8q_swiglu_bwd(a.gq, a.gsf, a.uq, a.usf, a.w, a.dy, a.rows, a.cols, out(dg), out(du), out<float>(dw), h.stream),
        "fp8q_swiglu_bwd");
  return {dg, du, dw};
}

std::tuple<Tensor, Tensor, Tensor, Tensor, OptTensor, OptTensor, OptTensor> swiglu_bwd_quant(
    const Tensor& gq, const Tensor& gsf, const Tensor& uq, const Tensor& usf, const Tensor& dy,
    const OptTensor& row_weights, bool recompute) {
  const Here h;
  const BwdArgs a(gq, gsf, uq, usf, dy, row_weights, h);
  Together small(h);
  for (int i = 0; i < (recompute ? 3 : 2); ++i) small.add(a.rows * (a.cols / 128));
  if (row_weights) small.add(4 * a.rows);
  auto [dgq, dgsf] = pair_of(a.rows, a.cols, h, small);
  auto [duq, dusf] = pair_of(a.rows, a.cols, h, small);
  OptTensor yq, ysf, dw;
  if (recompute) {
    auto [q, sf] = pair_of(a.rows, a.cols, h, small);
    yq = q;
    ysf = sf;
  }
  if (row_weights) dw = small.make({a.rows}, kF32);
  check(fp8q_swiglu_bwd_quant(a.gq, a.gsf, a.uq, a.usf, a.w, a.dy, a.rows, a.cols, out<uint8_t>(dgq), out<uint8_t>(dgsf),
                              out<uint8_t>(duq), out<uint8_t>(dusf), out<uint8_t>(yq), out<uint8_t>(ysf), out<float>(dw),
                              h.stream),
        "fp8q_swiglu_bwd_quant");
  return {dgq, dgsf, duq, dusf, yq, ysf, dw};
}

std::tuple<Tensor, Tensor> quantize_rowwise_mxfp4(const Tensor& x) {
  const Here h;
  matrix(x, "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  const void* p = in(x, "x", kBF16, h);
  Tensor q = h.empty({rows, cols / 2}, kU8), sf = h.empty({(int64_t)fp8q_mxfp4_sf_bytes(rows, cols)}, kU8);
  check(fp8q_quantize_rowwise_mxfp4(p, rows, cols, out<uint8_t>(q), out<uint8_t>(sf), h.stream),
        "fp8q_quantize_rowwise_mxfp4");
  return {q, sf};
}

std::tuple<Tensor, Tensor, Tensor, Tensor> permute_pad_mxfp4(const Tensor& x, const Tensor& topk_idx, int64_t experts,
                                                             int64_t align, const std::optional<int64_t>& max_rows) {
  const Here h;
  matrix(x, "x");
  matrix(topk_idx, "topk_idx");
  const int64_t T = x.size(0), H = x.size(1), K = topk_idx.size(1);
  shape(topk_idx, "topk_idx", {T, K});
  TORCH_CHECK_VALUE(experts >= 0 && experts <= INT32_MAX && align >= 0 && align <= INT32_MAX && K <= INT32_MAX,
                    "permute_pad_mxfp4: sizes out of range");
  const int64_t cap = max_rows ? *max_rows : T * K + experts * (align > 0 ? align - 1 : 0);
  TORCH_CHECK_VALUE(cap >= 0, "max_out_rows: not negative");
  const void* p = in(x, "x", kBF16, h);
  const int32_t* idx = in<int32_t>(topk_idx, "topk_idx", kI32, h);
  const size_t need = fp8q_permute_workspace_bytes(T, (int32_t)K, (int32_t)experts);
  Tensor q = h.empty({cap, H / 2}, kU8), sf = h.empty({(int64_t)fp8q_mxfp4_sf_bytes(cap, H)}, kU8);
  Together routing(h);
  routing.add(4 * (experts + 1));
  routing.add(4 * T * K);
  Tensor off = routing.make({experts + 1}, kI32), map = routing.make({T * K}, kI32), ws = h.empty({(int64_t)need + 16}, kU8);
  check(fp8q_permute_pad_mxfp4(p, T, H, idx, (int32_t)K, (int32_t)experts, (int32_t)align, out<uint8_t>(q),
                               out<uint8_t>(sf), cap, out<int32_t>(off), out<int32_t>(map), ws.data_ptr(), need,
                               h.stream),
        "fp8q_permute_pad_mxfp4");
  return {q, sf, off, map};
}

Tensor matmul_mxfp4(const Tensor& aq, const Tensor& asf, const Tensor& bq, const Tensor& bsf, const OptTensor& offsets,
                    const OptTensor& result) {
  const Here h;
  matrix(aq, "aq");
  matrix(bq, "bq");
  const int64_t m = aq.size(0), half = aq.size(1);
  const int64_t groups = offsets ? offsets->numel() - 1 : 1;
  TORCH_CHECK_VALUE(bq.size(1) == half && groups >= 1 && groups <= INT32_MAX && bq.size(0) % groups == 0, "codes ",
                    aq.sizes(), " and ", bq.sizes(), " do not fit (", groups, " groups)");
  const int64_t n = bq.size(0) / groups;
  const uint8_t *a = in<uint8_t>(aq, "aq", kU8, h), *b = in<uint8_t>(bq, "bq", kU8, h);
  const uint8_t *as = in<uint8_t>(asf, "asf", kU8, h), *bs = in<uint8_t>(bsf, "bsf", kU8, h);
  TORCH_CHECK_VALUE(asf.numel() >= (int64_t)fp8q_mxfp4_sf_bytes(m, 2 * half), "asf: ", asf.numel(), " bytes, ",
                    fp8q_mxfp4_sf_bytes(m, 2 * half), " needed");
  TORCH_CHECK_VALUE(bsf.numel() >= (int64_t)fp8q_mxfp4_sf_bytes(bq.size(0), 2 * half), "bsf: ", bsf.numel(), " bytes, ",
                    fp8q_mxfp4_sf_bytes(bq.size(0), 2 * half), " needed");
  const int32_t* off = in<int32_t>(offsets, "group_offsets", kI32, h);
  shape(result, "out", {m, n});
  Tensor o = result ? *result : h.empty({m, n}, kBF16);
  check(fp8q_matmul_mxfp4(a, as, m, b, bs, n, 2 * half, off, (int32_t)groups, in(o, "out", kBF16, h), h.stream),
        "fp8q_matmul_mxfp4");
  return o;
}

}  // namespace

PYBIND11_MODULE(_moe_binding, m) {
  m.attr("torch_version") = TORCH_VERSION;  // its classes' layouts are compiled in
  m.def("router_topk", &router_topk);
  m.def("router_topk_bwd", &router_topk_bwd);
  m.def("permute_row_weights", &permute_row_weights);
  m.def("swiglu_quant_stash", &swiglu_quant_stash);
  m.def("swiglu_bwd", &swiglu_bwd);
  m.def("swiglu_bwd_quant", &swiglu_bwd_quant);
  m.def("quantize_rowwise_mxfp4", &quantize_rowwise_mxfp4);
  m.def("permute_pad_mxfp4", &permute_pad_mxfp4);
  m.def("matmul_mxfp4", &matmul_mxfp4);
}
