// Python functions on torch tensors over include/attn_rope.h and include/attn_latent.h:
// argument marshalling only (the checks that need a tensor, outputs, the stream), as the
// ctypes binding does it for the other entry points.  It is C++ because the short
// calls are bound by the host: one request of 385 cached rows takes 13 us on the GPU,
// and a call took the host 31 us with its marshalling in Python, 17 as an operator of
// torch's dispatcher and 10 with this.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <optional>
#include <tuple>
#include <vector>

#include "attn_bwd.h"
#include "attn_latent.h"
#include "attn_rope.h"

namespace {

using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

constexpr int64_t kRow = ATTN_LATENT_ROW, kLat = ATTN_LATENT_DIM, kRot = kRow - kLat;
constexpr int64_t kNope = 128, kValue = 128;  // the expanded form's own key columns and values a head

void ok(attn_status_t status, const char* what) {
  TORCH_CHECK(status == ATTN_OK, what, ": ", attn_bwd_status_string(status), " (status ", static_cast<int>(status), ")");
}

void cuda(const char* name, const Tensor& t) { TORCH_CHECK(t.is_cuda(), name, " must be a CUDA tensor"); }

void on(const Tensor& q, const char* name, const Tensor& t) {
  TORCH_CHECK(t.device() == q.device(), name, " must be a CUDA tensor on the device of the other tensors");
}

attn_dtype_t dtype_of(const char* name, const Tensor& t) {
  if (t.scalar_type() == at::kHalf) return ATTN_DT_F16;
  TORCH_CHECK(t.scalar_type() == at::kBFloat16, name, ": unsupported dtype ", t.scalar_type(), ": fp16 or bf16");
  return ATTN_DT_BF16;
}

// A new contiguous tensor on q's device, straight from the allocator (through
// torch's dispatcher a call that makes two takes 1.3 us more).
Tensor fresh(const Tensor& q, at::IntArrayRef shape, at::ScalarType type) {
  return at::detail::empty_cuda(shape, type, q.device(), std::nullopt);
}

// Strides of a [B,S,H,D] tensor; those of dimensions of size one, which no address uses,
// are replaced by a value that passes the checks.
attn_strides_t bshd(const char* name, const Tensor& t) {
  TORCH_CHECK(t.dim() == 4, name, " must be a 4-D tensor");
  TORCH_CHECK(t.stride(3) == 1 || t.size(3) == 1, name, " must have a contiguous head dimension");
  return {t.size(0) > 1 ? t.stride(0) : 128, t.size(1) > 1 ? t.stride(1) : 128, t.size(2) > 1 ? t.stride(2) : 128};
}

void shaped(const char* name, const Tensor& t, at::IntArrayRef shape) {
  TORCH_CHECK(t.sizes() == shape, name, " must have shape ", shape);
}

const int32_t* vec(const char* name, const Tensor& t, int64_t n) {
  TORCH_CHECK(t.scalar_type() == at::kInt && t.dim() == 1 && t.is_contiguous() && (n < 0 || t.size(0) == n), name,
              " must be a contiguous int32 vector", n < 0 ? "" : " of ", n < 0 ? std::string() : std::to_string(n));
  return t.const_data_ptr<int32_t>();
}

attn_latent_cache_t rows_of(const Tensor& cache) {
  TORCH_CHECK(cache.dim() == 3 && cache.size(2) == kRow && cache.stride(2) == 1, "cache must be [num_blocks, page_size, ",
              kRow, "] with contiguous rows");
  const int64_t nb = cache.size(0), page = cache.size(1);
  const int64_t row = page > 1 ? cache.stride(1) : nb > 1 ? cache.stride(0) : kRow;
  TORCH_CHECK(nb <= 1 || page <= 1 || cache.stride(0) == page * row,
              "cache must have evenly spaced rows (stride(0) = page_size * stride(1))");
  return {cache.data_ptr(), row, nb, page};
}

int64_t row_stride(const char* name, const Tensor& t, int64_t T) {
  TORCH_CHECK(t.dim() == 3 && t.size(0) == 1 && t.size(1) == T && t.size(2) == kRow && t.stride(2) == 1, name,
              " must be [1, T, ", kRow, "] with contiguous rows");
  return T > 1 ? t.stride(1) : kRow;
}

const uint64_t* steps_of(const Tensor& q, const Tensor& steps, int64_t pairs) {
  on(q, "the table's steps", steps);
  TORCH_CHECK(steps.scalar_type() == at::kLong && steps.dim() == 1 && steps.is_contiguous() &&
                  (pairs < 0 || steps.size(0) == pairs),
              "the table's steps must be a contiguous int64 vector", pairs < 0 ? "" : " of ",
              pairs < 0 ? std::string() : std::to_string(pairs));
  return reinterpret_cast<const uint64_t*>(steps.const_data_ptr<int64_t>());
}

// The device of ``t`` current, and the stream of the call: the given one, or the
// device's current one; new tensors belong to it.
class Launch {
 public:
  Launch(const Tensor& t, std::optional<int64_t> stream) : device_(t.device()) {
    if (stream.has_value())
      stream_.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*stream), t.device().index()));
    queue_ = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
  }
  void* queue() const { return queue_; }

 private:
  c10::cuda::CUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard stream_;
  cudaStream_t queue_;
};

// o, lse [B,H,S] and the workspace of a forward, given or new.  A small workspace of the
// call's own lies behind lse.
struct Outputs {
  Tensor o, lse, own;
  attn_strides_t so, sl;
  void* ws;
  size_t bytes;

  Outputs(const Tensor& q, at::IntArrayRef shape, const MaybeTensor& given_o, const MaybeTensor& given_lse,
          const MaybeTensor& workspace, size_t need) {
    const int64_t B = shape[0], S = shape[1], H = shape[2], n = B * S * H;
    bool placed = false;
    TORCH_CHECK(given_o.has_value() == given_lse.has_value(), "out must be o and lse");
    if (given_o.has_value()) {
      o = *given_o, lse = *given_lse;
      on(q, "o", o), on(q, "lse", lse);
      TORCH_CHECK(o.scalar_type() == q.scalar_type() && o.sizes() == shape && lse.scalar_type() == at::kFloat &&
                      lse.sizes() == at::IntArrayRef({B, H, S}),
                  "out must be o (of q's dtype, ", shape, ") and lse (float32 ", at::IntArrayRef({B, H, S}), ")");
      so = bshd("o", o);
    } else {
      o = fresh(q, shape, q.scalar_type());
      so = {S * H * shape[3], H * shape[3], shape[3]};
      if (!workspace.has_value() && need <= 4096) {
        const int64_t at = (n + 63) / 64 * 64;
        lse = fresh(q, {at + static_cast<int64_t>(need) / 4}, at::kFloat);
        ws = lse.data_ptr<float>() + at, bytes = need, placed = true;
        lse.unsafeGetTensorImpl()->set_sizes_contiguous({B, H, S});
      } else {
        lse = fresh(q, {B, H, S}, at::kFloat);
      }
    }
    sl = {B > 1 ? lse.stride(0) : 1, S > 1 ? lse.stride(2) : 1, H > 1 ? lse.stride(1) : 1};
    if (workspace.has_value()) {
      on(q, "workspace", *workspace);
      TORCH_CHECK(workspace->is_contiguous(), "workspace must be contiguous");
      ws = workspace->data_ptr(), bytes = workspace->nbytes();
    } else if (!placed) {
      own = fresh(q, {static_cast<int64_t>(need)}, at::kByte);
      ws = own.data_ptr(), bytes = need;
    }
  }
};

attn_rope_tensor_t rope_tensor(const char* name, const Tensor& x, const MaybeTensor& out, int64_t start, Tensor* y) {
  const attn_strides_t sx = bshd(name, x);
  if (out.has_value()) {
    *y = *out;
    on(x, "out", *y);
    TORCH_CHECK(y->scalar_type() == x.scalar_type() && y->sizes() == x.sizes(), "out must have its inputs' dtypes and shapes");
  } else {
    *y = x.is_contiguous() ? fresh(x, x.sizes(), x.scalar_type()) : at::empty_like(x);
  }
  return {x.data_ptr(), sx, y->data_ptr(), bshd("out", *y), x.size(2), x.size(3), start};
}

std::vector<Tensor> rope(const Tensor& q, const Tensor& positions, const Tensor& steps, double scale, const MaybeTensor& k,
                         bool interleaved, int64_t start, int64_t k_start, bool inverse, const MaybeTensor& out_q,
                         const MaybeTensor& out_k, std::optional<int64_t> stream) {
  cuda("q", q);
  on(q, "positions", positions);
  const attn_dtype_t dt = dtype_of("q", q);
  TORCH_CHECK(q.dim() == 4, "q must be a 4-D tensor");
  const int64_t B = q.size(0), S = q.size(1);
  const uint64_t* const table = steps_of(q, steps, -1);
  TORCH_CHECK(positions.scalar_type() == at::kInt &&
                  (positions.sizes() == at::IntArrayRef({S}) || positions.sizes() == at::IntArrayRef({B, S})) &&
                  (S <= 1 || positions.stride(-1) == 1),
              "positions must be int32 [", S, "] or [", B, ", ", S, "] with contiguous rows");
  const int64_t pos_b = positions.dim() == 2 && B > 1 ? positions.stride(0) : 0;
  TORCH_CHECK((out_q.has_value() || !out_k.has_value()) && (!out_q.has_value() || out_k.has_value() == k.has_value()),
              "out must be (q, k), k None where none is given");
  const Launch launch(q, stream);
  std::vector<Tensor> y(k.has_value() ? 2 : 1);
  const attn_rope_tensor_t tq = rope_tensor("q", q, out_q, start, &y[0]);
  attn_rope_tensor_t tk{};
  if (k.has_value()) {
    on(q, "k", *k);
    TORCH_CHECK(k->scalar_type() == q.scalar_type() && k->dim() == 4 && k->size(0) == B && k->size(1) == S,
                "k must have q's dtype, batch and length");
    tk = rope_tensor("k", *k, out_k, k_start, &y[1]);
  }
  ok(attn_rope(&tq, k.has_value() ? &tk : nullptr, B, S, dt, positions.const_data_ptr<int32_t>(), pos_b, table,
               2 * steps.size(0), static_cast<float>(scale), interleaved, inverse, launch.queue()),
     "attn_rope");
  return y;
}

void latent_cache_write(const Tensor& kv, const Tensor& slot_map, const Tensor& cache, const MaybeTensor& norm_weight,
                        double norm_eps, const MaybeTensor& positions, const MaybeTensor& steps, double scale,
                        bool interleaved, const MaybeTensor& out, std::optional<int64_t> stream) {
  cuda("kv", kv);
  on(kv, "slot_map", slot_map), on(kv, "cache", cache);
  const attn_dtype_t dt = dtype_of("kv", kv);
  TORCH_CHECK(kv.dim() == 3 && cache.scalar_type() == kv.scalar_type(), "kv must be [1, T, ", kRow, "] of the cache's dtype");
  const int64_t T = kv.size(1), stride = row_stride("kv", kv, T);
  const attn_latent_cache_t rows = rows_of(cache);
  const int32_t* const slots = vec("slot_map", slot_map, T);
  const void* weight = nullptr;
  if (norm_weight.has_value()) {
    on(kv, "norm_weight", *norm_weight);
    TORCH_CHECK(norm_weight->scalar_type() == kv.scalar_type() && norm_weight->sizes() == at::IntArrayRef({kLat}) &&
                    norm_weight->is_contiguous(),
                "norm_weight must be a contiguous vector of ", kLat, " of kv's dtype");
    weight = norm_weight->data_ptr();
  }
  TORCH_CHECK(positions.has_value() == steps.has_value(), "positions and table go together");
  const int32_t* pos = nullptr;
  const uint64_t* table = nullptr;
  if (steps.has_value()) {
    on(kv, "positions", *positions);
    pos = vec("positions", *positions, T), table = steps_of(kv, *steps, kRot / 2);
  }
  void* to = nullptr;
  int64_t to_stride = 0;
  if (out.has_value()) {
    on(kv, "out", *out);
    TORCH_CHECK(out->scalar_type() == kv.scalar_type(), "out must have kv's dtype and shape");
    to = out->data_ptr(), to_stride = row_stride("out", *out, T);
  }
  const Launch launch(kv, stream);
  ok(attn_latent_cache_write(kv.data_ptr(), stride, slots, T, dt, weight, static_cast<float>(norm_eps), pos, table,
                             static_cast<float>(scale), interleaved, &rows, to, to_stride, launch.queue()),
     "attn_latent_cache_write");
}

std::tuple<Tensor, Tensor> forward_latent_cache(const Tensor& q, const Tensor& cache, const Tensor& block_table,
                                                const Tensor& cu_seqlens, const Tensor& kv_lens, double sm_scale,
                                                bool causal, const MaybeTensor& workspace, const MaybeTensor& o,
                                                const MaybeTensor& lse, std::optional<int64_t> stream) {
  cuda("q", q);
  on(q, "cache", cache), on(q, "block_table", block_table), on(q, "cu_seqlens", cu_seqlens), on(q, "kv_lens", kv_lens);
  const attn_dtype_t dt = dtype_of("q", q);
  const attn_strides_t sq = bshd("q", q);
  const int64_t T = q.size(1), H = q.size(2), n = kv_lens.dim() == 1 ? kv_lens.size(0) : -1;
  TORCH_CHECK(q.size(0) == 1 && q.size(3) == kRow && cache.scalar_type() == q.scalar_type(), "q must be [1, T, H, ", kRow,
              "] of the cache's dtype");
  const attn_latent_cache_t rows = rows_of(cache);
  const int32_t* const lens = vec("kv_lens", kv_lens, n);
  const int32_t* const cu = vec("cu_seqlens", cu_seqlens, n + 1);
  TORCH_CHECK(block_table.scalar_type() == at::kInt && block_table.dim() == 2 && block_table.size(0) == n &&
                  (block_table.size(1) <= 1 || block_table.stride(1) == 1),
              "block_table must be int32 [", n, ", max_blocks] with contiguous rows");
  const int64_t width = block_table.size(1);
  // (the stride of a single row says nothing)
  const int64_t stride = n > 1 ? block_table.stride(0) : std::max(block_table.stride(0), width);
  const Launch launch(q, stream);
  const Outputs out(q, {1, T, H, kLat}, o, lse, workspace, attn_fwd_latent_cache_workspace_size());
  ok(attn_fwd_latent_cache(q.data_ptr(), sq, T, H, dt, static_cast<float>(sm_scale), &rows,
                           block_table.const_data_ptr<int32_t>(), stride, width, cu, lens, n, causal, out.o.data_ptr(),
                           out.so, out.lse.data_ptr<float>(), out.sl, out.ws, out.bytes, launch.queue()),
     "attn_fwd_latent_cache");
  return {out.o, out.lse};
}

std::tuple<Tensor, Tensor> sparse_forward(const Tensor& q, const Tensor& kv, const Tensor& idx, double sm_scale,
                                          int64_t dv_dim, const MaybeTensor& workspace, const MaybeTensor& o,
                                          const MaybeTensor& lse, std::optional<int64_t> stream) {
  cuda("q", q);
  on(q, "kv", kv), on(q, "idx", idx);
  const attn_dtype_t dt = dtype_of("q", q);
  const attn_strides_t sq = bshd("q", q);
  const int64_t B = q.size(0), S = q.size(1), H = q.size(2), D = q.size(3);
  TORCH_CHECK(kv.dim() == 4 && kv.stride(3) == 1 && kv.scalar_type() == q.scalar_type() && kv.size(0) == B && kv.size(3) == D,
              "kv must be [", B, ", SKV, HKV, ", D, "] of q's dtype with a contiguous last dimension");
  const int64_t SKV = kv.size(1), HKV = kv.size(2);
  TORCH_CHECK(idx.scalar_type() == at::kInt && idx.dim() == 4 && idx.size(0) == B && idx.size(1) == S && idx.size(2) == HKV &&
                  (idx.size(3) <= 1 || idx.stride(3) == 1),
              "idx must be int32 [", B, ", ", S, ", ", HKV, ", topk] with unit slot stride");
  // (strides of dimensions of size one, which no address uses, follow from the others)
  const int64_t row = HKV > 1 ? kv.stride(2) : SKV > 1 ? kv.stride(1) : B > 1 ? kv.stride(0) : D;
  const attn_strides_t skv{B > 1 ? kv.stride(0) : SKV * HKV * row, SKV > 1 ? kv.stride(1) : HKV * row, row};
  TORCH_CHECK(dv_dim >= 1, "dv_dim must be positive");
  const Launch launch(q, stream);
  const Outputs out(q, {B, S, H, dv_dim}, o, lse, workspace, attn_fwd_sparse_workspace_size(B, S, HKV));
  ok(attn_fwd_sparse(q.data_ptr(), sq, kv.data_ptr(), skv, idx.const_data_ptr<int32_t>(),
                     {idx.stride(0), idx.stride(1), idx.stride(2)}, B, S, SKV, H, HKV, D, dv_dim, idx.size(3), dt,
                     static_cast<float>(sm_scale), out.o.data_ptr(), out.so, out.lse.data_ptr<float>(), out.sl, out.ws,
                     out.bytes, launch.queue()),
     "attn_fwd_sparse");
  return {out.o, out.lse};
}

std::tuple<Tensor, Tensor> forward_latent(const Tensor& q, const Tensor& k_nope, const Tensor& k_rope, const Tensor& v,
                                          double sm_scale, bool causal, const MaybeTensor& cu_seqlens,
                                          const MaybeTensor& workspace, const MaybeTensor& o, const MaybeTensor& lse,
                                          std::optional<int64_t> stream) {
  cuda("q", q);
  on(q, "k_nope", k_nope), on(q, "k_rope", k_rope), on(q, "v", v);
  const attn_dtype_t dt = dtype_of("q", q);
  const attn_strides_t sq = bshd("q", q), sk = bshd("k_nope", k_nope), sv = bshd("v", v);
  const int64_t B = q.size(0), S = q.size(1), H = q.size(2), Sk = k_nope.size(1);
  TORCH_CHECK(q.size(3) == kNope + kRot, "q must be [B, S, H, ", kNope + kRot, "]");
  TORCH_CHECK(k_nope.scalar_type() == q.scalar_type() && k_rope.scalar_type() == q.scalar_type() &&
                  v.scalar_type() == q.scalar_type(),
              "k_nope, k_rope and v must have q's dtype");
  shaped("k_nope", k_nope, {B, Sk, H, kNope}), shaped("v", v, {B, Sk, H, kValue});
  shaped("k_rope", k_rope, {B, Sk, kRot});
  TORCH_CHECK(k_rope.stride(2) == 1, "k_rope must have contiguous rows");
  // (a key length of 0 would stand for S)
  TORCH_CHECK(Sk >= 1 && Sk <= 0x7fffffff, "k_nope must hold between 1 and 2^31 - 1 keys");
  attn_mask_t mask{causal, -1, nullptr, 0, Sk != S ? static_cast<int32_t>(Sk) : 0};
  if (cu_seqlens.has_value()) {
    on(q, "cu_seqlens", *cu_seqlens);
    mask.cu_seqlens = vec("cu_seqlens", *cu_seqlens, -1);
    mask.num_seqs = static_cast<int32_t>(std::min<int64_t>(cu_seqlens->size(0) - 1, 0x7fffffff));
  }
  const Launch launch(q, stream);
  const Outputs out(q, {B, S, H, kValue}, o, lse, workspace, attn_fwd_latent_workspace_size(B, S, H, mask.num_seqs));
  ok(attn_fwd_latent(q.data_ptr(), sq, k_nope.data_ptr(), sk, k_rope.data_ptr(),
                     {B > 1 ? k_rope.stride(0) : 128, Sk > 1 ? k_rope.stride(1) : 128, 128}, v.data_ptr(), sv, B, S, H, dt,
                     static_cast<float>(sm_scale), &mask, out.o.data_ptr(), out.so, out.lse.data_ptr<float>(), out.sl,
                     out.ws, out.bytes, launch.queue()),
     "attn_fwd_latent");
  return {out.o, out.lse};
}

}  // namespace

// ---------------------------------------------------------------- Python functions

namespace {

// Positional arguments, taken in order.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : next_(args) {
    TORCH_CHECK(n == want, "expected ", want, " arguments, got ", n);
  }
  const Tensor& tensor(const char* name) {
    PyObject* const x = *next_++;
    TORCH_CHECK(THPVariable_Check(x), name, " must be a tensor");
    return THPVariable_Unpack(x);
  }
  MaybeTensor maybe(const char* name) {
    if (*next_ == Py_None) return ++next_, std::nullopt;
    return tensor(name);
  }
  double number(const char* name) {
    const double x = PyFloat_AsDouble(*next_++);
    no_error(name, "a number");
    return x;
  }
  int64_t integer(const char* name) {
    const int64_t x = PyLong_AsLongLong(*next_++);
    no_error(name, "an integer");
    return x;
  }
  bool flag(const char* name) {
    const int x = PyObject_IsTrue(*next_++);
    no_error(name, "true or false");
    return x != 0;
  }
  std::optional<int64_t> stream() {
    if (*next_ == Py_None) return ++next_, std::nullopt;
    return integer("stream");
  }

 private:
  static void no_error(const char* name, const char* what) {
    if (PyErr_Occurred() == nullptr) return;
    PyErr_Clear();
    TORCH_CHECK(false, name, " must be ", what);
  }
  PyObject* const* next_;
};

// Other threads may run Python meanwhile (a launch waits where the queue is full).
class Released {
 public:
  Released() : state_(PyEval_SaveThread()) {}
  ~Released() { PyEval_RestoreThread(state_); }

 private:
  PyThreadState* state_;
};

PyObject* pair(PyObject* x, PyObject* y) {
  PyObject* const t = x && y ? PyTuple_New(2) : nullptr;
  if (t == nullptr) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, x);
  PyTuple_SET_ITEM(t, 1, y);
  return t;
}
PyObject* pair(const std::tuple<Tensor, Tensor>& y) { return pair(THPVariable_Wrap(std::get<0>(y)), THPVariable_Wrap(std::get<1>(y))); }

PyObject* py_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 12);
  const Tensor &q = a.tensor("q"), &positions = a.tensor("positions"), &steps = a.tensor("the table's steps");
  const double scale = a.number("the table's scale");
  const MaybeTensor k = a.maybe("k");
  const bool interleaved = a.flag("interleaved");
  const int64_t start = a.integer("start"), k_start = a.integer("k_start");
  const bool inverse = a.flag("inverse");
  const MaybeTensor out_q = a.maybe("out"), out_k = a.maybe("out");
  const std::optional<int64_t> stream = a.stream();
  std::vector<Tensor> y;
  {
    const Released released;
    y = rope(q, positions, steps, scale, k, interleaved, start, k_start, inverse, out_q, out_k, stream);
  }
  return pair(THPVariable_Wrap(y[0]), y.size() > 1 ? THPVariable_Wrap(y[1]) : Py_NewRef(Py_None));
  END_HANDLE_TH_ERRORS
}

PyObject* py_latent_cache_write(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 11);
  const Tensor &kv = a.tensor("kv"), &slot_map = a.tensor("slot_map"), &cache = a.tensor("cache");
  const MaybeTensor weight = a.maybe("norm_weight");
  const double eps = a.number("norm_eps");
  const MaybeTensor positions = a.maybe("positions"), steps = a.maybe("the table's steps");
  const double scale = a.number("the table's scale");
  const bool interleaved = a.flag("interleaved");
  const MaybeTensor out = a.maybe("out");
  const std::optional<int64_t> stream = a.stream();
  {
    const Released released;
    latent_cache_write(kv, slot_map, cache, weight, eps, positions, steps, scale, interleaved, out, stream);
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyObject* py_forward_latent_cache(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 11);
  const Tensor &q = a.tensor("q"), &cache = a.tensor("cache"), &table = a.tensor("block_table"), &cu = a.tensor("cu_seqlens"),
               &lens = a.tensor("kv_lens");
  const double scale = a.number("sm_scale");
  const bool causal = a.flag("causal");
  const MaybeTensor workspace = a.maybe("workspace"), o = a.maybe("out"), lse = a.maybe("out");
  const std::optional<int64_t> stream = a.stream();
  std::tuple<Tensor, Tensor> y;
  {
    const Released released;
    y = forward_latent_cache(q, cache, table, cu, lens, scale, causal, workspace, o, lse, stream);
  }
  return pair(y);
  END_HANDLE_TH_ERRORS
}

PyObject* py_sparse_forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 9);
  const Tensor &q = a.tensor("q"), &kv = a.tensor("kv"), &idx = a.tensor("idx");
  const double scale = a.number("sm_scale");
  const int64_t dv = a.integer("dv_dim");
  const MaybeTensor workspace = a.maybe("workspace"), o = a.maybe("out"), lse = a.maybe("out");
  const std::optional<int64_t> stream = a.stream();
  std::tuple<Tensor, Tensor> y;
  {
    const Released released;
    y = sparse_forward(q, kv, idx, scale, dv, workspace, o, lse, stream);
  }
  return pair(y);
  END_HANDLE_TH_ERRORS
}

PyObject* py_forward_latent(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 11);
  const Tensor &q = a.tensor("q"), &k_nope = a.tensor("k_nope"), &k_rope = a.tensor("k_rope"), &v = a.tensor("v");
  const double scale = a.number("sm_scale");
  const bool causal = a.flag("causal");
  const MaybeTensor cu = a.maybe("cu_seqlens"), workspace = a.maybe("workspace"), o = a.maybe("out"), lse = a.maybe("out");
  const std::optional<int64_t> stream = a.stream();
  std::tuple<Tensor, Tensor> y;
  {
    const Released released;
    y = forward_latent(q, k_nope, k_rope, v, scale, causal, cu, workspace, o, lse, stream);
  }
  return pair(y);
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_libattn_torch() {
  static PyMethodDef methods[] = {method<py_rope>("rope"), method<py_latent_cache_write>("latent_cache_write"),
                                  method<py_forward_latent_cache>("forward_latent_cache"),
                                  method<py_sparse_forward>("sparse_forward"), method<py_forward_latent>("forward_latent"),
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "libattn_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&module);
}
