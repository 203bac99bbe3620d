// The operators of quantised layers on torch tensors: checks, results from
// torch's allocator, one call of the C ABI each.  layers.py documents them and
// is what users call.  On small tensors a call lasts as long as the host takes:
// rmsnorm_q8 of one row 4.8 us here, 13 us with the same steps in Python and ctypes.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <memory>
#include <string>

#include "lecb.h"

namespace {

struct ValueError : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Failed {   // a status of the C ABI
    int status;
    const char* where;
};

[[noreturn]] void refuse(const std::string& what) { throw ValueError(what); }

int type_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return LECB_F32;
        case at::kBFloat16: return LECB_BF16;
        case at::kHalf: return LECB_F16;
        case at::kChar: return LECB_I8;
        default: return -1;
    }
}
bool is_float(at::ScalarType t) { return type_of(t) >= 0 && t != at::kChar; }
bool is_scale(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
void check(bool ok, at::ScalarType t, const char* what) {
    if (!ok) refuse(std::string(what) + ": " + c10::toString(t) + " is not one of its types");
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) refuse(std::string(what) + ": a tensor is needed");
    return THPVariable_Unpack(o);
}
at::Tensor optional(PyObject* o, const char* what) { return o == Py_None ? at::Tensor() : tensor(o, what); }
at::ScalarType dtype(PyObject* o, const char* what) {
    if (!THPDtype_Check(o)) refuse(std::string(what) + ": a torch.dtype is needed");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

// The current device, on which every tensor has to be, and its current stream.
class Here {
   public:
    template <typename... Ts>
    explicit Here(const at::Tensor& x, const Ts&... ts) {
        if (!x.is_cuda()) away(x);   // before the GPU is asked for anything
        device_ = c10::hip::current_device();
        on(x);
        (on(ts), ...);
    }
    void* stream() const { return c10::hip::getCurrentHIPStream(device_).stream(); }

   private:
    [[noreturn]] static void away(const at::Tensor& t) {
        refuse("tensor on " + t.device().str() + ": the current GPU's memory is needed");
    }
    void on(const at::Tensor& t) const {
        if (t.defined() && (!t.is_cuda() || t.get_device() != device_)) away(t);
    }
    c10::DeviceIndex device_;
};

// x as rows: any leading dimensions that are one stride apart, adjacent columns.
struct Rows {
    int64_t rows, cols, stride;
    Rows(const at::Tensor& x, const char* what) {
        if (x.dim() == 0) refuse(std::string(what) + ": at least one dimension is needed");
        const auto size = x.sizes(), st = x.strides();
        cols = size.back();
        stride = cols;
        if (x.is_contiguous()) {
            rows = cols ? x.numel() / cols : 0;
            return;
        }
        if (cols > 1 && st.back() != 1) refuse(std::string(what) + ": the last dimension must be contiguous");
        rows = 1;
        bool any = false;
        for (int64_t d = x.dim() - 2; d >= 0; --d) {
            if (size[d] == 1) continue;
            if (!any)
                stride = st[d];
            else if (st[d] != stride * rows)
                refuse(std::string(what) + ": rows must be one stride apart");
            any = true;
            rows *= size[d];
        }
        if (stride < cols) refuse(std::string(what) + ": rows overlap");
    }
};

// Memory that rows take up.
struct Area {
    uint64_t begin, rows, bytes, stride;   // of a row, from one to the next
    Area(const at::Tensor& t, uint64_t rows, uint64_t cols, uint64_t row_stride)
        : begin(reinterpret_cast<uintptr_t>(t.data_ptr())), rows(rows), bytes(cols * t.element_size()),
          stride(row_stride * t.element_size()) {}
    bool operator==(const Area& o) const { return begin == o.begin && stride == o.stride && bytes == o.bytes; }
    uint64_t end() const { return begin + (rows - 1) * stride + bytes; }
    // The first of the rows that ends past `at`.
    uint64_t first_past(uint64_t at) const {
        return begin + bytes > at ? 0 : (at - begin - bytes) / stride + 1;
    }
    // Whether any row meets one of o's.  Rows of two areas may lie in turn, as the
    // columns of one buffer do.  With one stride, what holds for a row of o holds for
    // those after it, so the first that ends past this area's begin, and the one after
    // it, which begins there, tell; otherwise one row after another is looked at.
    bool meets(const Area& o) const {
        if (!rows || !o.rows || end() <= o.begin || o.end() <= begin) return false;
        if (rows == 1 && o.rows > 1) return o.meets(*this);
        const uint64_t from = o.first_past(begin);
        for (uint64_t j = from; j < o.rows && o.begin + j * o.stride < end(); ++j) {
            if (o.stride == stride && j > from + 1) break;
            const uint64_t at = o.begin + j * o.stride, i = first_past(at);
            if (i < rows && begin + i * stride < at + o.bytes) return true;
        }
        return false;
    }
};

// Whether gradients are being recorded for any of an entry's inputs.  No entry has
// a derivative; a tangent would be lost without a word, so it is refused.
template <typename... Ts>
bool recorded(const char* name, const Ts&... inputs) {
    if (((inputs.defined() && inputs._fw_grad(0).defined()) || ...))
        refuse(std::string(name) + ": forward-mode derivatives are not there");
    return at::GradMode::is_enabled() && ((inputs.defined() && inputs.requires_grad()) || ...);
}

// Lets a backward pass that reaches `results` end in an error that names the entry.
template <typename... Ts>
void no_backward(const char* name, std::initializer_list<at::Tensor> results, const Ts&... inputs) {
    const std::shared_ptr<torch::autograd::Node> node(new torch::autograd::NotImplemented(name), torch::autograd::deleteNode);
    node->set_next_edges(torch::autograd::collect_next_edges(inputs...));
    for (const at::Tensor& r : results)
        if (r.defined()) torch::autograd::set_history(r, node);
}

at::Tensor make(at::IntArrayRef size, at::ScalarType t, const at::Tensor& like) {
    // what at::empty comes to on a GPU, without its dispatch
    return at::Tensor(at::detail::empty_cuda(size, t, like.device(), std::nullopt));
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
void done(int status, const char* where) {
    if (status != LECB_OK) throw Failed{status, where};
}
int64_t up(int64_t n, int64_t step) { return n / step + (n % step != 0); }

// Weights as the kernels take them on trust: their fields may have been set since
// W4Weights checked them.
void check_weights(const at::Tensor& tiles, const at::Tensor& scales, int64_t n, int64_t k, int64_t group) {
    constexpr int64_t END = int64_t(1) << 31;
    if (n < 1 || k < 1 || n >= END || k >= END || (group != 32 && group != 64 && group != 128))
        refuse("weights: n and k are at least 1, group is 32, 64 or 128");
    const int64_t cells = up(n, 16) * up(k, 128);
    if (tiles.scalar_type() != at::kByte || tiles.numel() != cells * 1024 || !tiles.is_contiguous() ||
        !is_scale(scales.scalar_type()) || scales.numel() != cells * (2048 / group) || !scales.is_contiguous())
        refuse("weights: tiles and scales are not those of n, k and group");
}

// Runs the body of an entry: C++ exceptions become Python's.
template <typename F>
PyObject* entry(Py_ssize_t have, Py_ssize_t want, F body) {
    try {
        if (have != want) refuse("wrong number of arguments");
        return body();
    } catch (const ValueError& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const Failed& e) {
        PyObject* module = PyImport_ImportModule("lossless_entropy_coding_byte_amd");
        PyObject* type = module ? PyObject_GetAttrString(module, "LecbError") : nullptr;
        PyObject* error = type ? PyObject_CallFunction(type, "is", e.status, e.where) : nullptr;
        if (error) PyErr_SetObject(type, error);
        Py_XDECREF(error);
        Py_XDECREF(type);
        Py_XDECREF(module);
    } catch (python_error& e) {
        if (!PyErr_Occurred()) e.restore();
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

PyObject* share(PyObject* o) {
    Py_INCREF(o);
    return o;
}
// A tuple of new references.
template <typename... Os>
PyObject* tuple(Os... os) {
    PyObject* t = PyTuple_New(sizeof...(os));
    if (!t) throw python_error();
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(t, i++, os), ...);
    return t;
}

struct NoGil {
    PyThreadState* state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

// (x, weight, residual, eps, scale, out_h) -> (q, scale, h)
PyObject* rmsnorm_q8(PyObject*, PyObject* const* args, Py_ssize_t count) {
    return entry(count, 6, [&]() -> PyObject* {
        const char* name = "rmsnorm_q8";
        const at::Tensor& x = tensor(args[0], name);
        const at::Tensor& weight = tensor(args[1], "rmsnorm_q8: weight");
        const at::Tensor residual = optional(args[2], "rmsnorm_q8: residual");
        const double eps = PyFloat_AsDouble(args[3]);
        if (eps == -1.0 && PyErr_Occurred()) throw python_error();
        at::Tensor scale = optional(args[4], "rmsnorm_q8: scale"), h = optional(args[5], "rmsnorm_q8: out_h");
        const Rows xr(x, name);
        check(is_float(x.scalar_type()), x.scalar_type(), name);
        check(is_float(weight.scalar_type()), weight.scalar_type(), "rmsnorm_q8: weight");
        if (xr.cols < 1 || xr.cols > (int64_t)LECB_NORM_MAX_COLS)
            refuse("rmsnorm_q8: rows have 1 to " + std::to_string(LECB_NORM_MAX_COLS) + " columns");
        if (weight.numel() != xr.cols || !weight.is_contiguous())
            refuse("rmsnorm_q8: weight holds one contiguous number per column");
        const bool fixed = scale.defined(), given = h.defined();
        if (fixed && (scale.scalar_type() != at::kFloat || scale.numel() != 1))
            refuse("rmsnorm_q8: a fixed scale is one float32 number");
        if (given && !residual.defined()) refuse("rmsnorm_q8: without a residual h is x");
        const bool grads = recorded(name, x, weight, residual, scale, h);
        if (grads && given) refuse("rmsnorm_q8: out_h goes with inputs that gradients are not recorded for");
        int64_t rs = 0, hs = xr.cols;
        if (residual.defined()) {
            if (residual.sizes() != x.sizes() || residual.scalar_type() != x.scalar_type())
                refuse("rmsnorm_q8: residual has x's shape and type");
            rs = Rows(residual, "rmsnorm_q8: residual").stride;
        }
        if (given) {
            if (h.sizes() != x.sizes() || h.scalar_type() != x.scalar_type())
                refuse("rmsnorm_q8: out_h has x's shape and type");
            hs = Rows(h, "rmsnorm_q8: out_h").stride;
            const uint64_t rows = xr.rows, cols = xr.cols;
            const Area area(h, rows, cols, hs), ax(x, rows, cols, xr.stride), ar(residual, rows, cols, rs);
            if ((!(area == ax) && area.meets(ax)) || (!(area == ar) && area.meets(ar)) ||
                area.meets(Area(weight, 1, cols, cols)) || (fixed && area.meets(Area(scale, 1, 1, 1))))
                refuse("rmsnorm_q8: out_h overlaps what is read, other than as x or residual in place");
        }
        const Here here(x, weight, residual, scale, h);
        if (residual.defined() && !given) h = make(x.sizes(), x.scalar_type(), x);
        if (!fixed) scale = make(x.sizes().slice(0, x.dim() - 1), at::kFloat, x);
        const at::Tensor q = make(x.sizes(), at::kChar, x);
        void* stream = here.stream();
        int rc;
        {
            NoGil free;
            rc = lecb_rmsnorm_q8(ptr(x), xr.stride, ptr(residual), rs, ptr(weight), type_of(weight.scalar_type()),
                                 type_of(x.scalar_type()), xr.rows, (uint32_t)xr.cols, (float)eps, ptr(h), hs,
                                 static_cast<int8_t*>(ptr(q)), static_cast<float*>(ptr(scale)), fixed, stream);
        }
        done(rc, "lecb_rmsnorm_q8");
        if (given && !h.is_inference()) h.unsafeGetTensorImpl()->bump_version();   // for what autograd has kept of it
        if (grads) no_backward(name, {fixed ? at::Tensor() : scale, h}, x, weight, residual, scale);
        return tuple(THPVariable_Wrap(q), fixed ? share(args[4]) : THPVariable_Wrap(scale),
                     !residual.defined() ? share(args[0]) : given ? share(args[5]) : THPVariable_Wrap(h));
    });
}

// (q, scale, dtype) -> values
PyObject* dequantize_q8(PyObject*, PyObject* const* args, Py_ssize_t count) {
    return entry(count, 3, [&]() -> PyObject* {
        const char* name = "dequantize_q8";
        const at::Tensor& q = tensor(args[0], name);
        const at::Tensor& scale = tensor(args[1], name);
        const at::ScalarType t = dtype(args[2], name);
        check(is_float(t), t, name);
        if (q.scalar_type() != at::kChar || !q.is_contiguous() || q.dim() == 0)
            refuse("dequantize_q8: contiguous int8 codes are needed");
        const int64_t cols = q.sizes().back(), rows = cols ? q.numel() / cols : 0;
        if (scale.scalar_type() != at::kFloat || !scale.is_contiguous() || (scale.numel() != 1 && scale.numel() != rows))
            refuse("dequantize_q8: one float32 scale per row, or one");
        const bool grads = recorded(name, scale);
        const Here here(q, scale);
        const at::Tensor out = make(q.sizes(), t, q);
        void* stream = here.stream();
        int rc;
        {
            NoGil free;
            rc = lecb_dequantize_q8(static_cast<int8_t*>(ptr(q)), rows, cols, static_cast<float*>(ptr(scale)),
                                    scale.numel() != 1, ptr(out), type_of(t), stream);
        }
        done(rc, "lecb_dequantize_q8");
        if (grads) no_backward(name, {out}, scale);
        return THPVariable_Wrap(out);
    });
}

// (x, tiles, scales, n, k, group, x_scale, out_dtype, ws) -> y
PyObject* matvec_w4(PyObject*, PyObject* const* args, Py_ssize_t count) {
    return entry(count, 9, [&]() -> PyObject* {
        const char* name = "matvec_w4";
        const at::Tensor& x = tensor(args[0], name);
        const at::Tensor& tiles = tensor(args[1], name);
        const at::Tensor& scales = tensor(args[2], name);
        const int64_t n = integer(args[3]), k = integer(args[4]), group = integer(args[5]);
        check_weights(tiles, scales, n, k, group);
        const at::Tensor xscale = optional(args[6], "matvec_w4: x_scale");
        at::Tensor ws = optional(args[8], "matvec_w4: ws");
        const Rows xr(x, name);
        if (xr.cols != k)
            refuse("matvec_w4: x has " + std::to_string(xr.cols) + " columns, the weights " + std::to_string(k));
        const at::ScalarType xt = x.scalar_type();
        check(type_of(xt) >= 0 && xt != at::kFloat, xt, name);
        if (xscale.defined() && (xt != at::kChar || xscale.scalar_type() != at::kFloat || !xscale.is_contiguous() ||
                                 (xscale.numel() != 1 && xscale.numel() != xr.rows)))
            refuse("matvec_w4: x_scale goes with int8 x, one float32 per row or one");
        const at::ScalarType yt =
            args[7] != Py_None ? dtype(args[7], "matvec_w4: out_dtype") : xt == at::kChar ? at::kBFloat16 : xt;
        check(is_float(yt), yt, "matvec_w4: out_dtype");
        if (ws.defined() && (ws.scalar_type() != at::kByte || !ws.is_contiguous()))
            refuse("matvec_w4: ws is contiguous uint8");
        const bool grads = recorded(name, x, scales, xscale);
        const Here here(x, tiles, scales, xscale, ws);
        at::DimVector size(x.sizes());
        size.back() = n;
        const at::Tensor y = make(size, yt, x);
        if (!ws.defined()) {
            const int64_t need = (int64_t)lecb_matvec_w4_workspace_bytes(xr.rows, n, k);
            if (need) ws = make({need}, at::kByte, x);
        }
        void* stream = here.stream();
        int rc;
        {
            NoGil free;
            rc = lecb_matvec_w4(ptr(x), type_of(xt), xr.stride, static_cast<float*>(ptr(xscale)),
                                xscale.defined() && xscale.numel() != 1, xr.rows, static_cast<uint8_t*>(ptr(tiles)),
                                ptr(scales), type_of(scales.scalar_type()), (uint32_t)group, n, k, ptr(y), type_of(yt), n,
                                ptr(ws), ws.defined() ? ws.nbytes() : 0, stream);
        }
        done(rc, "lecb_matvec_w4");
        if (grads) no_backward(name, {y}, x, scales, xscale);
        return THPVariable_Wrap(y);
    });
}

// (w, group, scale dtype) -> (tiles, scales)
PyObject* quantize_w4(PyObject*, PyObject* const* args, Py_ssize_t count) {
    return entry(count, 3, [&]() -> PyObject* {
        const char* name = "quantize_w4";
        const at::Tensor& w = tensor(args[0], name);
        const int64_t group = integer(args[1]);
        const at::ScalarType st = dtype(args[2], "scale_dtype");
        if (w.dim() != 2 || w.numel() == 0) refuse("quantize_w4: a matrix [n, k] is needed");
        check(is_float(w.scalar_type()), w.scalar_type(), name);
        check(is_scale(st), st, "scale_dtype");
        if (group != 32 && group != 64 && group != 128) refuse("quantize_w4: group is 32, 64 or 128");
        const Rows wr(w, name);
        recorded(name, w);   // codes and scales are constants to what follows
        const Here here(w);
        const int64_t nt = up(w.size(0), 16), kt = up(wr.cols, 128);
        const at::Tensor tiles = make({nt, kt, 1024}, at::kByte, w), scales = make({nt, kt * (128 / group), 16}, st, w);
        void* stream = here.stream();
        int rc;
        {
            NoGil free;
            rc = lecb_quantize_w4(ptr(w), type_of(w.scalar_type()), wr.stride, w.size(0), wr.cols, (uint32_t)group,
                                  static_cast<uint8_t*>(ptr(tiles)), ptr(scales), type_of(st), stream);
        }
        done(rc, "lecb_quantize_w4");
        return tuple(THPVariable_Wrap(tiles), THPVariable_Wrap(scales));
    });
}

// (tiles, scales, group, n, k, dtype) -> weights
PyObject* dequantize_w4(PyObject*, PyObject* const* args, Py_ssize_t count) {
    return entry(count, 6, [&]() -> PyObject* {
        const char* name = "dequantize_w4";
        const at::Tensor& tiles = tensor(args[0], name);
        const at::Tensor& scales = tensor(args[1], name);
        const int64_t group = integer(args[2]), n = integer(args[3]), k = integer(args[4]);
        check_weights(tiles, scales, n, k, group);
        const at::ScalarType t = dtype(args[5], name);
        check(is_float(t), t, name);
        const bool grads = recorded(name, scales);
        const Here here(tiles, scales);
        const at::Tensor out = make({n, k}, t, tiles);
        void* stream = here.stream();
        int rc;
        {
            NoGil free;
            rc = lecb_dequantize_w4(static_cast<uint8_t*>(ptr(tiles)), ptr(scales), type_of(scales.scalar_type()),
                                    (uint32_t)group, n, k, ptr(out), type_of(t), k, stream);
        }
        done(rc, "lecb_dequantize_w4");
        if (grads) no_backward(name, {out}, scales);
        return THPVariable_Wrap(out);
    });
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef METHODS[] = {METHOD(rmsnorm_q8), METHOD(dequantize_q8), METHOD(matvec_w4), METHOD(quantize_w4),
                         METHOD(dequantize_w4), {nullptr, nullptr, 0, nullptr}};
PyModuleDef MODULE = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, METHODS, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&MODULE); }
