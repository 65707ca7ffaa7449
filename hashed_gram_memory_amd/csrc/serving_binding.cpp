// Python binding of the serving calls: a CPython extension over the C ABI.
//
// Marshalling only, as the package's ctypes binding, but a decode step makes
// these calls for every layer, and on few tokens a kernel takes 4 to 8 us:
// filling the descriptions from Python took 15 to 18 us a call, here the whole
// call takes 4 to 7 (the launch, about 2, and the outputs' allocation among
// it).  Functions take their arguments by place; hashed_gram_memory_amd/serving.py
// has the signatures and their documentation.
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>

#include <algorithm>
#include <stdexcept>
#include <string>

#include "engram.h"

namespace {

PyObject* g_error = nullptr;    // EngramError
PyObject* g_stream = nullptr;   // torch's raw current stream of a device
PyObject* g_memory = nullptr;   // torch.OutOfMemoryError

struct TypeProblem : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

std::string shape_of(const at::Tensor& t) {
    std::string s = std::string(c10::toString(t.scalar_type())) + " [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

// A call's arguments by place, None as absent.
struct Args {
    PyObject* const* at;
    c10::Device device{c10::kCUDA};
    at::ScalarType type = at::kBFloat16;

    bool given(int i) const { return at[i] != Py_None; }
    const at::Tensor& tensor(int i, const char* name) const {
        if (!THPVariable_Check(at[i])) throw TypeProblem(std::string(name) + " must be a torch.Tensor");
        return THPVariable_Unpack(at[i]);
    }
    // a tensor of the call's device, that no gradient is wanted of
    const at::Tensor& on_device(int i, const char* name) const {
        const at::Tensor& t = tensor(i, name);
        if (!t.is_cuda()) refuse(std::string(name) + " must be a device tensor, got " + t.device().str());
        if (t.device() != device) refuse(std::string(name) + " is on " + t.device().str() + ", not on " + device.str());
        if (t.requires_grad() && c10::GradMode::is_enabled())
            refuse(std::string(name) + " requires a gradient, and the operator has no backward");
        if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
            refuse(std::string(name) + " has a forward gradient, and the operator has no derivative");
        return t;
    }
    // the tensor that says the call's device and type
    const at::Tensor& lead(int i, const char* name) {
        const at::Tensor& t = tensor(i, name);
        if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf)
            refuse(std::string(name) + " must be bfloat16 or float16, got " + c10::toString(t.scalar_type()));
        if (t.dim() != 3) refuse(std::string(name) + " must be [n_tok, heads, head_dim], got " + shape_of(t));
        device = t.device();
        type = t.scalar_type();
        return t;
    }
    uint32_t kind() const { return type == at::kBFloat16 ? ENGRAM_BF16 : ENGRAM_F16; }
    long long number(int i) const {
        const long long x = PyLong_AsLongLong(at[i]);
        if (x == -1 && PyErr_Occurred()) throw Raised();
        return x;
    }
    double real(int i) const {
        const double x = PyFloat_AsDouble(at[i]);
        if (x == -1.0 && PyErr_Occurred()) throw Raised();
        return x;
    }
    bool truth(int i) const {
        const int x = PyObject_IsTrue(at[i]);
        if (x < 0) throw Raised();
        return x != 0;
    }
};

// A [n_tok, heads, dim] tensor; a stride of an axis of one is 0.
struct Rows {
    void* p = nullptr;
    int64_t tok = 0, head = 0;
};

Rows rows_of(const Args& a, int i, const char* name, int64_t dim) {
    const at::Tensor& t = a.on_device(i, name);
    if (t.dim() != 3 || t.scalar_type() != a.type || t.size(2) != dim)
        refuse(std::string(name) + " must be a " + c10::toString(a.type) + " tensor [n_tok, heads, " + std::to_string(dim) +
               "], got " + shape_of(t));
    if (t.stride(2) != 1 && dim > 1) refuse(std::string(name) + " must be contiguous along head_dim");
    return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

// As rows_of, for an output: of that shape, with no two elements in one place.
Rows out_rows(const Args& a, int i, const char* name, at::IntArrayRef shape) {
    const at::Tensor& t = a.on_device(i, name);
    if (t.sizes() != shape) refuse(std::string(name) + " must have its input's shape, got " + shape_of(t));
    const Rows r = rows_of(a, i, name, shape[2]);
    std::pair<int64_t, int64_t> inner{r.head, shape[1]}, outer{r.tok, shape[0]};
    if (outer < inner) std::swap(inner, outer);
    if ((inner.second > 1 && inner.first < shape[2]) ||
        (outer.second > 1 && outer.first < std::max(inner.first * inner.second, shape[2])))
        refuse(std::string(name) + " has overlapping rows");
    return r;
}

void* vector_of(const Args& a, int i, const char* name, at::ScalarType type, int64_t n) {
    if (!a.given(i)) return nullptr;
    const at::Tensor& t = a.on_device(i, name);
    if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " [" + std::to_string(n) + "], got " +
               shape_of(t));
    return t.data_ptr();
}

void* needed(const Args& a, int i, const char* name, at::ScalarType type, int64_t n) {
    a.tensor(i, name);
    return vector_of(a, i, name, type, n);
}

struct Rotation {
    const int32_t* positions = nullptr;
    const double* inv_freq = nullptr;
    uint32_t dim = 0;
};

Rotation rotation_of(const Args& a, int positions, int inv_freq, int64_t n_tok) {
    Rotation r;
    if (!a.given(inv_freq)) return r;  // nothing is rotated
    const at::Tensor& f = a.on_device(inv_freq, "inv_freq");
    if (f.scalar_type() != at::kDouble || f.dim() != 1 || !f.is_contiguous())
        refuse("inv_freq must be a contiguous float64 [rotary_dim / 2]");
    if (!a.given(positions)) refuse("inv_freq needs positions");
    r.positions = static_cast<const int32_t*>(vector_of(a, positions, "positions", at::kInt, n_tok));
    r.inv_freq = static_cast<const double*>(f.data_ptr());
    r.dim = static_cast<uint32_t>(std::min<int64_t>(2 * f.size(0), UINT32_MAX));
    return r;
}

engram_kv_cache cache_of(const Args& a, int k_at, int v_at, int k_scale, int v_scale) {
    engram_kv_cache c = {};
    const char* names[2] = {"k_cache", "v_cache"};
    const at::Tensor* t[2];
    int64_t stride[2];
    for (int s = 0; s < 2; ++s) {
        const at::Tensor& x = a.on_device(s ? v_at : k_at, names[s]);
        const auto type = x.scalar_type();
        if (x.dim() != 4 || (type != at::kBFloat16 && type != at::kHalf && type != at::kByte && type != at::kFloat8_e4m3fn &&
                             type != at::kChar))
            refuse(std::string(names[s]) + " must be a bfloat16, float16, uint8, float8_e4m3fn or int8 tensor "
                   "[n_pages, n_kv_heads, page_size, head_dim], got " + shape_of(x));
        const int64_t h = x.size(1), p = x.size(2), d = x.size(3);
        if ((x.stride(3) != 1 && d > 1) || (x.stride(2) != d && p > 1) || (x.stride(1) != p * d && h > 1))
            refuse(std::string(names[s]) + " must have contiguous pages");
        stride[s] = x.size(0) > 1 ? x.stride(0) : h * p * d;
        t[s] = &x;
    }
    if (t[0]->sizes() != t[1]->sizes() || t[0]->scalar_type() != t[1]->scalar_type())
        refuse("k_cache and v_cache must have the same shape and type");
    const auto type = t[0]->scalar_type();
    c.type = type == at::kBFloat16 ? ENGRAM_BF16 : type == at::kHalf ? ENGRAM_F16 : type == at::kChar ? ENGRAM_I8_PAGE : ENGRAM_E4M3;
    if (c.type == ENGRAM_E4M3 || c.type == ENGRAM_I8_PAGE) {
        // a scale for each page and head, or (e4m3) for each row
        if (c.type == ENGRAM_E4M3 && a.given(k_scale) && a.tensor(k_scale, "k_scale").dim() == 2) c.type = ENGRAM_E4M3_PAGE;
        const bool rows = c.type == ENGRAM_E4M3;
        for (int s = 0; s < 2; ++s) {
            const int i = s ? v_scale : k_scale;
            const char* name = s ? "v_scale" : "k_scale";
            if (!a.given(i)) refuse(std::string(rows ? "an e4m3 cache needs " : "a cache of codes needs ") + name);
            const at::Tensor& x = a.on_device(i, name);
            if (x.scalar_type() != at::kFloat || x.sizes() != t[0]->sizes().slice(0, rows ? 3 : 2) || !x.is_contiguous())
                refuse(std::string(name) + " must be a contiguous float32 [n_pages, n_kv_heads" + (rows ? ", page_size]" : "]") +
                       ", got " + shape_of(x));
            (s ? c.v_scale : c.k_scale) = static_cast<float*>(x.data_ptr());
        }
    } else if (a.given(k_scale) || a.given(v_scale)) {
        refuse("k_scale and v_scale belong to a cache of codes");
    }
    const auto u32 = [](int64_t x) { return static_cast<uint32_t>(std::min<int64_t>(x, UINT32_MAX)); };
    c.k = t[0]->data_ptr();
    c.v = t[1]->data_ptr();
    c.k_page_stride = stride[0];
    c.v_page_stride = stride[1];
    c.n_pages = t[0]->size(0);
    c.n_kv_heads = u32(t[0]->size(1));
    c.page_size = u32(t[0]->size(2));
    c.head_dim = u32(t[0]->size(3));
    return c;
}

const at::Tensor& table_of(const Args& a, int i) {
    const at::Tensor& t = a.on_device(i, "block_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2) refuse("block_table must be int32 [n_seq, width]");
    if (t.size(1) > 1 && t.stride(1) != 1) refuse("block_table must be contiguous along its width");
    return t;
}

void check(int status, const char* what) {
    if (status == ENGRAM_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", status, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

void* stream_of(c10::Device d) {
    PyObject* i = PyLong_FromLong(d.index());
    PyObject* r = i ? PyObject_CallOneArg(g_stream, i) : nullptr;
    Py_XDECREF(i);
    if (!r) throw Raised();
    void* s = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    if (!s && PyErr_Occurred()) throw Raised();
    return s;
}

// A call on the current stream of its device, without the interpreter's lock.
template <class F>
void launch(const Args& a, const char* what, F f) {
    void* const stream = stream_of(a.device);
    const c10::DeviceGuard guard(a.device);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = f(stream);
    Py_END_ALLOW_THREADS
    check(st, what);
}

// A call's workspace: the one given, or one allocated for `need` bytes.
struct Workspace {
    at::Tensor held;
    void* p = nullptr;
    size_t bytes = 0;
};
Workspace workspace_of(const Args& a, int i, size_t need) {
    Workspace w;
    if (a.given(i)) {
        const at::Tensor& t = a.on_device(i, "workspace");
        if (t.scalar_type() != at::kByte || !t.is_contiguous()) refuse("workspace must be a contiguous uint8 tensor");
        w.p = t.data_ptr();
        w.bytes = static_cast<size_t>(t.numel());
    } else if (need) {
        w.held = at::empty({static_cast<int64_t>(need)}, at::TensorOptions().device(a.device).dtype(at::kByte));
        w.p = w.held.data_ptr();
        w.bytes = need;
    }
    return w;
}

// Outputs of a call as parts of one allocation: a tensor of its own takes the allocator 0.8 us, a part 0.1.
class Parts {
public:
    Parts(c10::Device device, int64_t bytes) : all_(at::empty({bytes}, at::TensorOptions().device(device).dtype(at::kByte))) {}
    // n elements from the next multiple of 16 bytes on (the room is the caller's to see to: room())
    at::Tensor part(at::ScalarType type, int64_t n) {
        const int64_t size = static_cast<int64_t>(c10::elementSize(type));
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all_.storage()), all_.key_set(),
                                                                c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_storage_offset(at_ / size);
        t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
        at_ += room(n * size);
        return t;
    }
    static int64_t room(int64_t bytes) { return (bytes + 15) & ~int64_t(15); }

private:
    at::Tensor all_;
    int64_t at_ = 0;
};

PyObject* pack(std::initializer_list<at::Tensor> tensors) {
    PyObject* all = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
    Py_ssize_t at = 0;
    for (const at::Tensor& t : tensors) {
        PyObject* x = all ? THPVariable_Wrap(t) : nullptr;
        if (!x) {
            Py_XDECREF(all);
            return nullptr;
        }
        PyTuple_SET_ITEM(all, at++, x);
    }
    return all;
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Raised&) {
    } catch (const TypeProblem& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_memory, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* none_or(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

// q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded(n_args, 10, [&]() -> PyObject* {
        Args a{args};
        if (!a.given(0) && !a.given(1)) refuse("q or k is needed");
        const at::Tensor& lead = a.given(0) ? a.lead(0, "q") : a.lead(1, "k");
        const int64_t n_tok = lead.size(0), dim = lead.size(2);
        at::Tensor out[2];
        Rows src[2], dst[2];
        const void* weight[2] = {};
        int64_t heads[2] = {};
        const char* names[2][3] = {{"q", "q_weight", "q_out"}, {"k", "k_weight", "k_out"}};
        for (int s = 0; s < 2; ++s) {
            if (!a.given(s)) {
                if (a.given(4 + s) || a.given(8 + s))
                    refuse(std::string(names[s][1]) + " and " + names[s][2] + " need " + names[s][0]);
                continue;
            }
            src[s] = rows_of(a, s, names[s][0], dim);
            const at::Tensor& x = a.tensor(s, names[s][0]);
            if (x.size(0) != n_tok) refuse("q and k must have the same tokens");
            heads[s] = x.size(1);
            weight[s] = vector_of(a, 4 + s, names[s][1], a.type, dim);
            if (a.given(8 + s)) {
                out[s] = a.tensor(8 + s, names[s][2]);
                dst[s] = out_rows(a, 8 + s, names[s][2], x.sizes());
            } else {
                out[s] = at::empty(x.sizes(), x.options().requires_grad(false));
                dst[s] = {out[s].data_ptr(), heads[s] * dim, dim};
            }
        }
        const Rotation r = rotation_of(a, 2, 3, n_tok);
        engram_norm_rope_desc d = {};
        d.q = src[0].p;
        d.k = src[1].p;
        d.q_out = dst[0].p;
        d.k_out = dst[1].p;
        d.q_weight = weight[0];
        d.k_weight = weight[1];
        d.positions = r.positions;
        d.inv_freq = r.inv_freq;
        d.n_tok = n_tok;
        d.q_token_stride = src[0].tok;
        d.q_head_stride = src[0].head;
        d.k_token_stride = src[1].tok;
        d.k_head_stride = src[1].head;
        d.q_out_token_stride = dst[0].tok;
        d.q_out_head_stride = dst[0].head;
        d.k_out_token_stride = dst[1].tok;
        d.k_out_head_stride = dst[1].head;
        d.n_q_heads = static_cast<uint32_t>(std::min<int64_t>(heads[0], UINT32_MAX));
        d.n_k_heads = static_cast<uint32_t>(std::min<int64_t>(heads[1], UINT32_MAX));
        d.head_dim = static_cast<uint32_t>(std::min<int64_t>(dim, UINT32_MAX));
        d.rotary_dim = r.dim;
        d.interleaved = a.truth(7);
        d.type = a.kind();
        d.eps = static_cast<float>(a.real(6));
        launch(a, "engram_qk_norm_rope", [&](void* stream) { return engram_qk_norm_rope(&d, stream); });
        PyObject* both[2] = {none_or(out[0]), none_or(out[1])};
        PyObject* pair = both[0] && both[1] ? PyTuple_Pack(2, both[0], both[1]) : nullptr;
        Py_XDECREF(both[0]);
        Py_XDECREF(both[1]);
        return pair;
    });
}

// k, v, k_cache, v_cache, slots, positions, inv_freq, k_weight, eps, interleaved, k_scale, v_scale
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded(n_args, 12, [&]() -> PyObject* {
        Args a{args};
        const at::Tensor& k = a.lead(0, "k");
        const engram_kv_cache c = cache_of(a, 2, 3, 10, 11);
        if (c.type == ENGRAM_E4M3_PAGE || c.type == ENGRAM_I8_PAGE)
            refuse("a cache with a scale for each page and head takes kv_append_pages");
        const Rows kr = rows_of(a, 0, "k", c.head_dim), vr = rows_of(a, 1, "v", c.head_dim);
        if (a.tensor(1, "v").sizes() != k.sizes() || k.size(1) != c.n_kv_heads)
            refuse("k and v must be [n_tok, " + std::to_string(c.n_kv_heads) + ", " + std::to_string(c.head_dim) + "]");
        engram_append_desc d = {};
        d.cache = &c;
        d.k = kr.p;
        d.v = vr.p;
        d.n_tok = k.size(0);
        d.slots = static_cast<const int64_t*>(needed(a, 4, "slots", at::kLong, d.n_tok));
        d.k_weight = vector_of(a, 7, "k_weight", a.type, c.head_dim);
        const Rotation r = rotation_of(a, 5, 6, d.n_tok);
        d.positions = r.positions;
        d.inv_freq = r.inv_freq;
        d.rotary_dim = r.dim;
        d.k_token_stride = kr.tok;
        d.k_head_stride = kr.head;
        d.v_token_stride = vr.tok;
        d.v_head_stride = vr.head;
        d.interleaved = a.truth(9);
        d.type = a.kind();
        d.eps = static_cast<float>(a.real(8));
        launch(a, "engram_kv_append", [&](void* stream) { return engram_kv_append(&d, stream); });
        Py_RETURN_NONE;
    });
}

// q, k_cache, v_cache, block_table, kv_len, cu_q, max_q_len, scale, window, k_scale, v_scale, out, return_lse, workspace,
// size_only: the workspace's bytes instead of the call
PyObject* paged_attention(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded(n_args, 15, [&]() -> PyObject* {
        Args a{args};
        const at::Tensor& q = a.lead(0, "q");
        const bool size_only = a.truth(14);
        const engram_kv_cache c = cache_of(a, 1, 2, 9, 10);
        const Rows qr = rows_of(a, 0, "q", c.head_dim);
        const at::Tensor& table = table_of(a, 3);
        engram_attention_desc d = {};
        d.cache = &c;
        d.q = qr.p;
        d.block_table = static_cast<const int32_t*>(table.data_ptr());
        d.n_seq = table.size(0);
        d.n_tok = q.size(0);
        d.kv_len = static_cast<const int32_t*>(needed(a, 4, "kv_len", at::kInt, d.n_seq));
        d.cu_q = static_cast<const int32_t*>(vector_of(a, 5, "cu_q", at::kInt, d.n_seq + 1));
        d.max_q_len = a.given(6) ? a.number(6) : 0;
        d.table_width = table.size(1);
        d.table_stride = d.n_seq > 1 ? table.stride(0) : d.table_width;
        d.window = a.number(8);
        d.q_token_stride = qr.tok;
        d.q_head_stride = qr.head;
        d.n_q_heads = static_cast<uint32_t>(std::min<int64_t>(q.size(1), UINT32_MAX));
        d.type = a.kind();
        d.scale = a.given(7) ? static_cast<float>(a.real(7)) : 1.0f / std::sqrt(static_cast<float>(c.head_dim));
        at::Tensor out, lse;
        if (a.given(11)) {
            out = a.tensor(11, "out");
            const Rows r = out_rows(a, 11, "out", q.sizes());
            d.out = r.p;
            d.out_token_stride = r.tok;
            d.out_head_stride = r.head;
        } else {
            if (!size_only) out = at::empty(q.sizes(), q.options().requires_grad(false));
            d.out = size_only ? qr.p : out.data_ptr();
            d.out_token_stride = q.size(1) * q.size(2);
            d.out_head_stride = q.size(2);
        }
        if (a.truth(12) && !size_only) {
            lse = at::empty(q.sizes().slice(0, 2), q.options().dtype(at::kFloat).requires_grad(false));
            d.lse = static_cast<float*>(lse.data_ptr());
        }
        size_t need = 0;
        check(engram_paged_attention_workspace(&d, &need), "engram_paged_attention_workspace");
        if (size_only) return PyLong_FromSize_t(need);
        const Workspace ws = workspace_of(a, 13, need);
        launch(a, "engram_paged_attention", [&](void* stream) { return engram_paged_attention(&d, ws.p, ws.bytes, stream); });
        if (!lse.defined()) return THPVariable_Wrap(out);
        return pack({out, lse});
    });
}

// k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, cu_q, max_q_len, positions, inv_freq, k_weight, eps, interleaved
PyObject* kv_append_pages(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded(n_args, 15, [&]() -> PyObject* {
        Args a{args};
        const at::Tensor& k = a.lead(0, "k");
        const engram_kv_cache c = cache_of(a, 2, 3, 4, 5);
        if (c.type != ENGRAM_E4M3_PAGE && c.type != ENGRAM_I8_PAGE)
            refuse("kv_append_pages wants a cache of codes with scales [n_pages, n_kv_heads]");
        const Rows kr = rows_of(a, 0, "k", c.head_dim), vr = rows_of(a, 1, "v", c.head_dim);
        if (a.tensor(1, "v").sizes() != k.sizes() || k.size(1) != c.n_kv_heads)
            refuse("k and v must be [n_tok, " + std::to_string(c.n_kv_heads) + ", " + std::to_string(c.head_dim) + "]");
        const at::Tensor& table = table_of(a, 6);
        engram_append_pages_desc d = {};
        d.cache = &c;
        d.k = kr.p;
        d.v = vr.p;
        d.n_tok = k.size(0);
        d.n_seq = table.size(0);
        d.block_table = static_cast<const int32_t*>(table.data_ptr());
        d.kv_len = static_cast<const int32_t*>(needed(a, 7, "kv_len", at::kInt, d.n_seq));
        d.cu_q = static_cast<const int32_t*>(vector_of(a, 8, "cu_q", at::kInt, d.n_seq + 1));
        d.max_q_len = a.given(9) ? a.number(9) : 0;
        d.table_width = table.size(1);
        d.table_stride = d.n_seq > 1 ? table.stride(0) : d.table_width;
        d.k_weight = vector_of(a, 12, "k_weight", a.type, c.head_dim);
        const Rotation r = rotation_of(a, 10, 11, d.n_tok);
        d.positions = r.positions;
        d.inv_freq = r.inv_freq;
        d.rotary_dim = r.dim;
        d.k_token_stride = kr.tok;
        d.k_head_stride = kr.head;
        d.v_token_stride = vr.tok;
        d.v_head_stride = vr.head;
        d.eps = static_cast<float>(a.real(13));
        d.interleaved = a.truth(14);
        d.type = a.kind();
        launch(a, "engram_kv_append_pages", [&](void* stream) { return engram_kv_append_pages(&d, stream); });
        Py_RETURN_NONE;
    });
}

// lengths, new_tokens, block_table, held, free_pages, n_free, page_size, n_tok, workspace, size_only
PyObject* page_tables(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded(n_args, 10, [&]() -> PyObject* {
        Args a{args};
        a.device = a.tensor(2, "block_table").device();
        const at::Tensor& table = table_of(a, 2);
        engram_page_tables_desc d = {};
        d.n_seq = table.size(0);
        d.table_width = table.size(1);
        d.table_stride = d.n_seq > 1 ? table.stride(0) : d.table_width;
        d.block_table = static_cast<int32_t*>(table.data_ptr());
        d.lengths = static_cast<const int32_t*>(needed(a, 0, "lengths", at::kInt, d.n_seq));
        d.new_tokens = static_cast<const int32_t*>(vector_of(a, 1, "new_tokens", at::kInt, d.n_seq));
        d.held = static_cast<int32_t*>(needed(a, 3, "held", at::kInt, d.n_seq));
        const at::Tensor& stack = a.on_device(4, "free_pages");
        if (stack.scalar_type() != at::kInt || stack.dim() != 1 || !stack.is_contiguous())
            refuse("free_pages must be a contiguous int32 [n_pages], got " + shape_of(stack));
        d.free_pages = static_cast<int32_t*>(stack.data_ptr());
        d.n_pages = stack.size(0);
        d.n_free = static_cast<int32_t*>(needed(a, 5, "n_free", at::kInt, 1));
        const long long page = a.number(6);
        d.page_size = page > 0 && page <= UINT32_MAX ? static_cast<uint32_t>(page) : 0u;
        d.n_tok = a.number(7);
        if (d.n_tok < 0) refuse("n_tok is negative");
        const bool size_only = a.truth(9);
        static int64_t nothing[2];  // stands for outputs that are not there yet: sizes are looked at before any is allocated
        d.slots = nothing;
        d.positions = d.cu_q = d.kv_len = d.n_short = reinterpret_cast<int32_t*>(nothing);
        size_t need = 0;
        check(engram_page_tables_workspace(&d, &need), size_only ? "engram_page_tables_workspace" : "engram_page_tables");
        if (size_only) return PyLong_FromSize_t(need);
        Parts parts(a.device, Parts::room(8 * d.n_tok) + Parts::room(4 * d.n_tok) + Parts::room(4 * d.n_seq + 4) +
                                  Parts::room(4 * d.n_seq) + 16);
        const at::Tensor slots = parts.part(at::kLong, d.n_tok), positions = parts.part(at::kInt, d.n_tok);
        const at::Tensor cu_q = parts.part(at::kInt, d.n_seq + 1), kv_len = parts.part(at::kInt, d.n_seq);
        const at::Tensor n_short = parts.part(at::kInt, 1);
        d.slots = static_cast<int64_t*>(slots.data_ptr());
        d.positions = static_cast<int32_t*>(positions.data_ptr());
        d.cu_q = static_cast<int32_t*>(cu_q.data_ptr());
        d.kv_len = static_cast<int32_t*>(kv_len.data_ptr());
        d.n_short = static_cast<int32_t*>(n_short.data_ptr());
        const Workspace ws = workspace_of(a, 8, need);
        launch(a, "engram_page_tables", [&](void* stream) { return engram_page_tables(&d, ws.p, ws.bytes, stream); });
        return pack({slots, positions, cu_q, kv_len, n_short});
    });
}

// target, draft, uniform, last_uniform, draft_probs, cu_draft, workspace, size_only
PyObject* verify_draft(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded(n_args, 8, [&]() -> PyObject* {
        Args a{args};
        a.device = a.tensor(0, "target").device();
        engram_verify_draft_desc d = {};
        const auto rows = [&](int i, const char* name, at::ScalarType type) -> const at::Tensor& {
            const at::Tensor& t = a.on_device(i, name);
            if (t.scalar_type() != type || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
                refuse(std::string(name) + " must be [rows, vocab] of " + c10::toString(type) + ", contiguous along vocab, got " +
                       shape_of(t));
            return t;
        };
        const auto type = a.tensor(0, "target").scalar_type();
        if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
            refuse(std::string("target must be float32, bfloat16 or float16, got ") + c10::toString(type));
        const at::Tensor& p = rows(0, "target", type);
        const at::Tensor& draft = a.on_device(1, "draft");
        if (draft.dim() != 1) refuse("draft must be int32 [n_draft], got " + shape_of(draft));
        d.n_draft = draft.size(0);
        d.n_seq = p.size(0) - d.n_draft;
        if (d.n_seq < 0) refuse("target must have a row for each draft and one more for each request");
        d.vocab = p.size(1);
        d.target = p.data_ptr();
        d.target_stride = p.size(0) > 1 ? p.stride(0) : 0;
        d.type = type == at::kFloat ? ENGRAM_F32 : type == at::kBFloat16 ? ENGRAM_BF16 : ENGRAM_F16;
        d.draft = static_cast<const int32_t*>(needed(a, 1, "draft", at::kInt, d.n_draft));
        d.uniform = static_cast<const float*>(needed(a, 2, "uniform", at::kFloat, d.n_draft));
        d.last_uniform = static_cast<const float*>(needed(a, 3, "last_uniform", at::kFloat, d.n_seq));
        if (a.given(4)) {
            const at::Tensor& q = rows(4, "draft_probs", type);
            if (q.size(0) != d.n_draft || q.size(1) != d.vocab)
                refuse("draft_probs must be [" + std::to_string(d.n_draft) + ", " + std::to_string(d.vocab) + "], got " + shape_of(q));
            d.draft_probs = q.data_ptr();
            d.draft_stride = q.size(0) > 1 ? q.stride(0) : 0;
        }
        d.cu_draft = static_cast<const int32_t*>(vector_of(a, 5, "cu_draft", at::kInt, d.n_seq + 1));
        const bool size_only = a.truth(7);
        at::Tensor tokens, accepted;
        static int32_t nothing[1];  // stands for outputs that are not there yet
        if (size_only) {
            d.tokens = d.n_accepted = nothing;
        } else {
            Parts parts(a.device, Parts::room(4 * p.size(0)) + Parts::room(4 * d.n_seq));
            tokens = parts.part(at::kInt, p.size(0));
            accepted = parts.part(at::kInt, d.n_seq);
            d.tokens = static_cast<int32_t*>(tokens.data_ptr());
            d.n_accepted = static_cast<int32_t*>(accepted.data_ptr());
        }
        size_t need = 0;
        check(engram_verify_draft_workspace(&d, &need), "engram_verify_draft_workspace");
        if (size_only) return PyLong_FromSize_t(need);
        const Workspace ws = workspace_of(a, 6, need);
        launch(a, "engram_verify_draft", [&](void* stream) { return engram_verify_draft(&d, ws.p, ws.bytes, stream); });
        return pack({tokens, accepted});
    });
}

// setup(EngramError, raw current stream of a device, torch.OutOfMemoryError)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded(n_args, 3, [&]() -> PyObject* {
        for (int i = 0; i < 3; ++i) Py_INCREF(args[i]);
        Py_XSETREF(g_error, args[0]);
        Py_XSETREF(g_stream, args[1]);
        Py_XSETREF(g_memory, args[2]);
        Py_RETURN_NONE;
    });
}

#define ENGRAM_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENGRAM_FAST(qk_norm_rope), ENGRAM_FAST(kv_append), ENGRAM_FAST(paged_attention),
                           ENGRAM_FAST(kv_append_pages), ENGRAM_FAST(page_tables), ENGRAM_FAST(verify_draft), ENGRAM_FAST(setup),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&g_module); }
