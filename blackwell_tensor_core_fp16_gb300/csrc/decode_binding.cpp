// Python binding of the decode-step operators (module _decode): the torch entry points of decode.py.
// A call on a few tokens runs for a few microseconds on the GPU, so its checks, its outputs'
// allocation and the launch are done here, on the tensors themselves; the same in Python took 12
// to 16 us.  Every operand is checked before anything is enqueued; a failed check raises
// ValueError, a refusal of the C call GemmError with its message.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/decode.h"

namespace {

using at::ScalarType;
using at::Tensor;
using Sizes = std::initializer_list<int64_t>;

// An exception that becomes Python's ValueError.
struct Refused {
    std::string why;
};

[[noreturn]] void refuse(const std::string& why) { throw Refused{why}; }

const char* name_of(ScalarType t)
{
    switch (t) {
    case ScalarType::Half: return "torch.float16";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    default: return c10::toString(t);
    }
}

template <typename Range>
std::string list_of(const Range& sizes)
{
    std::ostringstream s;
    s << "[";
    const char* sep = "";
    for (const int64_t x : sizes) {
        s << sep << x;
        sep = ", ";
    }
    s << "]";
    return s.str();
}

const Tensor& tensor(PyObject* x, const char* name)
{
    if (!THPVariable_Check(x)) {
        std::string text = std::string(name) + " must be a tensor";
        PyErr_SetString(PyExc_TypeError, text.c_str());
        throw python_error();
    }
    return THPVariable_Unpack(x);
}

// The type, device and shape of one operand.
void check(const Tensor& t, const char* name, ScalarType dtype, const at::Device& device, Sizes sizes)
{
    if (t.scalar_type() != dtype)
        refuse(std::string(name) + " must be " + name_of(dtype) + ", not " + name_of(t.scalar_type()));
    if (t.device() != device)
        refuse(std::string(name) + " is on " + t.device().str() + ", the other operands on " +
               device.str());
    if (!t.sizes().equals(at::IntArrayRef(sizes)))
        refuse(std::string(name) + " must be " + list_of(sizes) + ", not " + list_of(t.sizes()));
}

// Copies the strides of all but the last dimension, which must be dense.
template <size_t N>
void strides(const Tensor& t, const char* name, int64_t (&to)[N])
{
    if (t.stride(N) != 1 && t.size(N) > 1)
        refuse(std::string(name) + "'s last dimension must be contiguous");
    for (size_t d = 0; d < N; ++d) to[d] = t.stride(d);
}

void contiguous(const Tensor& t, const char* name)
{
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}

// Refuses a tensor that is written and whose elements may share memory: its strides are not those
// of a dense tensor's permuted and padded dimensions.
void separate(const Tensor& t, const char* name)
{
    if (t.is_contiguous()) return;
    int64_t order[8], reach = t.size(t.dim() - 1), count = 0;
    for (int64_t d = 0; d + 1 < t.dim(); ++d)
        if (t.size(d) > 1) order[count++] = d;
    std::sort(order, order + count, [&](int64_t a, int64_t b) { return t.stride(a) < t.stride(b); });
    for (int64_t x = 0; x < count; ++x) {
        if (t.stride(order[x]) < reach) refuse(std::string(name) + "'s elements overlap");
        reach += t.stride(order[x]) * (t.size(order[x]) - 1);
    }
}

int32_t half_dtype(const Tensor& q)
{
    const ScalarType t = q.scalar_type();
    if (t != ScalarType::Half && t != ScalarType::BFloat16)
        refuse("16-bit operands must be float16 or bfloat16");
    if (!q.is_cuda()) refuse("operands must be CUDA tensors");
    return t == ScalarType::Half ? DECODE_F16 : DECODE_BF16;
}

// The stream of a call (None: torch's current one) and its device, current while it lives, so that
// new tensors belong to the stream the call runs on.
class Where {
public:
    Where(PyObject* stream, const at::Device& device)
    {
        if (stream == Py_None) {
            guard_.set_device(device);
            stream_ = c10::cuda::getCurrentCUDAStream(device.index());
            return;
        }
        PyObject* handle = PyLong_Check(stream) ? Py_NewRef(stream)
                                                : PyObject_GetAttrString(stream, "cuda_stream");
        if (handle == nullptr) throw python_error();
        auto* raw = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
        Py_DECREF(handle);
        if (PyErr_Occurred()) throw python_error();
        const auto own = c10::cuda::getCurrentCUDAStream(device.index());
        if (own.stream() != raw && !PyLong_Check(stream)) {
            // torch's own Stream object: rebuilt from its parts, so that the allocator knows it
            int64_t part[3];
            const char* names[3] = {"stream_id", "device_index", "device_type"};
            for (int x = 0; x < 3; ++x) {
                PyObject* v = PyObject_GetAttrString(stream, names[x]);
                if (v == nullptr) throw python_error();
                part[x] = PyLong_AsLongLong(v);
                Py_DECREF(v);
                if (PyErr_Occurred()) throw python_error();
            }
            if (part[1] != device.index()) refuse("stream is on another device than the operands");
            stream_ = c10::cuda::CUDAStream(c10::Stream::unpack3(
                part[0], static_cast<c10::DeviceIndex>(part[1]), static_cast<c10::DeviceType>(part[2])));
        } else {
            stream_ = own.stream() == raw ? own
                                          : c10::cuda::getStreamFromExternal(raw, device.index());
        }
        on_.reset_stream(*stream_);
    }
    cudaStream_t get() const { return stream_->stream(); }

private:
    c10::cuda::OptionalCUDAGuard guard_;
    c10::cuda::OptionalCUDAStreamGuard on_;
    std::optional<c10::cuda::CUDAStream> stream_;
};

Tensor empty(Sizes sizes, ScalarType dtype, const at::Device& device)
{
    return Tensor(at::detail::empty_cuda(at::IntArrayRef(sizes), dtype, device, std::nullopt));
}

template <typename T = void>
T* pointer(const Tensor& t)
{
    return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
const T* source(const Tensor& t)
{
    return static_cast<const T*>(t.const_data_ptr());
}

// GemmError(status, message), as the package raises it.
void ok(int rc)
{
    if (rc == DECODE_OK) return;
    PyObject* package = PyImport_ImportModule("blackwell_tensor_core_fp16_gb300");
    PyObject* type = package ? PyObject_GetAttrString(package, "GemmError") : nullptr;
    PyObject* error = type ? PyObject_CallFunction(type, "is", rc, decode_last_error()) : nullptr;
    if (error != nullptr) PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(type);
    Py_XDECREF(package);
    throw python_error();
}

double number(PyObject* x)
{
    const double v = PyFloat_AsDouble(x);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int64_t integer(PyObject* x)
{
    const int64_t v = PyLong_AsLongLong(x);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* x)
{
    const int v = PyObject_IsTrue(x);
    if (v < 0) throw python_error();
    return v != 0;
}

// gated_delta_step(q, k, v, alpha, beta, state, scale, slots, out, stream)
PyObject* gated_delta_step(PyObject* const* args)
{
    const Tensor &q = tensor(args[0], "q"), &k = tensor(args[1], "k"), &v = tensor(args[2], "v"),
                 &alpha = tensor(args[3], "alpha"), &beta = tensor(args[4], "beta"),
                 &state = tensor(args[5], "state");
    decode_gdn_step_args a{};
    a.dtype = half_dtype(q);
    if (q.dim() != 4 || k.dim() != 4 || v.dim() != 4 || state.dim() != 4)
        refuse("q, k and v must be [n, tokens, heads, head_dim], state [slots, h_v, d, d]");
    const auto dev = q.device();
    const ScalarType half = q.scalar_type();
    const int64_t d = q.size(3);
    a.n = q.size(0), a.tokens = q.size(1), a.h_q = q.size(2), a.head_dim = d;
    a.h_k = k.size(2), a.h_v = v.size(2), a.n_slots = state.size(0);
    check(k, "k", half, dev, {a.n, a.tokens, a.h_k, d});
    check(v, "v", half, dev, {a.n, a.tokens, a.h_v, d});
    check(alpha, "alpha", ScalarType::Float, dev, {a.n, a.tokens, a.h_v});
    check(beta, "beta", ScalarType::Float, dev, {a.n, a.tokens, a.h_v});
    check(state, "state", ScalarType::Float, dev, {a.n_slots, a.h_v, d, d});
    strides(q, "q", a.q_stride);
    strides(k, "k", a.k_stride);
    strides(v, "v", a.v_stride);
    strides(alpha, "alpha", a.alpha_stride);
    strides(beta, "beta", a.beta_stride);
    if (state.stride(3) != 1 || state.stride(2) != d || (a.h_v > 1 && state.stride(1) != d * d))
        refuse("state must be contiguous within a slot");
    a.state_stride = state.stride(0);
    if (args[7] != Py_None) {
        const Tensor& slots = tensor(args[7], "slots");
        check(slots, "slots", ScalarType::Int, dev, {a.n});
        contiguous(slots, "slots");
        a.slots = source<int32_t>(slots);
    }
    a.scale = static_cast<float>(number(args[6]));
    const int64_t h_o = std::max(a.h_q, a.h_v);
    if (args[8] != Py_None) {
        check(tensor(args[8], "out"), "out", half, dev, {a.n, a.tokens, h_o, d});
        contiguous(tensor(args[8], "out"), "out");
    }
    const Where on(args[9], dev);
    const Tensor out = args[8] != Py_None ? THPVariable_Unpack(args[8])
                                          : empty({a.n, a.tokens, h_o, d}, half, dev);
    a.q = source(q), a.k = source(k), a.v = source(v);
    a.alpha = source<float>(alpha), a.beta = source<float>(beta);
    a.state = pointer<float>(state);
    a.o = pointer(out);
    ok(decode_gdn_step(&a, on.get()));
    return THPVariable_Wrap(out);
}

// qk_norm_rope(q, k, q_weight, k_weight, norm, eps, positions, rotary, sections, interleaved, v,
//              k_cache, v_cache, slots, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject* const* args)
{
    const Tensor &q = tensor(args[0], "q"), &k = tensor(args[1], "k");
    decode_qk_norm_rope_args a{};
    a.dtype = half_dtype(q);
    if (q.dim() != 3 || k.dim() != 3) refuse("q and k must be [tokens, heads, head_dim]");
    const auto dev = q.device();
    const ScalarType half = q.scalar_type();
    const int64_t d = q.size(2);
    a.tokens = q.size(0), a.h_q = q.size(1), a.head_dim = d, a.h_k = k.size(1);
    check(k, "k", half, dev, {a.tokens, a.h_k, d});
    strides(q, "q", a.q_stride);
    strides(k, "k", a.k_stride);
    for (const int x : {2, 3}) {
        if (args[x] == Py_None) continue;
        const char* name = x == 2 ? "q_weight" : "k_weight";
        const Tensor& w = tensor(args[x], name);
        check(w, name, half, dev, {d});
        contiguous(w, name);
        (x == 2 ? a.q_weight : a.k_weight) = source(w);
    }
    a.norm = static_cast<int32_t>(integer(args[4]));
    a.eps = static_cast<float>(number(args[5]));
    if (args[7] != Py_None) {
        const Tensor& rotary = tensor(args[7], "rotary");
        if (rotary.dim() != 2 || !rotary.is_contiguous())
            refuse("rotary must be a contiguous [rows, rot] table");
        a.table_rows = rotary.size(0), a.rot = rotary.size(1);
        check(rotary, "rotary", ScalarType::Float, dev, {a.table_rows, a.rot});
        if (args[6] == Py_None) refuse("a rotation needs positions [tokens] or [axes, tokens]");
        const Tensor& positions = tensor(args[6], "positions");
        if (positions.dim() != 1 && positions.dim() != 2)
            refuse("a rotation needs positions [tokens] or [axes, tokens]");
        a.axes = positions.dim() == 1 ? 1 : positions.size(0);
        if (positions.dim() == 1) {
            check(positions, "positions", ScalarType::Int, dev, {a.tokens});
            if (a.tokens > 1 && positions.stride(0) != 1)
                refuse("positions's last dimension must be contiguous");
            if (args[8] != Py_None) refuse("sections need positions [axes, tokens]");
        } else {
            check(positions, "positions", ScalarType::Int, dev, {a.axes, a.tokens});
            int64_t stride[1];
            strides(positions, "positions", stride);
            a.position_stride = stride[0];
            PyObject* list = args[8] == Py_None ? nullptr : PySequence_Fast(args[8], "sections");
            if (list == nullptr && args[8] != Py_None) throw python_error();
            const int64_t count = list == nullptr ? -1 : PySequence_Fast_GET_SIZE(list);
            int64_t sum = 0;
            const bool fits = count == a.axes && count >= 1 && count <= DECODE_MAX_AXES;
            bool small = true;                     // the struct holds 32 bits of each
            for (int64_t x = 0; fits && x < count; ++x) {
                const int64_t pairs = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(list, x));
                a.sections[x] = static_cast<int32_t>(pairs);
                small = small && a.sections[x] == pairs;
                sum += a.sections[x];
            }
            Py_XDECREF(list);
            if (PyErr_Occurred()) throw python_error();
            if (!fits) refuse("positions of 1 to 4 axes need as many sections");
            if (!small) refuse("a section of more pairs than any head holds");
            if (sum != a.rot / 2)
                refuse("sections of " + std::to_string(sum) + " pairs do not hold rot / 2 = " +
                       std::to_string(a.rot / 2));
        }
        a.positions = source<int32_t>(positions);
        a.table = source<float>(rotary);
    } else if (args[6] != Py_None || args[8] != Py_None) {
        refuse("positions and sections need a rotary table");
    }
    a.interleaved = truth(args[9]);
    const bool cache = args[11] != Py_None;
    if (cache) {
        if (args[10] == Py_None || args[12] == Py_None || args[13] == Py_None || args[15] != Py_None)
            refuse("k_cache comes with v, v_cache and slots, and without k_out");
        const Tensor &v = tensor(args[10], "v"), &kc = tensor(args[11], "k_cache"),
                     &vc = tensor(args[12], "v_cache"), &slots = tensor(args[13], "slots");
        if (kc.dim() != 4) refuse("k_cache must be [pages, page_size, h_k, d]");
        a.pages = kc.size(0), a.page_size = kc.size(1);
        check(v, "v", half, dev, {a.tokens, a.h_k, d});
        check(kc, "k_cache", half, dev, {a.pages, a.page_size, a.h_k, d});
        check(vc, "v_cache", half, dev, {a.pages, a.page_size, a.h_k, d});
        check(slots, "slots", ScalarType::Int, dev, {a.tokens});
        contiguous(slots, "slots");
        strides(v, "v", a.v_stride);
        strides(kc, "k_cache", a.k_cache_stride);
        strides(vc, "v_cache", a.v_cache_stride);
        separate(kc, "k_cache");
        separate(vc, "v_cache");
        a.v = source(v), a.k_cache = pointer(kc), a.v_cache = pointer(vc);
        a.slots = source<int32_t>(slots);
    } else if (args[10] != Py_None || args[12] != Py_None || args[13] != Py_None) {
        refuse("v, v_cache and slots come with k_cache");
    }
    for (const int x : {14, 15}) {
        if (args[x] == Py_None) continue;
        const char* name = x == 14 ? "q_out" : "k_out";
        const Tensor& t = tensor(args[x], name);
        check(t, name, half, dev, {a.tokens, x == 14 ? a.h_q : a.h_k, d});
        strides(t, name, x == 14 ? a.q_out_stride : a.k_out_stride);
        separate(t, name);
    }
    const Where on(args[16], dev);
    Tensor q_out, k_out;
    if (args[14] != Py_None) {
        q_out = THPVariable_Unpack(args[14]);
    } else {
        q_out = empty({a.tokens, a.h_q, d}, half, dev);
        a.q_out_stride[0] = a.h_q * d, a.q_out_stride[1] = d;
    }
    if (args[15] != Py_None) {
        k_out = THPVariable_Unpack(args[15]);
    } else if (!cache) {
        k_out = empty({a.tokens, a.h_k, d}, half, dev);
        a.k_out_stride[0] = a.h_k * d, a.k_out_stride[1] = d;
    }
    a.q = source(q), a.k = source(k);
    a.q_out = pointer(q_out);
    if (!cache) a.k_out = pointer(k_out);
    ok(decode_qk_norm_rope(&a, on.get()));
    return Py_BuildValue("NN", THPVariable_Wrap(q_out),
                         cache ? Py_NewRef(Py_None) : THPVariable_Wrap(k_out));
}

// paged_attention(q, k_cache, v_cache, page_table, lens, scale, window, return_lse, out, workspace,
//                 stream)
PyObject* paged_attention(PyObject* const* args)
{
    const Tensor &q = tensor(args[0], "q"), &kc = tensor(args[1], "k_cache"),
                 &vc = tensor(args[2], "v_cache"), &table = tensor(args[3], "page_table"),
                 &lens = tensor(args[4], "lens");
    decode_paged_attention_args a{};
    a.dtype = half_dtype(q);
    if (q.dim() != 3 || kc.dim() != 4 || table.dim() != 2)
        refuse("q must be [n, h_q, d], the caches [pages, page_size, h_kv, d] and page_table "
               "[n, width]");
    const auto dev = q.device();
    const ScalarType half = q.scalar_type();
    const int64_t d = q.size(2);
    a.n = q.size(0), a.h_q = q.size(1), a.head_dim = d;
    a.pages = kc.size(0), a.page_size = kc.size(1), a.h_kv = kc.size(2);
    a.table_width = table.size(1);
    check(kc, "k_cache", half, dev, {a.pages, a.page_size, a.h_kv, d});
    check(vc, "v_cache", half, dev, {a.pages, a.page_size, a.h_kv, d});
    check(table, "page_table", ScalarType::Int, dev, {a.n, a.table_width});
    check(lens, "lens", ScalarType::Int, dev, {a.n});
    contiguous(lens, "lens");
    strides(q, "q", a.q_stride);
    strides(kc, "k_cache", a.k_stride);
    strides(vc, "v_cache", a.v_stride);
    int64_t table_stride[1];
    strides(table, "page_table", table_stride);
    a.table_stride = table_stride[0];
    a.scale = args[5] == Py_None ? 1.0f / std::sqrt(static_cast<float>(d))
                                 : static_cast<float>(number(args[5]));
    if (args[6] != Py_None) {
        a.window = integer(args[6]);
        if (a.window < 1) refuse("window must be at least 1");
    }
    if (args[8] != Py_None) {
        check(tensor(args[8], "out"), "out", half, dev, {a.n, a.h_q, d});
        contiguous(tensor(args[8], "out"), "out");
    }
    if (args[9] != Py_None) {
        const Tensor& w = tensor(args[9], "workspace");
        if (w.device() != dev || !w.is_contiguous())
            refuse("workspace must be a contiguous tensor on " + dev.str());
    }
    const Where on(args[10], dev);
    const Tensor out = args[8] != Py_None ? THPVariable_Unpack(args[8])
                                          : empty({a.n, a.h_q, d}, half, dev);
    Tensor lse, workspace;
    if (truth(args[7])) {
        lse = empty({a.n, a.h_q}, ScalarType::Float, dev);
        a.lse = pointer<float>(lse);
    }
    if (args[9] != Py_None) {
        workspace = THPVariable_Unpack(args[9]);
    } else {
        size_t bytes = 0;
        ok(decode_paged_attention_workspace_bytes(a.h_q, a.h_kv, d, &bytes));
        workspace = empty({static_cast<int64_t>(bytes)}, ScalarType::Byte, dev);
    }
    a.q = source(q), a.k_cache = source(kc), a.v_cache = source(vc);
    a.page_table = source<int32_t>(table), a.lens = source<int32_t>(lens);
    a.o = pointer(out);
    a.workspace = pointer(workspace);
    a.workspace_bytes = static_cast<int64_t>(workspace.nbytes());
    ok(decode_paged_attention(&a, on.get()));
    if (!lse.defined()) return THPVariable_Wrap(out);
    return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// The Python entry: a fixed number of positional arguments (decode.py has the signatures), and every
// C++ exception turned into Python's.
template <PyObject* (*kFunction)(PyObject* const*), Py_ssize_t kArguments>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    if (count != kArguments) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are wanted", count, kArguments);
        return nullptr;
    }
    try {
        return kFunction(args);
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.why.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"gated_delta_step", reinterpret_cast<PyCFunction>(entry<gated_delta_step, 10>), METH_FASTCALL,
     nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(entry<qk_norm_rope, 17>), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(entry<paged_attention, 11>), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decode", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode() { return PyModule_Create(&module); }
