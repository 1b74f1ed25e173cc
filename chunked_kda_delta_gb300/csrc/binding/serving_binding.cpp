// serving_binding.cpp -- argument marshalling of the serving operators (page operations, 8-bit
// key/value cache, penalties on logits, beam selection) as a CPython extension on torch tensors.
//
// Every function checks its tensors (type, layout, shape, device), allocates what it returns, and
// makes one call of the C ABI in include/kda.h on the given or the current stream; all of the
// computation is in that call's kernels.  A decoding step makes these calls many times
// for a few microseconds of GPU work each: with the same checks in Python and ctypes calls in a
// row took 13 to 34 us each, most of it in the interpreter; here 4 to 9, or what the GPU takes.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <initializer_list>
#include <string>
#include <vector>

#include "../../../include/kda.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct Refused {
    std::string why;
};
[[noreturn]] void refuse(std::string why) { throw Refused{std::move(why)}; }

std::string text(IntArrayRef sizes) {
    std::string s = "(";
    for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
    return s + ")";
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

// A contiguous tensor of one of these types and exactly this shape on `device`.
const Tensor& vector(PyObject* o, const char* name, std::initializer_list<ScalarType> types, IntArrayRef shape,
                     const at::Device& device) {
    const Tensor& t = tensor(o, name);
    if (t.sizes() != shape) refuse(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    bool ok = t.device() == device && t.is_contiguous();
    bool type = false;
    for (ScalarType s : types) type |= t.scalar_type() == s;
    if (!ok || !type)
        refuse(std::string(name) + " must be a contiguous " + c10::toString(*types.begin()) + " tensor on " + device.str());
    return t;
}

void on_cuda(const Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be on cuda");
}

int64_t number(PyObject* o) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    return x;
}
int32_t number32(PyObject* o, const char* name) {
    const int64_t x = number(o);
    if (x != (int32_t)x) refuse(std::string(name) + " is out of range");
    return (int32_t)x;
}

// A call's scratch is torch's memory: what is captured into a graph belongs to that graph, and calls in
// a row reuse a block of their stream without a request to CUDA.  (The library's own pool costs a call
// 2 us on the host, and 0.3 to 0.8 us in a graph.)
void* allocate(void*, size_t bytes, void* stream) noexcept {
    try {
        return c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, static_cast<cudaStream_t>(stream));
    } catch (...) {
        return nullptr;
    }
}
void release(void*, void* scratch, size_t, void*) noexcept {
    try {
        c10::cuda::CUDACachingAllocator::raw_delete(scratch);
    } catch (...) {
    }
}
// For this thread and one call.  Torch keeps its blocks by the stream's handle, of which
// cudaStreamPerThread is one for the streams of all threads: there the library's own pool serves.
struct TorchScratch {
    kda_scratch_allocator before;
    bool set;
    explicit TorchScratch(cudaStream_t stream) : set(stream != cudaStreamPerThread) {
        const kda_scratch_allocator torch{allocate, release, nullptr};
        if (set) kda_set_scratch_allocator(&torch, &before);
    }
    TorchScratch(const TorchScratch&) = delete;
    ~TorchScratch() {
        if (set) kda_set_scratch_allocator(&before, nullptr);
    }
};

// The device made current, and the stream of the call: a raw handle, or the device's current one.
// Results come from that stream's memory: a block of another stream's may still be written by
// work that this stream does not wait for.  They are recorded on the current stream too, where the
// caller most likely drops them.
struct Place {
    c10::cuda::CUDAGuard guard;
    at::Device device;
    c10::cuda::CUDAStream current;
    c10::cuda::CUDAStream own;
    void* stream;

    Place(const at::Device& d, PyObject* handle)
        : guard(d.index()), device(d), current(c10::cuda::getCurrentCUDAStream(d.index())), own(current) {
        if (given(handle)) {
            const auto h = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
            if (PyErr_Occurred()) throw python_error();
            if (h == nullptr || h == cudaStreamLegacy) own = c10::cuda::getDefaultCUDAStream(d.index());
            else if (h != current.stream()) own = c10::cuda::getStreamFromExternal(h, d.index());
        }
        stream = own.stream();
    }
    Tensor empty(IntArrayRef shape, ScalarType type) const {
        // (The allocation itself: 0.3 to 0.6 us less a tensor than a call of at::empty.)
        const auto allocate = [&] {
            return Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
        };
        if (own.stream() == current.stream()) return allocate();
        const c10::cuda::CUDAStreamGuard set(own);
        Tensor t = allocate();
        if (t.numel()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
        return t;
    }
    // The given int32 tensor, or a new one, in the shape of `like`.
    Tensor result(PyObject* o, const char* name, const Tensor& like) const {
        return given(o) ? vector(o, name, {ScalarType::Int}, like.sizes(), device) : empty(like.sizes(), ScalarType::Int);
    }
};

template <typename T = void>
T* ptr(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

// KdaError(status, message) of the Python package.
[[noreturn]] void raise_status(kda_status status) {
    PyObject* mod = PyImport_ImportModule("chunked_kda_delta_gb300.kda");
    PyObject* type = mod ? PyObject_GetAttrString(mod, "KdaError") : nullptr;
    PyObject* err = type ? PyObject_CallFunction(type, "is", (int)status, kda_last_error_message()) : nullptr;
    if (err) PyErr_SetObject(type, err);
    Py_XDECREF(err);
    Py_XDECREF(type);
    Py_XDECREF(mod);
    throw python_error();
}
void check(kda_status status) {
    if (status != KDA_OK) raise_status(status);
}

PyObject* pack(std::initializer_list<Tensor> ts) {
    PyObject* tuple = PyTuple_New((Py_ssize_t)ts.size());
    if (!tuple) throw python_error();
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) {
        PyObject* o = THPVariable_Wrap(t);
        if (!o) {
            Py_DECREF(tuple);
            throw python_error();
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

// ---- pages -----------------------------------------------------------------------------
struct Pages {
    const Tensor& tables;
    const Tensor& refs;
    kda_page_shape shape;
    at::Device device;
};
Pages pages_of(PyObject* tables_o, PyObject* refs_o) {
    const Tensor& tables = tensor(tables_o, "tables");
    const Tensor& refs = tensor(refs_o, "refs");
    on_cuda(tables, "tables");
    if (tables.dim() != 2 || tables.size(1) < 1) refuse("tables must be [rows, width]");
    if (refs.dim() != 1) refuse("refs must be [pages]");
    vector(tables_o, "tables", {ScalarType::Int}, tables.sizes(), tables.device());
    vector(refs_o, "refs", {ScalarType::Int}, refs.sizes(), tables.device());
    if (tables.size(0) > INT32_MAX || tables.size(1) > INT32_MAX || refs.size(0) > INT32_MAX) refuse("tables or refs are too large");
    return Pages{tables, refs, kda_page_shape{(int32_t)tables.size(0), (int32_t)tables.size(1), (int32_t)refs.size(0)}, tables.device()};
}
struct Pools {
    std::array<kda_pool, KDA_MAX_POOLS> pool;
    int32_t n = 0;
};
// [pages, ...] tensors, or [layers, pages, ...] ones, with contiguous pages.  `pages` < 0 is taken
// from the first.
void read_pools(PyObject* seq, int64_t& pages, const at::Device& device, bool layers_first, Pools& out) {
    if (THPVariable_Check(seq)) refuse("pools must be a sequence of tensors");
    PyObject* fast = PySequence_Fast(seq, "pools must be a sequence of tensors");
    if (!fast) throw python_error();
    struct Release {
        PyObject* o;
        ~Release() { Py_DECREF(o); }
    } release{fast};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
    if (n > KDA_MAX_POOLS) refuse("at most " + std::to_string(KDA_MAX_POOLS) + " pools");
    const int64_t lead = layers_first ? 1 : 0;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const Tensor& t = tensor(PySequence_Fast_GET_ITEM(fast, i), "a pool");
        if (pages < 0 && t.dim() > lead) pages = t.size(lead);
        if (t.device() != device || t.dim() <= lead || t.size(lead) != pages)
            refuse("a pool must be a tensor on " + device.str() + " with " + std::to_string(pages) + " pages in dim " + std::to_string(lead));
        int64_t inner = 1;
        for (int64_t d = t.dim() - 1; d > lead; --d) {
            if (t.size(d) != 1 && t.stride(d) != inner) refuse("the pages of a pool must be contiguous");
            inner *= t.size(d);
        }
        const int64_t elem = (int64_t)t.element_size(), step = t.stride(lead) * elem;
        kda_pool& p = out.pool[i];
        p.base = t.data_ptr();
        p.page_bytes = inner * elem;
        p.page_stride = pages <= 1 && step < p.page_bytes ? p.page_bytes : step;
        p.layer_stride = layers_first ? t.stride(0) * elem : 0;
        const int64_t layers = layers_first ? t.size(0) : 1;
        if (layers > INT32_MAX) refuse("a pool has too many layers");
        p.layers = (int32_t)layers;
    }
    out.n = (int32_t)n;
}

// (tables, refs, want, new_tables, new_refs, stream)
PyObject* pages_alloc(PyObject* const* a) {
    const Pages g = pages_of(a[0], a[1]);
    const Tensor& want = vector(a[2], "want", {ScalarType::Int}, {g.shape.rows}, g.device);
    Place on(g.device, a[5]);
    Tensor nt = on.result(a[3], "new_tables", g.tables), nr = on.result(a[4], "new_refs", g.refs);
    const TorchScratch scratch(on.own);
    check(kda_pages_alloc(&g.shape, ptr<int32_t>(g.tables), ptr<int32_t>(g.refs), ptr<int32_t>(want), ptr<int32_t>(nt), ptr<int32_t>(nr), on.stream));
    return pack({nt, nr});
}

// (tables, refs, drop, new_tables, new_refs, stream)
PyObject* pages_free(PyObject* const* a) {
    const Pages g = pages_of(a[0], a[1]);
    const Tensor& drop = vector(a[2], "drop", {ScalarType::Bool, ScalarType::Byte}, {g.shape.rows}, g.device);
    Place on(g.device, a[5]);
    Tensor nt = on.result(a[3], "new_tables", g.tables), nr = on.result(a[4], "new_refs", g.refs);
    const TorchScratch scratch(on.own);
    check(kda_pages_free(&g.shape, ptr<int32_t>(g.tables), ptr<int32_t>(g.refs), ptr<uint8_t>(drop), ptr<int32_t>(nt), ptr<int32_t>(nr), on.stream));
    return pack({nt, nr});
}

// (tables, refs, parents, lens, page_tokens, pools, layers_first, new_tables, new_refs, stream)
PyObject* pages_fork(PyObject* const* a) {
    const Pages g = pages_of(a[0], a[1]);
    const Tensor& parents = vector(a[2], "parents", {ScalarType::Int}, {g.shape.rows}, g.device);
    const int32_t page_tokens = number32(a[4], "page_tokens");
    if (page_tokens > 0 && !given(a[3])) refuse("lens is needed with page_tokens");
    const int32_t* lens = given(a[3]) ? ptr<int32_t>(vector(a[3], "lens", {ScalarType::Int}, {g.shape.rows}, g.device)) : nullptr;
    Pools pools;
    int64_t pages = g.shape.pages;
    read_pools(a[5], pages, g.device, a[6] == Py_True, pools);
    Place on(g.device, a[9]);
    Tensor nt = on.result(a[7], "new_tables", g.tables), nr = on.result(a[8], "new_refs", g.refs);
    const TorchScratch scratch(on.own);
    check(kda_pages_fork(&g.shape, ptr<int32_t>(g.tables), ptr<int32_t>(g.refs), ptr<int32_t>(parents), lens, page_tokens, pools.pool.data(),
                         pools.n, ptr<int32_t>(nt), ptr<int32_t>(nr), on.stream));
    return pack({nt, nr});
}

// (tables, refs, pools, layers_first, new_tables, new_refs, stream)
PyObject* pages_compact(PyObject* const* a) {
    const Pages g = pages_of(a[0], a[1]);
    Pools pools;
    int64_t pages = g.shape.pages;
    read_pools(a[2], pages, g.device, a[3] == Py_True, pools);
    Place on(g.device, a[6]);
    Tensor nt = on.result(a[4], "new_tables", g.tables), nr = on.result(a[5], "new_refs", g.refs);
    Tensor map = on.empty(g.refs.sizes(), ScalarType::Int), live = on.empty({1}, ScalarType::Int);
    const TorchScratch scratch(on.own);
    check(kda_pages_compact(&g.shape, ptr<int32_t>(g.tables), ptr<int32_t>(g.refs), pools.pool.data(), pools.n, ptr<int32_t>(nt),
                            ptr<int32_t>(nr), ptr<int32_t>(map), ptr<int32_t>(live), on.stream));
    return pack({nt, nr, map, live});
}

// (src, dst, pools, layers_first, stream)
PyObject* pages_copy(PyObject* const* a) {
    const Tensor& src = tensor(a[0], "src");
    if (!src.is_cuda() || src.dim() != 1) refuse("src must be [count] on cuda");
    vector(a[0], "src", {ScalarType::Int}, src.sizes(), src.device());
    const Tensor& dst = vector(a[1], "dst", {ScalarType::Int}, src.sizes(), src.device());
    Pools pools;
    int64_t pages = -1;
    read_pools(a[2], pages, src.device(), a[3] == Py_True, pools);
    if (pools.n && pages <= INT32_MAX && src.size(0) <= INT32_MAX) {
        Place on(src.device(), a[4]);
        check(kda_pages_copy((int32_t)pages, (int32_t)src.size(0), ptr<int32_t>(src), ptr<int32_t>(dst), pools.pool.data(), pools.n, on.stream));
    } else if (pools.n) {
        refuse("too many pages or pairs");
    }
    Py_RETURN_NONE;
}

// ---- 8-bit key/value cache -------------------------------------------------------------
struct Cache {
    kda_kvcache c;
    at::Device device;
    const int32_t* lens;
    const int32_t* cu;
};
// k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens
Cache cache_of(PyObject* const* a) {
    const Tensor& kc = tensor(a[0], "k_codes");
    on_cuda(kc, "k_codes");
    if (kc.dim() != 4) refuse("k_codes must be [pages, heads, page_tokens, head_dim]");
    const at::Device device = kc.device();
    vector(a[0], "k_codes", {ScalarType::Float8_e4m3fn, ScalarType::Byte}, kc.sizes(), device);
    const Tensor& vc = vector(a[1], "v_codes", {ScalarType::Float8_e4m3fn, ScalarType::Byte}, kc.sizes(), device);
    const Tensor& ks = vector(a[2], "k_scale", {ScalarType::Float}, {kc.size(0), kc.size(1)}, device);
    const Tensor& vs = vector(a[3], "v_scale", {ScalarType::Float}, {kc.size(0), kc.size(1)}, device);
    const Tensor& tables = tensor(a[4], "tables");
    if (tables.dim() != 2 || tables.size(1) < 1) refuse("tables must be [rows, width]");
    vector(a[4], "tables", {ScalarType::Int}, tables.sizes(), device);
    for (int d = 0; d < 4; ++d)
        if (kc.size(d) > INT32_MAX) refuse("the cache is too large");
    if (tables.size(0) > INT32_MAX - 1 || tables.size(1) > INT32_MAX) refuse("tables are too large");
    const int64_t rows = tables.size(0);
    Cache x{kda_kvcache{}, device, nullptr, nullptr};
    x.c.k_codes = kc.data_ptr();
    x.c.v_codes = vc.data_ptr();
    x.c.k_scale = ptr<float>(ks);
    x.c.v_scale = ptr<float>(vs);
    x.c.pages = (int32_t)kc.size(0);
    x.c.num_kv_heads = (int32_t)kc.size(1);
    x.c.page_tokens = (int32_t)kc.size(2);
    x.c.head_dim = (int32_t)kc.size(3);
    x.c.tables = ptr<int32_t>(tables);
    x.c.rows = (int32_t)rows;
    x.c.width = (int32_t)tables.size(1);
    x.lens = ptr<int32_t>(vector(a[5], "lens", {ScalarType::Int}, {rows}, device));
    if (given(a[6])) x.cu = ptr<int32_t>(vector(a[6], "cu_tokens", {ScalarType::Int}, {rows + 1}, device));
    return x;
}

int32_t act_type(const Tensor& t, const char* name, const at::Device& device) {
    if (t.device() != device || (t.scalar_type() != ScalarType::BFloat16 && t.scalar_type() != ScalarType::Half))
        refuse(std::string(name) + " must be bf16 or fp16 on " + device.str());
    return t.scalar_type() == ScalarType::Half ? KDA_ACT_F16 : KDA_ACT_BF16;
}
// [tokens, heads, dim] with contiguous heads; the token stride.
int64_t act_stride(const Tensor& t, const char* name, int64_t heads, int64_t dim) {
    if (t.dim() != 3 || (heads >= 0 && t.size(1) != heads) || t.size(2) != dim)
        refuse(std::string(name) + " must be [tokens, " + (heads >= 0 ? std::to_string(heads) : "heads") + ", " + std::to_string(dim) + "]");
    if (t.numel() && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != dim)))
        refuse(std::string("the heads of ") + name + " must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * dim;
}

// (k, v, k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens, stream)
PyObject* kvcache_append(PyObject* const* a) {
    const Cache x = cache_of(a + 2);
    const Tensor& k = tensor(a[0], "k");
    const Tensor& v = tensor(a[1], "v");
    if (k.scalar_type() != v.scalar_type() || k.sizes() != v.sizes()) refuse("k and v must have the same type and shape");
    const int32_t type = act_type(k, "k", x.device);
    act_type(v, "v", x.device);
    const int64_t ks = act_stride(k, "k", x.c.num_kv_heads, x.c.head_dim), vs = act_stride(v, "v", x.c.num_kv_heads, x.c.head_dim);
    Place on(x.device, a[9]);
    check(kda_kvcache_append(&x.c, k.data_ptr(), v.data_ptr(), type, ks, vs, k.size(0), x.lens, x.cu, on.stream));
    Py_RETURN_NONE;
}

// (q, k, v, rotary, k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens, positions, interleaved, out, stream)
PyObject* kvcache_append_rotary(PyObject* const* a) {
    const Cache x = cache_of(a + 4);
    const Tensor& q = tensor(a[0], "q");
    const Tensor& k = tensor(a[1], "k");
    const Tensor& v = tensor(a[2], "v");
    if (k.scalar_type() != v.scalar_type() || k.sizes() != v.sizes()) refuse("k and v must have the same type and shape");
    const int32_t type = act_type(q, "q", x.device);
    if (k.scalar_type() != q.scalar_type()) refuse("q and k must have the same type");
    act_type(k, "k", x.device);
    act_type(v, "v", x.device);
    const int64_t qs = act_stride(q, "q", -1, x.c.head_dim), ks = act_stride(k, "k", x.c.num_kv_heads, x.c.head_dim),
                  vs = act_stride(v, "v", x.c.num_kv_heads, x.c.head_dim);
    if (q.size(1) > INT32_MAX) refuse("q has too many heads");
    if (q.size(0) != k.size(0)) refuse("q and k must have the same tokens");
    const Tensor& table = tensor(a[3], "rotary");
    if (table.dim() != 2 || table.size(1) > INT32_MAX) refuse("rotary must be [positions, rotary_dim]");
    vector(a[3], "rotary", {ScalarType::Float}, table.sizes(), x.device);
    const int32_t* positions = given(a[11]) ? ptr<int32_t>(vector(a[11], "positions", {ScalarType::Int}, {q.size(0)}, x.device)) : nullptr;
    const int interleaved = PyObject_IsTrue(a[12]);
    if (interleaved < 0) throw python_error();
    Place on(x.device, a[14]);
    Tensor out;
    if (given(a[13])) {
        out = tensor(a[13], "out");
        if (out.scalar_type() != q.scalar_type() || out.sizes() != q.sizes()) refuse("out must have q's type and shape");
        act_type(out, "out", x.device);
    } else {
        out = on.empty(q.sizes(), q.scalar_type());
    }
    const int64_t os = act_stride(out, "out", q.size(1), x.c.head_dim);
    check(kda_kvcache_append_rotary(&x.c, q.data_ptr(), k.data_ptr(), v.data_ptr(), (int32_t)q.size(1), type, qs, ks, vs, q.size(0), x.lens, x.cu,
                                    ptr<float>(table), table.size(0), (int32_t)table.size(1), interleaved, positions, out.data_ptr(), os, on.stream));
    return THPVariable_Wrap(out);
}

// (q, k_codes, v_codes, k_scale, v_scale, tables, lens, cu_tokens, scale, out, stream), with shared prefixes cu_rows as the last
template <bool kShared>
PyObject* kvcache_attention(PyObject* const* a) {
    const Cache x = cache_of(a + 1);
    const Tensor& q = tensor(a[0], "q");
    const int32_t type = act_type(q, "q", x.device);
    const int64_t qs = act_stride(q, "q", -1, x.c.head_dim);
    if (q.size(1) > INT32_MAX) refuse("q has too many heads");
    double scale = 1.0 / std::sqrt((double)x.c.head_dim);
    if (given(a[8])) {
        scale = PyFloat_AsDouble(a[8]);
        if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    }
    const int32_t* cu_rows = nullptr;
    int64_t groups = 0;
    if (kShared) {
        const Tensor& t = tensor(a[11], "cu_rows");
        if (t.dim() != 1 || t.size(0) < 1 || t.size(0) > INT32_MAX) refuse("cu_rows must be [groups + 1]");
        cu_rows = ptr<int32_t>(vector(a[11], "cu_rows", {ScalarType::Int}, t.sizes(), x.device));
        groups = t.size(0) - 1;
    }
    Place on(x.device, a[10]);
    Tensor out;
    if (given(a[9])) {
        out = tensor(a[9], "out");
        if (out.scalar_type() != q.scalar_type() || out.sizes() != q.sizes()) refuse("out must have q's type and shape");
        act_type(out, "out", x.device);
    } else {
        out = on.empty(q.sizes(), q.scalar_type());
    }
    const int64_t os = act_stride(out, "out", q.size(1), x.c.head_dim);
    const TorchScratch scratch(on.own);
    if (kShared)
        check(kda_kvcache_attention_shared(&x.c, q.data_ptr(), (int32_t)q.size(1), type, qs, q.size(0), x.lens, x.cu, cu_rows, (int32_t)groups,
                                           (float)scale, out.data_ptr(), os, on.stream));
    else
        check(kda_kvcache_attention(&x.c, q.data_ptr(), (int32_t)q.size(1), type, qs, q.size(0), x.lens, x.cu, (float)scale, out.data_ptr(), os, on.stream));
    return THPVariable_Wrap(out);
}

// ---- logits ----------------------------------------------------------------------------
// Rows of logits [..., vocab] at one stride.
struct Rows {
    IntArrayRef lead;
    int64_t n, vocab, stride;
};
Rows rows_of(const Tensor& x, const char* name) {
    const int64_t dims = x.dim();
    Rows r{x.sizes().slice(0, dims - 1), 1, x.size(dims - 1), 0};
    for (int64_t d : r.lead) r.n *= d;
    r.stride = r.vocab;
    if (!r.n) return r;
    bool ok = r.vocab <= 1 || x.stride(dims - 1) == 1, first = true;
    int64_t next = 0;  // stride of the dimension before
    for (int64_t d = dims - 2; d >= 0; --d) {
        if (x.size(d) == 1) continue;
        if (first) next = r.stride = x.stride(d);
        ok &= x.stride(d) == next;
        next *= x.size(d);
        first = false;
    }
    if (!ok) refuse(std::string(name) + " must have contiguous rows at one stride");
    return r;
}
// A contiguous tensor [..., (width)] with logits' leading dimensions, which may be one; its width.
const Tensor* per_row(PyObject* o, const char* name, ScalarType type, const Rows& rows, bool wide, int64_t& width, const at::Device& device) {
    if (!given(o)) return nullptr;
    const Tensor& t = tensor(o, name);
    const int64_t lead = t.dim() - (wide ? 1 : 0);
    bool ok = t.device() == device && t.is_contiguous() && t.scalar_type() == type;
    ok = ok && (lead == 1 ? t.size(0) == rows.n : lead == (int64_t)rows.lead.size() && t.sizes().slice(0, lead) == rows.lead);
    if (!ok)
        refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor on " + device.str() + " with logits' " +
               std::to_string(rows.n) + " rows" + (wide ? " in its leading dimensions" : ""));
    if (wide) width = t.size(t.dim() - 1);
    return &t;
}

// (logits, history, lens, prompt_lens, repetition, presence, frequency, bias_tokens, bias, mask, out, stream)
PyObject* logits_penalize(PyObject* const* a) {
    const Tensor& x = tensor(a[0], "logits");
    const ScalarType type = x.scalar_type();
    if (!x.is_cuda() || x.dim() < 1 || (type != ScalarType::Float && type != ScalarType::BFloat16 && type != ScalarType::Half))
        refuse("logits must be fp32, bf16 or fp16 [..., vocab] on cuda");
    const at::Device device = x.device();
    const Rows rows = rows_of(x, "logits");
    if (rows.n > INT32_MAX || rows.vocab > INT32_MAX) refuse("logits are too large");
    int64_t width = 0, biases = 0, values = 0, words = 0, none = 0;
    const Tensor* history = per_row(a[1], "history", ScalarType::Int, rows, true, width, device);
    const Tensor* lens = per_row(a[2], "lens", ScalarType::Int, rows, false, none, device);
    const Tensor* prompt = per_row(a[3], "prompt_lens", ScalarType::Int, rows, false, none, device);
    const Tensor* repetition = per_row(a[4], "repetition", ScalarType::Float, rows, false, none, device);
    const Tensor* presence = per_row(a[5], "presence", ScalarType::Float, rows, false, none, device);
    const Tensor* frequency = per_row(a[6], "frequency", ScalarType::Float, rows, false, none, device);
    const Tensor* bias_tokens = per_row(a[7], "bias_tokens", ScalarType::Int, rows, true, biases, device);
    const Tensor* bias = per_row(a[8], "bias", ScalarType::Float, rows, true, values, device);
    const Tensor* mask = per_row(a[9], "mask", ScalarType::Int, rows, true, words, device);
    if (!history && (lens || prompt || repetition || presence || frequency)) refuse("lengths and penalties need a history");
    if (!bias_tokens != !bias || biases != values) refuse("bias_tokens and bias must have the same shape");
    if (width > INT32_MAX || biases > INT32_MAX) refuse("history or bias is too wide");
    if (mask && words < (rows.vocab + 31) / 32) refuse("mask must have " + std::to_string((rows.vocab + 31) / 32) + " words a row");
    Place on(device, a[11]);
    Tensor out;
    int64_t stride = rows.vocab;
    if (given(a[10])) {
        out = tensor(a[10], "out");
        if (out.scalar_type() != type || out.sizes() != x.sizes() || out.device() != device) refuse("out must have logits' type, shape and device");
        stride = rows_of(out, "out").stride;
    } else if (rows.n && rows.stride != rows.vocab) {
        // Padded rows give padded rows: each starts on 16 bytes.
        const int64_t each = 16 / (int64_t)x.element_size();
        stride = (rows.vocab + each - 1) / each * each;
        std::vector<int64_t> shape(rows.lead.begin(), rows.lead.end());
        shape.push_back(stride);
        out = on.empty(shape, type).narrow((int64_t)shape.size() - 1, 0, rows.vocab);
    } else {
        out = on.empty(x.sizes(), type);
    }
    auto ints = [](const Tensor* t) { return t ? ptr<int32_t>(*t) : nullptr; };
    auto floats = [](const Tensor* t) { return t ? ptr<float>(*t) : nullptr; };
    const kda_logits_rules rules{ints(history), ints(lens), ints(prompt), floats(repetition), floats(presence), floats(frequency), ints(bias_tokens),
                                 floats(bias), ints(mask), words, (int32_t)width, (int32_t)biases};
    check(kda_logits_penalize(&rules, rows.n, (int32_t)rows.vocab, x.data_ptr(),
                              type == ScalarType::Float ? KDA_LOGITS_F32 : type == ScalarType::BFloat16 ? KDA_LOGITS_BF16 : KDA_LOGITS_F16, rows.stride,
                              out.data_ptr(), stride, on.stream));
    return THPVariable_Wrap(out);
}

// ---- beam selection --------------------------------------------------------------------
// (logits, scores, num_out, done, eos, stream)
PyObject* beam_select(PyObject* const* a) {
    const Tensor& x = tensor(a[0], "logits");
    const ScalarType type = x.scalar_type();
    if (!x.is_cuda() || x.dim() != 3 || (type != ScalarType::Float && type != ScalarType::BFloat16 && type != ScalarType::Half))
        refuse("logits must be fp32, bf16 or fp16 [batch, beams, vocab] on cuda");
    const at::Device device = x.device();
    const int64_t batch = x.size(0), beams = x.size(1), vocab = x.size(2);
    const int64_t stride = beams > 1 ? x.stride(1) : batch > 1 ? x.stride(0) : vocab;
    if (batch > INT32_MAX || beams > INT32_MAX || vocab > INT32_MAX) refuse("logits are too large");
    if (batch && beams && ((vocab > 1 && x.stride(2) != 1) || (batch > 1 && x.stride(0) != beams * stride)))
        refuse("logits must have contiguous rows at one stride");
    const Tensor& scores = vector(a[1], "scores", {ScalarType::Float}, {batch, beams}, device);
    const bool has_done = given(a[3]);
    const Tensor& done = has_done ? vector(a[3], "done", {ScalarType::Bool, ScalarType::Byte}, {batch, beams}, device) : scores;
    const int64_t k = given(a[2]) ? number(a[2]) : beams;
    if (k < 1) refuse("num_out must be at least 1");
    if (k > INT32_MAX) refuse("num_out is out of range");
    const int32_t eos = number32(a[4], "eos");
    Place on(device, a[5]);
    // (k past the ABI's limit is refused by the call: allocate nothing for it)
    const int64_t places = k <= 64 ? k : 1;
    Tensor s = on.empty({batch, places}, ScalarType::Float), t = on.empty({batch, places}, ScalarType::Int);
    Tensor p = on.empty({batch, places}, ScalarType::Int), d;
    if (has_done) d = on.empty({batch, places}, done.scalar_type());
    const TorchScratch scratch(on.own);
    check(kda_beam_select((int32_t)batch, (int32_t)beams, (int32_t)vocab, (int32_t)k, x.data_ptr(),
                          type == ScalarType::Float ? KDA_LOGITS_F32 : type == ScalarType::BFloat16 ? KDA_LOGITS_BF16 : KDA_LOGITS_F16, stride,
                          ptr<float>(scores), has_done ? ptr<uint8_t>(done) : nullptr, eos, ptr<float>(s), ptr<int32_t>(t), ptr<int32_t>(p),
                          has_done ? ptr<uint8_t>(d) : nullptr, on.stream));
    return has_done ? pack({s, t, p, d}) : pack({s, t, p});
}

// Arguments counted, C++ exceptions turned into Python's.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.why.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<pages_alloc, 6>("pages_alloc"),
    method<pages_free, 6>("pages_free"),
    method<pages_fork, 10>("pages_fork"),
    method<pages_compact, 7>("pages_compact"),
    method<pages_copy, 5>("pages_copy"),
    method<kvcache_append, 10>("kvcache_append"),
    method<kvcache_append_rotary, 15>("kvcache_append_rotary"),
    method<kvcache_attention<false>, 11>("kvcache_attention"),
    method<kvcache_attention<true>, 12>("kvcache_attention_shared"),
    method<logits_penalize, 12>("logits_penalize"),
    method<beam_select, 6>("beam_select"),
    PyMethodDef{nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_serving() { return PyModule_Create(&module); }
