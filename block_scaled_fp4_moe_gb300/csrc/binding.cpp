// binding.cpp -- the host side of attn.py's calls: checks torch tensors and
// passes their addresses to the C ABI (moe_attn.h).  Marshalling only.
//
// A decode step makes five to ten of these calls a layer, of a few microseconds on
// the GPU each; the checks of a dozen tensors through Python attributes took as
// long as the kernels.  The library itself stays free of torch: this module
// is given the addresses of its functions.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "moe_attn.h"

namespace {

struct Library {
    decltype(&moe_kv_build_tables) build_tables;
    decltype(&moe_kv_append) append;
    decltype(&moe_kv_attention) attention;
    decltype(&moe_quantize_fp8_weight) quantize;
    decltype(&moe_linear_fp8) linear;
    decltype(&moe_rms_norm) norm;
    decltype(&moe_rotary) rotary;
    decltype(&moe_latent_append) latent_append;
    decltype(&moe_latent_attention) latent_attention;
} lib;

std::string show(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i)
        r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

[[noreturn]] void fail(const char *name, const std::string &what) {
    throw std::invalid_argument(std::string(name) + ": " + what);
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o))
        fail(name, "expected a tensor");
    return THPVariable_Unpack(o);
}

// The device of a call: that of its first tensor, on which all others have to be.  The call's kernels run there, whatever device is
// current, on its current stream unless one is given.
class Device {
public:
    void meet(const at::Tensor &t, const char *name) {
        const int i = t.get_device();
        if (index_ < 0) {
            index_ = i;
            first_ = name;
        } else if (i != index_) {
            fail(name, "expected a tensor on cuda:" + std::to_string(index_) + " as " + first_ + ", got cuda:" + std::to_string(i));
        }
    }
    c10::DeviceIndex index() const { return (c10::DeviceIndex)index_; }

private:
    int index_ = -1;
    const char *first_ = "";
};

// A CUDA tensor of this type, on the call's device.
const at::Tensor &cuda(Device &dev, PyObject *o, at::ScalarType type, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (!t.is_cuda())
        fail(name, "expected a CUDA tensor");
    if (t.scalar_type() != type)
        fail(name, std::string("expected ") + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    dev.meet(t, name);
    return t;
}

const at::Tensor &whole(Device &dev, PyObject *o, at::ScalarType type, const char *name) {
    const at::Tensor &t = cuda(dev, o, type, name);
    if (!t.is_contiguous())
        fail(name, "expected a contiguous tensor");
    return t;
}

void want(const at::Tensor &t, std::initializer_list<int64_t> shape, const char *name) {
    const at::IntArrayRef s(shape.begin(), shape.size());
    if (t.sizes() != s)
        fail(name, "expected shape " + show(s) + ", got " + show(t.sizes()));
}

// [tokens, heads, dim] with contiguous dims.
const at::Tensor &heads(Device &dev, PyObject *o, const char *name) {
    const at::Tensor &t = cuda(dev, o, at::kBFloat16, name);
    if (t.dim() != 3 || (t.stride(2) != 1 && t.size(2) > 1))
        fail(name, "expected [tokens, heads, dim] with contiguous dims");
    return t;
}

// The stride of an axis; that of an axis of one element is never used, whatever it says.
int64_t step(const at::Tensor &t, int axis) { return t.size(axis) > 1 ? t.stride(axis) : 0; }

template <typename P>
P *at_of(const at::Tensor &t) {
    return reinterpret_cast<P *>(t.data_ptr());
}

int narrow(int64_t v, const char *name) {
    if (v < -0x7FFFFFFFll || v > 0x7FFFFFFFll)
        fail(name, "too large");
    return (int)v;
}

int integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw std::runtime_error("");
    return narrow(v, name);
}

double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw std::runtime_error("");
    return v;
}

int truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw std::runtime_error("");
    return v;
}

cudaStream_t stream_of(const Device &dev, PyObject *o) {
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred())
        throw std::runtime_error("");
    return static_cast<cudaStream_t>(p);
}

// k, v, k_scale, v_scale at o[0..3].
moe_kv_cache_t cache_of(Device &dev, PyObject *const *o) {
    const at::Tensor &k = whole(dev, o[0], at::kByte, "k"), &v = whole(dev, o[1], at::kByte, "v");
    const at::Tensor &ks = whole(dev, o[2], at::kByte, "k_scale"), &vs = whole(dev, o[3], at::kByte, "v_scale");
    if (k.dim() != 6)
        fail("k", "expected six axes, got " + show(k.sizes()));
    const int64_t nb = k.size(0), h = k.size(1), subs = k.size(2), chunks = k.size(3);
    want(k, {nb, h, subs, chunks, 16, 16}, "k");
    want(v, {nb, h, subs, 16 * chunks, 16}, "v");
    want(ks, {nb, h}, "k_scale");
    want(vs, {nb, h}, "v_scale");
    return moe_kv_cache_t{at_of<uint8_t>(k), at_of<uint8_t>(v), at_of<uint8_t>(ks), at_of<uint8_t>(vs), narrow(nb, "k"),
                          narrow(h, "k"), narrow(16 * chunks, "k"), narrow(16 * subs, "k")};
}

void weight_of(const at::Tensor &codes, const at::Tensor &scale) {
    if (codes.dim() != 2)
        fail("codes", "expected a matrix, got " + show(codes.sizes()));
    want(scale, {(codes.size(0) + 127) / 128, (codes.size(1) + 127) / 128}, "scale");
}

// A bf16 vector of n values, or nothing.
const uint16_t *vector_of(Device &dev, PyObject *o, int64_t n, const char *name) {
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = whole(dev, o, at::kBFloat16, name);
    want(t, {n}, name);
    return at_of<uint16_t>(t);
}

// A bf16 matrix with contiguous rows.
const at::Tensor &matrix(Device &dev, PyObject *o, const char *name) {
    const at::Tensor &t = cuda(dev, o, at::kBFloat16, name);
    if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
        fail(name, "expected a matrix with contiguous rows");
    return t;
}

// The dims of one latent vector's cache at o.
moe_latent_cache_t latent_cache_of(Device &dev, PyObject *o) {
    const at::Tensor &t = whole(dev, o, at::kBFloat16, "cache");
    if (t.dim() != 3 || t.size(2) <= 64)
        fail("cache", "expected [blocks, block_size, latent_dim + 64], got " + show(t.sizes()));
    return moe_latent_cache_t{at_of<uint16_t>(t), narrow(t.size(0), "cache"), narrow(t.size(2) - 64, "cache"), narrow(t.size(1), "cache")};
}

// The body of a call: counts its arguments and turns what it throws into Python's errors.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t expected, const F &body) {
    try {
        if (n != expected)
            throw std::invalid_argument("expected " + std::to_string(expected) + " arguments, got " + std::to_string(n));
        if (!lib.latent_attention)
            throw std::invalid_argument("set_library() comes first");
        return body();
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *set_library(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 9) {
        PyErr_SetString(PyExc_ValueError, "expected nine addresses");
        return nullptr;
    }
    void *p[9];
    for (int i = 0; i < 9; ++i) {
        p[i] = PyLong_AsVoidPtr(o[i]);
        if (!p[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    lib = Library{reinterpret_cast<decltype(lib.build_tables)>(p[0]), reinterpret_cast<decltype(lib.append)>(p[1]),
                  reinterpret_cast<decltype(lib.attention)>(p[2]), reinterpret_cast<decltype(lib.quantize)>(p[3]),
                  reinterpret_cast<decltype(lib.linear)>(p[4]), reinterpret_cast<decltype(lib.norm)>(p[5]),
                  reinterpret_cast<decltype(lib.rotary)>(p[6]), reinterpret_cast<decltype(lib.latent_append)>(p[7]),
                  reinterpret_cast<decltype(lib.latent_attention)>(p[8])};
    Py_RETURN_NONE;
}

// (k, v, k_scale, v_scale)
PyObject *check_cache(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        Device dev;
        cache_of(dev, o);
        Py_RETURN_NONE;
    });
}

PyObject *check_weight(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 2, [&] {
        Device dev;
        const at::Tensor &c = whole(dev, o[0], at::kByte, "codes");
        weight_of(c, whole(dev, o[1], at::kByte, "scale"));
        Py_RETURN_NONE;
    });
}

// (ctx_lens, new_lens, block_size, free_blocks, free_head, block_table, kv_lens, q_offsets, slot_map, positions,
//  free_head_out, ws, stream)
PyObject *kv_build_tables(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        Device dev;
        const at::Tensor &ctx = whole(dev, o[0], at::kInt, "ctx_lens"), &fresh = whole(dev, o[1], at::kInt, "new_lens");
        const at::Tensor &free = whole(dev, o[3], at::kInt, "free_blocks"), &head = whole(dev, o[4], at::kInt, "free_head");
        const at::Tensor &table = whole(dev, o[5], at::kInt, "block_table"), &kv = whole(dev, o[6], at::kInt, "kv_lens");
        const at::Tensor &qo = whole(dev, o[7], at::kInt, "q_offsets"), &slots = whole(dev, o[8], at::kLong, "slot_map");
        const at::Tensor &pos = whole(dev, o[9], at::kInt, "positions"), &out = whole(dev, o[10], at::kInt, "free_head_out");
        const at::Tensor &ws = whole(dev, o[11], at::kByte, "ws");
        const int64_t B = ctx.numel(), T = slots.numel();
        want(fresh, {B}, "new_lens");
        want(kv, {B}, "kv_lens");
        want(qo, {B + 1}, "q_offsets");
        want(pos, {T}, "positions");
        if (table.dim() != 2 || table.size(0) != B)
            fail("block_table", "expected " + std::to_string(B) + " rows, got " + show(table.sizes()));
        if (head.numel() != 1 || out.numel() != 1)
            fail("free_head", "expected one value");
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.build_tables(
            at_of<int32_t>(ctx), at_of<int32_t>(fresh), narrow(B, "ctx_lens"), narrow(T, "slot_map"), integer(o[2], "block_size"),
            at_of<int32_t>(free), narrow(free.numel(), "free_blocks"), at_of<int32_t>(head), at_of<int32_t>(table),
            narrow(table.size(1), "block_table"), at_of<int32_t>(kv), at_of<int32_t>(qo), at_of<int64_t>(slots),
            at_of<int32_t>(pos), at_of<int32_t>(out), at_of<void>(ws), (size_t)ws.numel(), stream_of(dev, o[12])));
    });
}

// (k, v, slot_map, cache x 4, ws, stream)
PyObject *kv_append(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        Device dev;
        const moe_kv_cache_t c = cache_of(dev, o + 3);
        const at::Tensor &k = heads(dev, o[0], "k"), &v = heads(dev, o[1], "v"), &slots = whole(dev, o[2], at::kLong, "slot_map");
        const at::Tensor &ws = whole(dev, o[7], at::kByte, "ws");
        const int64_t T = slots.numel();
        want(k, {T, c.kv_heads, c.head_dim}, "k");
        want(v, {T, c.kv_heads, c.head_dim}, "v");
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.append(at_of<uint16_t>(k), step(k, 0), step(k, 1), at_of<uint16_t>(v), step(v, 0),
                                          step(v, 1), at_of<int64_t>(slots), narrow(T, "slot_map"), &c, at_of<void>(ws),
                                          (size_t)ws.numel(), stream_of(dev, o[8])));
    });
}

// (q, cache x 4, block_table, q_offsets, kv_lens, softmax_scale, out, lse, ws, causal, window, stream)
PyObject *kv_attention(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        Device dev;
        const moe_kv_cache_t c = cache_of(dev, o + 1);
        const at::Tensor &q = heads(dev, o[0], "q"), &table = whole(dev, o[5], at::kInt, "block_table");
        const at::Tensor &qo = whole(dev, o[6], at::kInt, "q_offsets"), &kv = whole(dev, o[7], at::kInt, "kv_lens");
        const at::Tensor &out = whole(dev, o[9], at::kBFloat16, "out"), &ws = whole(dev, o[11], at::kByte, "ws");
        const int64_t B = kv.numel(), T = q.size(0), H = q.size(1);
        want(q, {T, H, c.head_dim}, "q");
        want(out, {T, H, c.head_dim}, "out");
        want(qo, {B + 1}, "q_offsets");
        if (table.dim() != 2 || table.size(0) != B)
            fail("block_table", "expected " + std::to_string(B) + " rows, got " + show(table.sizes()));
        float *lse = nullptr;
        if (o[10] != Py_None) {
            const at::Tensor &l = whole(dev, o[10], at::kFloat, "lse");
            want(l, {T, H}, "lse");
            lse = at_of<float>(l);
        }
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.attention(
            at_of<uint16_t>(q), step(q, 0), step(q, 1), narrow(T, "q"), narrow(H, "q"), &c, at_of<int32_t>(table),
            narrow(table.size(1), "block_table"), at_of<int32_t>(qo), at_of<int32_t>(kv), narrow(B, "kv_lens"),
            (float)real(o[8]), truth(o[12]), integer(o[13], "window"), at_of<uint16_t>(out), lse, at_of<void>(ws),
            (size_t)ws.numel(), stream_of(dev, o[14])));
    });
}

// (w, codes, scale, stream)
PyObject *quantize_fp8_weight(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        Device dev;
        const at::Tensor &w = whole(dev, o[0], at::kBFloat16, "w"), &codes = whole(dev, o[1], at::kByte, "codes");
        const at::Tensor &scale = whole(dev, o[2], at::kByte, "scale");
        weight_of(codes, scale);
        want(w, {codes.size(0), codes.size(1)}, "w");
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.quantize(at_of<uint16_t>(w), narrow(w.size(0), "w"), narrow(w.size(1), "w"),
                                            at_of<uint8_t>(codes), at_of<uint8_t>(scale), stream_of(dev, o[3])));
    });
}

// (x, codes, scale, y, ws, stream)
PyObject *linear_fp8(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        Device dev;
        const at::Tensor &x = cuda(dev, o[0], at::kBFloat16, "x"), &codes = whole(dev, o[1], at::kByte, "codes");
        const at::Tensor &scale = whole(dev, o[2], at::kByte, "scale"), &y = whole(dev, o[3], at::kBFloat16, "y");
        const at::Tensor &ws = whole(dev, o[4], at::kByte, "ws");
        weight_of(codes, scale);
        const int64_t N = codes.size(0), K = codes.size(1);
        if (x.dim() != 2 || (x.stride(1) != 1 && x.size(1) > 1))
            fail("x", "expected a matrix with contiguous rows");
        const int64_t T = x.size(0);
        want(x, {T, K}, "x");
        want(y, {T, N}, "y");
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.linear(at_of<uint16_t>(x), T > 1 ? x.stride(0) : K, narrow(T, "x"), at_of<uint8_t>(codes),
                                          at_of<uint8_t>(scale), narrow(N, "codes"), narrow(K, "codes"), at_of<uint16_t>(y),
                                          at_of<void>(ws), (size_t)ws.numel(), stream_of(dev, o[5])));
    });
}

// (x, weight, eps, y, residual, residual_out, post_weight, gate, scale, stream)
PyObject *rms_norm(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        Device dev;
        const at::Tensor &x = matrix(dev, o[0], "x");
        const int64_t T = x.size(0), H = x.size(1);
        const uint16_t *weight = vector_of(dev, o[1], H, "weight"), *post = vector_of(dev, o[6], H, "post_weight");
        uint16_t *y = nullptr;
        if (o[3] != Py_None) {
            const at::Tensor &t = whole(dev, o[3], at::kBFloat16, "y");
            want(t, {T, H}, "y");
            y = at_of<uint16_t>(t);
        }
        const at::Tensor *res[2] = {nullptr, nullptr};
        for (int i = 0; i < 2; ++i) {
            const char *name = i ? "residual_out" : "residual";
            if (o[4 + i] == Py_None)
                continue;
            const at::ScalarType type = res[0] ? res[0]->scalar_type() : tensor(o[4 + i], name).scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
            res[i] = &whole(dev, o[4 + i], type, name);
            want(*res[i], {T, H}, name);
        }
        const at::Tensor *first = res[0] ? res[0] : res[1];
        const uint16_t *gate = nullptr;
        int64_t ld_gate = 0;
        if (o[7] != Py_None) {
            const at::Tensor &g = cuda(dev, o[7], at::kBFloat16, "gate");
            if (g.dim() == 1) {
                want(g, {H}, "gate");
                if (g.stride(0) != 1 && H > 1)
                    fail("gate", "expected contiguous values");
            } else {
                matrix(dev, o[7], "gate");
                want(g, {T, H}, "gate");
                ld_gate = T > 1 ? g.stride(0) : H;
            }
            gate = at_of<uint16_t>(g);
        }
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.norm(at_of<uint16_t>(x), T > 1 ? x.stride(0) : H, narrow(T, "x"), narrow(H, "x"), post, gate, ld_gate,
                                        (float)real(o[8]), res[0] ? at_of<void>(*res[0]) : nullptr, res[1] ? at_of<void>(*res[1]) : nullptr,
                                        first && first->scalar_type() == at::kFloat, weight, (float)real(o[2]), y, stream_of(dev, o[9])));
    });
}

// (q, positions, turns, amplitude, q_out, k, k_out, interleaved, offset, q_norm, k_norm, eps, stream)
PyObject *rotary(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        Device dev;
        const at::Tensor &q = heads(dev, o[0], "q"), &q_out = heads(dev, o[4], "q_out");
        const at::Tensor &pos = whole(dev, o[1], at::kInt, "positions"), &turns = whole(dev, o[2], at::kLong, "turns");
        const int64_t T = q.size(0), D = q.size(2);
        want(pos, {T}, "positions");
        want(q_out, {T, q.size(1), D}, "q_out");
        if (turns.dim() != 1)
            fail("turns", "expected a vector, got " + show(turns.sizes()));
        const at::Tensor *k = nullptr, *k_out = nullptr;
        if ((o[5] == Py_None) != (o[6] == Py_None))
            fail("k_out", "expected with k, and only then");
        if (o[5] != Py_None) {
            k = &heads(dev, o[5], "k");
            k_out = &heads(dev, o[6], "k_out");
            want(*k, {T, k->size(1), D}, "k");
            want(*k_out, {T, k->size(1), D}, "k_out");
        } else if (o[10] != Py_None) {
            fail("k_norm", "expected with k only");
        }
        const uint16_t *q_norm = vector_of(dev, o[9], D, "q_norm"), *k_norm = vector_of(dev, o[10], D, "k_norm");
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.rotary(
            at_of<uint16_t>(q), step(q, 0), step(q, 1), at_of<uint16_t>(q_out), step(q_out, 0), step(q_out, 1), narrow(q.size(1), "q"),
            k ? at_of<uint16_t>(*k) : nullptr, k ? step(*k, 0) : 0, k ? step(*k, 1) : 0, k ? at_of<uint16_t>(*k_out) : nullptr,
            k ? step(*k_out, 0) : 0, k ? step(*k_out, 1) : 0, k ? narrow(k->size(1), "k") : 0, narrow(T, "q"), narrow(D, "q"),
            at_of<int32_t>(pos), at_of<uint64_t>(turns), narrow(turns.size(0), "turns"), (float)real(o[3]), truth(o[7]),
            integer(o[8], "offset"), q_norm, k_norm, (float)real(o[11]), stream_of(dev, o[12])));
    });
}

// (cache)
PyObject *check_latent_cache(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 1, [&] {
        Device dev;
        latent_cache_of(dev, o[0]);
        Py_RETURN_NONE;
    });
}

// (c, k, slot_map, cache, ws, positions, turns, amplitude, interleaved, norm, eps, stream)
PyObject *latent_append(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        Device dev;
        const moe_latent_cache_t cache = latent_cache_of(dev, o[3]);
        const at::Tensor &c = matrix(dev, o[0], "c"), &k = matrix(dev, o[1], "k"), &slots = whole(dev, o[2], at::kLong, "slot_map");
        const at::Tensor &ws = whole(dev, o[4], at::kByte, "ws");
        const int64_t T = slots.numel();
        want(c, {T, cache.latent_dim}, "c");
        want(k, {T, 64}, "k");
        if ((o[5] == Py_None) != (o[6] == Py_None))
            fail("positions", "expected with a table, and only then");
        const int32_t *pos = nullptr;
        const uint64_t *turns = nullptr;
        if (o[5] != Py_None) {
            const at::Tensor &p = whole(dev, o[5], at::kInt, "positions"), &t = whole(dev, o[6], at::kLong, "turns");
            want(p, {T}, "positions");
            want(t, {32}, "turns");
            pos = at_of<int32_t>(p);
            turns = at_of<uint64_t>(t);
        }
        const uint16_t *norm = vector_of(dev, o[9], cache.latent_dim, "norm");
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.latent_append(at_of<uint16_t>(c), step(c, 0), at_of<uint16_t>(k), step(k, 0), at_of<int64_t>(slots),
                                                 narrow(T, "slot_map"), pos, turns, (float)real(o[7]), truth(o[8]), norm, (float)real(o[10]),
                                                 &cache, at_of<void>(ws), (size_t)ws.numel(), stream_of(dev, o[11])));
    });
}

// (q_latent, q_rope, cache, block_table, q_offsets, kv_lens, softmax_scale, out, lse, ws, causal, stream)
PyObject *latent_attention(PyObject *, PyObject *const *o, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        Device dev;
        const moe_latent_cache_t cache = latent_cache_of(dev, o[2]);
        const at::Tensor &ql = heads(dev, o[0], "q_latent"), &qr = heads(dev, o[1], "q_rope"), &table = whole(dev, o[3], at::kInt, "block_table");
        const at::Tensor &qo = whole(dev, o[4], at::kInt, "q_offsets"), &kv = whole(dev, o[5], at::kInt, "kv_lens");
        const at::Tensor &out = whole(dev, o[7], at::kBFloat16, "out"), &ws = whole(dev, o[9], at::kByte, "ws");
        const int64_t B = kv.numel(), T = ql.size(0), H = ql.size(1);
        want(ql, {T, H, cache.latent_dim}, "q_latent");
        want(qr, {T, H, 64}, "q_rope");
        want(out, {T, H, cache.latent_dim}, "out");
        want(qo, {B + 1}, "q_offsets");
        if (table.dim() != 2 || table.size(0) != B)
            fail("block_table", "expected " + std::to_string(B) + " rows, got " + show(table.sizes()));
        float *lse = nullptr;
        if (o[8] != Py_None) {
            const at::Tensor &l = whole(dev, o[8], at::kFloat, "lse");
            want(l, {T, H}, "lse");
            lse = at_of<float>(l);
        }
        const c10::cuda::CUDAGuard guard(dev.index());
        return PyLong_FromLong(lib.latent_attention(
            at_of<uint16_t>(ql), step(ql, 0), step(ql, 1), at_of<uint16_t>(qr), step(qr, 0), step(qr, 1), narrow(T, "q_latent"),
            narrow(H, "q_latent"), &cache, at_of<int32_t>(table), narrow(table.size(1), "block_table"), at_of<int32_t>(qo), at_of<int32_t>(kv),
            narrow(B, "kv_lens"), (float)real(o[6]), truth(o[10]), at_of<uint16_t>(out), lse, at_of<void>(ws), (size_t)ws.numel(),
            stream_of(dev, o[11])));
    });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(set_library), FAST(check_cache), FAST(check_weight), FAST(kv_build_tables), FAST(kv_append),
                         FAST(kv_attention), FAST(quantize_fp8_weight), FAST(linear_fp8), FAST(rms_norm), FAST(rotary),
                         FAST(check_latent_cache), FAST(latent_append), FAST(latent_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_native() { return PyModule_Create(&module); }
