// Marshalling of the calls of include/adaln_ops.h and adaln_tune.h for Python: checks PyTorch
// tensors, copies inputs whose layout the C ABI refuses, allocates missing
// outputs and workspaces, and calls the C ABI on the current stream.  No
// computation.  In Python these steps took 10 to 35 us a call, several times
// the launches themselves and, for single tokens, the kernels.
//
// The C functions come as addresses (`bind`), so that this module works with
// whichever build of the library the process has loaded.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>

#include <array>
#include <initializer_list>
#include <string>
#include <utility>
#include <vector>

#include "adaln_ops.h"
#include "adaln_tune.h"

namespace {

// ---- the library's functions -------------------------------------------------

struct Library {
    decltype(&adaln_qk_norm_rope_fwd) qk_fwd;
    decltype(&adaln_f32_qk_norm_rope_fwd) f32_qk_fwd;
    decltype(&adaln_qk_norm_rope_bwd_workspace_bytes) qk_bwd_bytes;
    decltype(&adaln_qk_norm_rope_bwd) qk_bwd;
    decltype(&adaln_f32_qk_norm_rope_bwd) f32_qk_bwd;
    decltype(&adaln_embed_fwd) embed_fwd;
    decltype(&adaln_f32_embed_fwd) f32_embed_fwd;
    decltype(&adaln_embed_bwd_workspace_bytes) embed_bwd_bytes;
    decltype(&adaln_embed_bwd) embed_bwd;
    decltype(&adaln_f32_embed_bwd) f32_embed_bwd;
    decltype(&adaln_grad_norm_workspace_bytes) grad_bytes;
    decltype(&adaln_grad_norm) grad_norm;
    decltype(&adaln_grad_clip) grad_clip;
    decltype(&adaln_ckpt8_row_bytes) ckpt8_bytes;
    decltype(&adaln_ckpt8_pack) ckpt8_pack;
    decltype(&adaln_f32_ckpt8_pack) f32_ckpt8_pack;
    decltype(&adaln_ckpt8_unpack) ckpt8_unpack;
    decltype(&adaln_f32_ckpt8_unpack) f32_ckpt8_unpack;
    decltype(&adaln_out_fwd_ckpt8) fwd_ckpt8;
    decltype(&adaln_f32_out_fwd_ckpt8) f32_fwd_ckpt8;
    decltype(&adaln_out_bwd_ckpt8_workspace_bytes) bwd_ckpt8_bytes;
    decltype(&adaln_out_bwd_ckpt8) bwd_ckpt8;
    decltype(&adaln_f32_out_bwd_ckpt8) f32_bwd_ckpt8;
    decltype(&adaln_out_again_ckpt8) again_ckpt8;
    decltype(&adaln_f32_out_again_ckpt8) f32_again_ckpt8;
    decltype(&adaln_lora_state_bytes) lora_state_bytes;
    decltype(&adaln_lora_fwd) lora_fwd;
    decltype(&adaln_f32_lora_fwd) f32_lora_fwd;
    decltype(&adaln_lora_bwd_workspace_bytes) lora_bwd_bytes;
    decltype(&adaln_f32_lora_bwd_workspace_bytes) f32_lora_bwd_bytes;
    decltype(&adaln_lora_bwd) lora_bwd;
    decltype(&adaln_f32_lora_bwd) f32_lora_bwd;
} lib;
PyObject *raise_status;  // called with (name, status); raises

// ---- refusals ------------------------------------------------------------------

struct Refused {};  // thrown with the Python error set

template <typename... A>
[[noreturn]] void refuse(PyObject *type, const char *format, A... args) {
    PyErr_Format(type, format, args...);
    throw Refused();
}

void status(const char *name, adaln_status st) {
    if (st == ADALN_OK) return;
    PyObject *r = PyObject_CallFunction(raise_status, "si", name, (int)st);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
    throw Refused();
}

// ---- tensors -------------------------------------------------------------------

using at::Tensor;
using at::ScalarType;
using Shape = std::initializer_list<int64_t>;

const char *type_name(ScalarType t) {
    return t == at::kBFloat16 ? "torch.bfloat16" : t == at::kFloat ? "torch.float32" : t == at::kInt ? "torch.int32"
           : t == at::kByte                                                                    ? "torch.uint8"
                                                                                               : "torch.int64";
}

bool given(PyObject *o) { return o != Py_None; }

// the tensor behind o: on the current device `dev`, of type t (or u)
const Tensor &tensor(PyObject *o, const char *name, int dev, ScalarType t, ScalarType u) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s: expected a CUDA tensor", name);
    const Tensor &x = THPVariable_Unpack(o);
    if (!x.is_cuda()) refuse(PyExc_TypeError, "%s: expected a CUDA tensor", name);
    if (x.scalar_type() != t && x.scalar_type() != u)
        refuse(PyExc_TypeError, t == u ? "%s: expected %s" : "%s: expected %s or %s", name, type_name(t), type_name(u));
    if (x.get_device() != dev)
        refuse(PyExc_ValueError, "%s: on cuda:%d, but the current device is %d", name, (int)x.get_device(), dev);
    return x;
}

int current_device() { return c10::cuda::current_device(); }

// The current device, known to be one: o is a CUDA tensor (without CUDA there is none).
int device_of(PyObject *o, const char *name) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        refuse(PyExc_TypeError, "%s: expected a CUDA tensor", name);
    return current_device();
}

void shape_is(const Tensor &x, at::IntArrayRef want, const char *name) {
    if (x.sizes() == want) return;
    std::string s = "(", g = "(";
    for (int64_t n : want) s += std::to_string(n) + ",";
    for (int64_t n : x.sizes()) g += std::to_string(n) + ",";
    refuse(PyExc_ValueError, "%s: expected shape %s), got %s)", name, s.c_str(), g.c_str());
}

bool aligned(const Tensor &x) { return ((uintptr_t)x.data_ptr() & 15u) == 0; }

// a dense 16-byte aligned input: x, or a copy of it
Tensor flat(const Tensor &x) {
    if (!x.is_contiguous()) return x.contiguous();
    return aligned(x) ? x : x.clone();
}
Tensor flat(PyObject *o, const char *name, int dev, ScalarType t, ScalarType u, at::IntArrayRef shape) {
    const Tensor &x = tensor(o, name, dev, t, u);
    shape_is(x, shape, name);
    return flat(x);
}

Tensor make(at::IntArrayRef shape, ScalarType t, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(t).device(at::Device(at::kCUDA, (c10::DeviceIndex)dev)));
}

// a dense 16-byte aligned output: o, or a new one
Tensor result(PyObject *o, const char *name, int dev, ScalarType t, at::IntArrayRef shape) {
    if (!given(o)) return make(shape, t, dev);
    const Tensor &x = tensor(o, name, dev, t, t);
    shape_is(x, shape, name);
    if (!x.is_contiguous() || !aligned(x))
        refuse(PyExc_ValueError, "%s: must be contiguous and 16-byte aligned", name);
    return x;
}

// a workspace of `need` bytes: o, or a new one
Tensor scratch(PyObject *o, size_t need, int dev) {
    if (!given(o)) return need ? make({(int64_t)need}, at::kByte, dev) : Tensor();
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda() || !THPVariable_Unpack(o).is_contiguous())
        refuse(PyExc_ValueError, "workspace: expected a contiguous CUDA tensor");
    const Tensor &x = THPVariable_Unpack(o);
    if (x.get_device() != dev)
        refuse(PyExc_ValueError, "workspace: on cuda:%d, but the current device is %d", (int)x.get_device(), dev);
    if (x.nbytes() < need) refuse(PyExc_ValueError, "workspace: %zu bytes needed", need);
    return x;
}

void *ptr(const Tensor &x) { return x.defined() ? x.data_ptr() : nullptr; }
void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}
long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
// a size for the C ABI, which refuses what int cannot hold by the largest value
int size_of(long long v) { return v > 0x7FFFFFFF ? 0x7FFFFFFF : v < -1 ? -1 : (int)v; }
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}

// ---- head rows -------------------------------------------------------------------

// Head rows [B, S, H, Dh]: x itself where its channels are dense and its rows
// 16-byte aligned, else a copy (an input) or a refusal (an output).
struct Rows {
    Tensor x;
    adaln_heads h;
    Rows() = default;
    Rows(Tensor t, const char *name, bool copy) : x(std::move(t)) {
        if (!usable()) {
            if (!copy) refuse(PyExc_ValueError, "%s: channels must be dense and rows 16-byte aligned", name);
            x = x.clone(at::MemoryFormat::Contiguous);
        }
        const auto st = x.strides();
        h = adaln_heads{x.data_ptr(), st[0], st[1], st[2]};
    }
    bool usable() const {
        if (x.numel() == 0) return true;
        const int64_t step = 16 / x.element_size();
        if ((x.stride(3) != 1 && x.size(3) > 1) || !aligned(x)) return false;
        for (int i = 0; i < 3; ++i)
            if (x.size(i) > 1 && x.stride(i) % step != 0) return false;
        return true;
    }
};
Rows rows_in(PyObject *o, const char *name, int dev, ScalarType t, at::IntArrayRef shape) {
    const Tensor &x = tensor(o, name, dev, t, t);
    shape_is(x, shape, name);
    return Rows(x, name, true);
}
Rows rows_out(PyObject *o, const char *name, int dev, ScalarType t, at::IntArrayRef shape) {
    if (!given(o)) return Rows(make(shape, t, dev), name, false);
    const Tensor &x = tensor(o, name, dev, t, t);
    shape_is(x, shape, name);
    return Rows(x, name, false);
}

// what forward and backward share
struct HeadSizes {
    int dev;
    std::array<int64_t, 4> q, k;  // shapes
    bool keys;
    int B, S, Hq, Hk, Dh, Dr, P, is64;
    Tensor wq, wk, cos, sin, pos;

    HeadSizes(ScalarType t, PyObject *oq, PyObject *ok, PyObject *owq, PyObject *owk, PyObject *ocos, PyObject *osin,
              PyObject *opos) {
        if (!THPVariable_Check(oq) || THPVariable_Unpack(oq).dim() != 4)
            refuse(PyExc_ValueError, "q: expected a tensor [B, S, H, Dh]");
        dev = device_of(oq, "q");
        const auto n = THPVariable_Unpack(oq).sizes();
        q = k = {n[0], n[1], n[2], n[3]};
        keys = given(ok);
        k[2] = 0;
        if (keys) {
            if (!THPVariable_Check(ok) || THPVariable_Unpack(ok).dim() != 4)
                refuse(PyExc_ValueError, "k: expected a tensor [B, S, H, Dh]");
            k[2] = THPVariable_Unpack(ok).size(2);
            if (given(owk)) wk = flat(owk, "wk", dev, t, t, {q[3]});
        }
        if (given(owq)) wq = flat(owq, "wq", dev, t, t, {q[3]});
        int64_t p = 0x7FFFFFFF, half = 0;
        if (given(ocos) != given(osin)) refuse(PyExc_ValueError, "cos, sin: give both or neither");
        if (given(ocos)) {
            if (!THPVariable_Check(ocos) || THPVariable_Unpack(ocos).dim() != 2)
                refuse(PyExc_ValueError, "cos: expected a tensor [P, Dr / 2]");
            p = THPVariable_Unpack(ocos).size(0);
            half = THPVariable_Unpack(ocos).size(1);
            cos = flat(ocos, "cos", dev, at::kFloat, at::kFloat, {p, half});
            sin = flat(osin, "sin", dev, at::kFloat, at::kFloat, {p, half});
        }
        is64 = 0;
        if (given(opos)) {
            pos = flat(opos, "pos", dev, at::kInt, at::kLong, {q[0], q[1]});
            is64 = pos.scalar_type() == at::kLong;
        }
        B = size_of(q[0]), S = size_of(q[1]), Hq = size_of(q[2]), Hk = size_of(k[2]), Dh = size_of(q[3]);
        Dr = size_of(2 * half), P = size_of(p);
    }
};

// without k there is nothing to write to the outputs for it, or to read
void no_keys(std::initializer_list<std::pair<PyObject *, const char *>> args) {
    for (const auto &a : args)
        if (given(a.first)) refuse(PyExc_ValueError, "%s: given without k", a.second);
}

ScalarType float_type(PyObject *o) { return truth(o) ? at::kFloat : at::kBFloat16; }

// qk_fwd(f32, q, k, wq, wk, cos, sin, pos, q_out, k_out, eps, interleaved)
PyObject *qk_fwd(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const HeadSizes z(t, a[1], a[2], a[3], a[4], a[5], a[6], a[7]);
    const float eps = (float)number(a[10]);
    const int inter = truth(a[11]);
    const Rows q = rows_in(a[1], "q", z.dev, t, z.q), qo = rows_out(a[8], "q_out", z.dev, t, z.q);
    Rows k, ko;
    if (z.keys) {
        k = rows_in(a[2], "k", z.dev, t, z.k);
        ko = rows_out(a[9], "k_out", z.dev, t, z.k);
    } else {
        no_keys({{a[9], "k_out"}});
    }
    const adaln_heads *kh = z.keys ? &k.h : nullptr, *koh = z.keys ? &ko.h : nullptr;
    const float *c = (const float *)ptr(z.cos), *s = (const float *)ptr(z.sin);
    if (t == at::kFloat)
        status("adaln_f32_qk_norm_rope_fwd",
               lib.f32_qk_fwd(&q.h, kh, (const float *)ptr(z.wq), (const float *)ptr(z.wk), c, s, ptr(z.pos), z.is64,
                              &qo.h, koh, z.B, z.S, z.Hq, z.Hk, z.Dh, z.Dr, z.P, inter, eps, stream_of(z.dev)));
    else
        status("adaln_qk_norm_rope_fwd",
               lib.qk_fwd(&q.h, kh, (const adaln_bf16 *)ptr(z.wq), (const adaln_bf16 *)ptr(z.wk), c, s, ptr(z.pos),
                          z.is64, &qo.h, koh, z.B, z.S, z.Hq, z.Hk, z.Dh, z.Dr, z.P, inter, eps, stream_of(z.dev)));
    return Py_BuildValue("(NN)", THPVariable_Wrap(qo.x), z.keys ? THPVariable_Wrap(ko.x) : Py_NewRef(a[9]));
}

// qk_bwd(f32, d_q_out, d_k_out, q, k, wq, wk, cos, sin, pos, d_q, d_k, dwq_acc, dwk_acc, accumulate, want_w,
//        workspace, eps, interleaved)
PyObject *qk_bwd(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const HeadSizes z(t, a[3], a[4], a[5], a[6], a[7], a[8], a[9]);
    const bool accumulate = truth(a[14]), want_w = truth(a[15]);
    const float eps = (float)number(a[17]);
    const int inter = truth(a[18]);
    const Rows gq = rows_in(a[1], "d_q_out", z.dev, t, z.q), q = rows_in(a[3], "q", z.dev, t, z.q),
               dq = rows_out(a[10], "d_q", z.dev, t, z.q);
    Rows gk, k, dk;
    if (z.keys) {
        gk = rows_in(a[2], "d_k_out", z.dev, t, z.k);
        k = rows_in(a[4], "k", z.dev, t, z.k);
        dk = rows_out(a[11], "d_k", z.dev, t, z.k);
    } else {
        no_keys({{a[2], "d_k_out"}, {a[11], "d_k"}, {a[13], "dwk_acc"}});
    }
    // given accumulators are filled; want_w allocates the missing ones
    Tensor dwq, dwk, ws;
    size_t need = 0;
    if (want_w && accumulate && (!given(a[12]) || (z.keys && !given(a[13]))))
        refuse(PyExc_ValueError, "accumulate: dwq_acc and dwk_acc must be given");
    if (want_w || given(a[12])) dwq = result(a[12], "dwq_acc", z.dev, at::kFloat, {z.q[3]});
    if ((want_w && z.Hk) || given(a[13])) dwk = result(a[13], "dwk_acc", z.dev, at::kFloat, {z.q[3]});
    if (dwq.defined() || dwk.defined()) {
        need = lib.qk_bwd_bytes(z.B, z.S, z.Hq, z.Hk, z.Dh);
        ws = scratch(a[16], need, z.dev);
    }
    const adaln_heads *gkh = z.keys ? &gk.h : nullptr, *kh = z.keys ? &k.h : nullptr, *dkh = z.keys ? &dk.h : nullptr;
    const float *c = (const float *)ptr(z.cos), *s = (const float *)ptr(z.sin);
    float *pq = (float *)ptr(dwq), *pk = (float *)ptr(dwk);
    if (t == at::kFloat)
        status("adaln_f32_qk_norm_rope_bwd",
               lib.f32_qk_bwd(&gq.h, gkh, &q.h, kh, (const float *)ptr(z.wq), (const float *)ptr(z.wk), c, s,
                              ptr(z.pos), z.is64, &dq.h, dkh, pq, pk, accumulate, ptr(ws), need, z.B, z.S, z.Hq, z.Hk,
                              z.Dh, z.Dr, z.P, inter, eps, stream_of(z.dev)));
    else
        status("adaln_qk_norm_rope_bwd",
               lib.qk_bwd(&gq.h, gkh, &q.h, kh, (const adaln_bf16 *)ptr(z.wq), (const adaln_bf16 *)ptr(z.wk), c, s,
                          ptr(z.pos), z.is64, &dq.h, dkh, pq, pk, accumulate, ptr(ws), need, z.B, z.S, z.Hq, z.Hk, z.Dh,
                          z.Dr, z.P, inter, eps, stream_of(z.dev)));
    return Py_BuildValue("(NNNN)", THPVariable_Wrap(dq.x), z.keys ? THPVariable_Wrap(dk.x) : Py_NewRef(a[11]),
                         dwq.defined() ? THPVariable_Wrap(dwq) : Py_NewRef(a[12]),
                         dwk.defined() ? THPVariable_Wrap(dwk) : Py_NewRef(a[13]));
}

// ---- embedding -------------------------------------------------------------------

std::vector<int64_t> with_last(const Tensor &x, int64_t D) {
    std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
    shape.push_back(D);
    return shape;
}

// embed_fwd(f32, tokens, table, scale, out)
PyObject *embed_fwd(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const int dev = device_of(a[1], "tokens");
    const Tensor tokens = flat(tensor(a[1], "tokens", dev, at::kInt, at::kLong));
    if (!THPVariable_Check(a[2]) || THPVariable_Unpack(a[2]).dim() != 2)
        refuse(PyExc_ValueError, "table: expected a tensor [V, D]");
    const Tensor table = flat(tensor(a[2], "table", dev, t, t));
    const float scale = (float)number(a[3]);
    const int64_t V = table.size(0), D = table.size(1);
    const Tensor out = result(a[4], "out", dev, t, with_last(tokens, D));
    const int is64 = tokens.scalar_type() == at::kLong, n = size_of(tokens.numel());
    if (t == at::kFloat)
        status("adaln_f32_embed_fwd", lib.f32_embed_fwd(ptr(tokens), is64, (const float *)ptr(table), scale,
                                                        (float *)ptr(out), n, size_of(V), size_of(D), stream_of(dev)));
    else
        status("adaln_embed_fwd", lib.embed_fwd(ptr(tokens), is64, (const adaln_bf16 *)ptr(table), scale,
                                                (adaln_bf16 *)ptr(out), n, size_of(V), size_of(D), stream_of(dev)));
    return THPVariable_Wrap(out);
}

// embed_bwd(f32, d_out, tokens, V, scale, d_table_acc, d_table, accumulate, workspace)
PyObject *embed_bwd(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const int dev = device_of(a[2], "tokens");
    const Tensor tokens = flat(tensor(a[2], "tokens", dev, at::kInt, at::kLong));
    if (!THPVariable_Check(a[1]) || THPVariable_Unpack(a[1]).dim() < 1)
        refuse(PyExc_ValueError, "d_out: expected a tensor [..., D]");
    const int64_t D = THPVariable_Unpack(a[1]).size(-1), V = integer(a[3]);
    const Tensor d_out = flat(a[1], "d_out", dev, t, t, with_last(tokens, D));
    const float scale = (float)number(a[4]);
    const bool accumulate = truth(a[7]);
    if (V < 0) refuse(PyExc_ValueError, "V: must not be negative");
    const int n = size_of(tokens.numel());
    const size_t need = lib.embed_bwd_bytes(n, size_of(V), size_of(D));
    const Tensor ws = scratch(a[8], need, dev);
    Tensor acc, low;
    if (given(a[6])) {
        low = result(a[6], "d_table", dev, at::kBFloat16, {V, D});
        if (given(a[5])) acc = result(a[5], "d_table_acc", dev, at::kFloat, {V, D});  // refused by the C ABI
    } else {
        if (accumulate && !given(a[5])) refuse(PyExc_ValueError, "accumulate: d_table_acc must be given");
        acc = result(a[5], "d_table_acc", dev, at::kFloat, {V, D});
    }
    const int is64 = tokens.scalar_type() == at::kLong;
    if (t == at::kFloat)
        status("adaln_f32_embed_bwd",
               lib.f32_embed_bwd((const float *)ptr(d_out), ptr(tokens), is64, scale, (float *)ptr(acc), accumulate,
                                 ptr(ws), need, n, size_of(V), size_of(D), stream_of(dev)));
    else
        status("adaln_embed_bwd",
               lib.embed_bwd((const adaln_bf16 *)ptr(d_out), ptr(tokens), is64, scale, (float *)ptr(acc),
                             (adaln_bf16 *)ptr(low), accumulate, ptr(ws), need, n, size_of(V), size_of(D),
                             stream_of(dev)));
    return THPVariable_Wrap(low.defined() ? low : acc);
}

// ---- gradient lists -----------------------------------------------------------------

struct List {
    PyObject *seq;  // keeps the tensors for the call
    std::vector<adaln_tensor> t;
    List(PyObject *o, const char *name, int dev) : seq(PySequence_Fast(o, "expected a sequence of tensors")) {
        if (!seq) throw Refused();
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
        try {
            t.reserve((size_t)n);
            for (Py_ssize_t i = 0; i < n; ++i) {
                const Tensor &x = tensor(PySequence_Fast_GET_ITEM(seq, i), name, dev, at::kFloat, at::kBFloat16);
                if (!x.is_contiguous()) refuse(PyExc_ValueError, "%s: tensors must be contiguous", name);
                t.push_back({x.data_ptr(), x.numel(), x.scalar_type() == at::kBFloat16 ? ADALN_BF16 : ADALN_F32, 0});
            }
        } catch (...) {
            Py_DECREF(seq);
            throw;
        }
    }
    List(const List &) = delete;
    ~List() { Py_DECREF(seq); }
    int count() const { return size_of((long long)t.size()); }
};

// grad_workspace_bytes(grads)
PyObject *grad_workspace_bytes(PyObject *const *a) {
    const List grads(a[0], "grads", current_device());
    return PyLong_FromSize_t(lib.grad_bytes(grads.t.data(), grads.count()));
}

// grad_norm(grads, norm, workspace)
PyObject *grad_norm(PyObject *const *a) {
    const int dev = current_device();
    const List grads(a[0], "grads", dev);
    const Tensor norm = result(a[1], "norm", dev, at::kFloat, {1});
    const size_t need = lib.grad_bytes(grads.t.data(), grads.count());
    const Tensor ws = scratch(a[2], need, dev);
    status("adaln_grad_norm",
           lib.grad_norm(grads.t.data(), grads.count(), (float *)ptr(norm), ptr(ws), need, stream_of(dev)));
    return THPVariable_Wrap(norm);
}

// grad_clip(grads, max_norm, outs, stats, workspace)
PyObject *grad_clip(PyObject *const *a) {
    const int dev = current_device();
    const List grads(a[0], "grads", dev);
    const double max_norm = number(a[1]);
    struct Keep {
        PyObject *o;
        ~Keep() { Py_XDECREF(o); }
    } keep{given(a[2]) ? Py_NewRef(a[2]) : PyList_New(0)};
    PyObject *outs = keep.o;
    if (!outs) throw Refused();
    if (!given(a[2])) {
        for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(grads.seq); ++i) {
            PyObject *t = THPVariable_Wrap(at::empty_like(THPVariable_Unpack(PySequence_Fast_GET_ITEM(grads.seq, i))));
            const int bad = t ? PyList_Append(outs, t) : -1;
            Py_XDECREF(t);
            if (bad) throw Refused();
        }
    }
    const List to(outs, "outs", dev);
    if (to.t.size() != grads.t.size()) refuse(PyExc_ValueError, "outs: expected as many tensors as grads");
    const Tensor stats = result(a[3], "stats", dev, at::kFloat, {2});
    const size_t need = lib.grad_bytes(grads.t.data(), grads.count());
    const Tensor ws = scratch(a[4], need, dev);
    status("adaln_grad_clip", lib.grad_clip(grads.t.data(), to.t.data(), grads.count(), max_norm, (float *)ptr(stats),
                                            ptr(ws), need, stream_of(dev)));
    // the caller's own object, but for an iterator, which is used up by now
    return Py_BuildValue("(ON)", PyIter_Check(outs) ? to.seq : outs, THPVariable_Wrap(stats));
}

// ---- activations in 8 bits ----------------------------------------------------------

// the sizes of a dense [..., D] tensor without its last dimension
std::vector<int64_t> leading(const Tensor &x) {
    return std::vector<int64_t>(x.sizes().begin(), x.sizes().end() - 1);
}
std::vector<int64_t> with(std::vector<int64_t> shape, int64_t last) {
    shape.push_back(last);
    return shape;
}

int64_t rows_before(const std::vector<int64_t> &lead) {
    int64_t rows = 1;
    for (int64_t n : lead) rows *= n;
    return rows;
}

const Tensor &of_dim(PyObject *o, const char *name, int64_t least, int64_t most, const char *shape) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s: expected a CUDA tensor", name);
    const Tensor &x = THPVariable_Unpack(o);
    if (x.dim() < least || x.dim() > most) refuse(PyExc_ValueError, "%s: expected a tensor %s", name, shape);
    return x;
}

// bytes of a record of D channels; refuses a D without records
int64_t record(int64_t D) {
    const size_t n = lib.ckpt8_bytes(size_of(D));
    if (n == 0) refuse(PyExc_ValueError, "ckpt: no records of %lld channels", (long long)D);
    return (int64_t)n;
}

// ckpt8_pack(f32, x, ckpt)
PyObject *ckpt8_pack(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const int dev = device_of(a[1], "x");
    of_dim(a[1], "x", 1, 64, "[..., D]");
    const Tensor x = flat(tensor(a[1], "x", dev, t, t));
    const auto lead = leading(x);
    const int64_t D = x.size(-1), rows = rows_before(lead);
    const Tensor ckpt = result(a[2], "ckpt", dev, at::kByte, with(lead, record(D)));
    if (t == at::kFloat)
        status("adaln_f32_ckpt8_pack", lib.f32_ckpt8_pack((const float *)ptr(x), (uint8_t *)ptr(ckpt), rows,
                                                          size_of(D), stream_of(dev)));
    else
        status("adaln_ckpt8_pack", lib.ckpt8_pack((const adaln_bf16 *)ptr(x), (uint8_t *)ptr(ckpt), rows, size_of(D),
                                                  stream_of(dev)));
    return THPVariable_Wrap(ckpt);
}

// ckpt8_unpack(f32, ckpt, D, out)
PyObject *ckpt8_unpack(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const int dev = device_of(a[1], "ckpt");
    const int64_t D = integer(a[2]);
    const auto lead = leading(of_dim(a[1], "ckpt", 1, 64, "[..., row_bytes]"));
    const Tensor ckpt = flat(a[1], "ckpt", dev, at::kByte, at::kByte, with(lead, record(D)));
    const Tensor out = result(a[3], "out", dev, t, with(lead, D));
    if (t == at::kFloat)
        status("adaln_f32_ckpt8_unpack", lib.f32_ckpt8_unpack((const uint8_t *)ptr(ckpt), (float *)ptr(out),
                                                              rows_before(lead), size_of(D), stream_of(dev)));
    else
        status("adaln_ckpt8_unpack", lib.ckpt8_unpack((const uint8_t *)ptr(ckpt), (adaln_bf16 *)ptr(out),
                                                      rows_before(lead), size_of(D), stream_of(dev)));
    return THPVariable_Wrap(out);
}

// out_fwd_ckpt8(f32, x, emb, out, mean, rstd, ckpt, eps)
PyObject *out_fwd_ckpt8(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const int dev = device_of(a[1], "x");
    of_dim(a[1], "x", 3, 3, "[B, S, D]");
    const Tensor x = flat(tensor(a[1], "x", dev, t, t));
    const int64_t B = x.size(0), S = x.size(1), D = x.size(2);
    const Tensor emb = flat(a[2], "emb", dev, t, t, {B, 2 * D});
    const Tensor ckpt = result(a[6], "ckpt", dev, at::kByte, {B, S, record(D)});
    const Tensor out = result(a[3], "out", dev, t, {B, S, D}), mean = result(a[4], "mean", dev, at::kFloat, {B, S}),
                 rstd = result(a[5], "rstd", dev, at::kFloat, {B, S});
    const float eps = (float)number(a[7]);
    if (t == at::kFloat)
        status("adaln_f32_out_fwd_ckpt8",
               lib.f32_fwd_ckpt8((const float *)ptr(x), (const float *)ptr(emb), (float *)ptr(out), (float *)ptr(mean),
                                 (float *)ptr(rstd), (uint8_t *)ptr(ckpt), size_of(B), size_of(S), size_of(D), eps,
                                 stream_of(dev)));
    else
        status("adaln_out_fwd_ckpt8",
               lib.fwd_ckpt8((const adaln_bf16 *)ptr(x), (const adaln_bf16 *)ptr(emb), (adaln_bf16 *)ptr(out),
                             (float *)ptr(mean), (float *)ptr(rstd), (uint8_t *)ptr(ckpt), size_of(B), size_of(S),
                             size_of(D), eps, stream_of(dev)));
    return Py_BuildValue("(NNNN)", THPVariable_Wrap(out), THPVariable_Wrap(mean), THPVariable_Wrap(rstd),
                         THPVariable_Wrap(ckpt));
}

// out_bwd_ckpt8(f32, dy, ckpt, emb, mean, rstd, dx, d_emb, workspace)
PyObject *out_bwd_ckpt8(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const int dev = device_of(a[1], "dy");
    of_dim(a[1], "dy", 3, 3, "[B, S, D]");
    const Tensor dy = flat(tensor(a[1], "dy", dev, t, t));
    const int64_t B = dy.size(0), S = dy.size(1), D = dy.size(2);
    const Tensor ckpt = flat(a[2], "ckpt", dev, at::kByte, at::kByte, {B, S, record(D)});
    const Tensor emb = flat(a[3], "emb", dev, t, t, {B, 2 * D});
    const Tensor mean = flat(a[4], "mean", dev, at::kFloat, at::kFloat, {B, S}),
                 rstd = flat(a[5], "rstd", dev, at::kFloat, at::kFloat, {B, S});
    const Tensor dx = result(a[6], "dx", dev, t, {B, S, D}), d_emb = result(a[7], "d_emb", dev, at::kFloat, {B, 2 * D});
    const int b = size_of(B), s = size_of(S), d = size_of(D);
    const size_t need = lib.bwd_ckpt8_bytes(b, s, d);
    const Tensor ws = scratch(a[8], need, dev);
    if (t == at::kFloat)
        status("adaln_f32_out_bwd_ckpt8",
               lib.f32_bwd_ckpt8((const float *)ptr(dy), (const uint8_t *)ptr(ckpt), (const float *)ptr(emb),
                                 (const float *)ptr(mean), (const float *)ptr(rstd), (float *)ptr(dx),
                                 (float *)ptr(d_emb), ptr(ws), need, b, s, d, stream_of(dev)));
    else
        status("adaln_out_bwd_ckpt8",
               lib.bwd_ckpt8((const adaln_bf16 *)ptr(dy), (const uint8_t *)ptr(ckpt), (const adaln_bf16 *)ptr(emb),
                             (const float *)ptr(mean), (const float *)ptr(rstd), (adaln_bf16 *)ptr(dx),
                             (float *)ptr(d_emb), ptr(ws), need, b, s, d, stream_of(dev)));
    return Py_BuildValue("(NN)", THPVariable_Wrap(dx), THPVariable_Wrap(d_emb));
}

// out_again_ckpt8(f32, ckpt, emb, mean, rstd, out)
PyObject *out_again_ckpt8(PyObject *const *a) {
    const ScalarType t = float_type(a[0]);
    const int dev = device_of(a[1], "ckpt");
    const Tensor &c = of_dim(a[1], "ckpt", 3, 3, "[B, S, row_bytes]");
    const int64_t B = c.size(0), S = c.size(1), D = of_dim(a[2], "emb", 2, 2, "[B, 2D]").size(1) / 2;
    const Tensor ckpt = flat(a[1], "ckpt", dev, at::kByte, at::kByte, {B, S, record(D)});
    const Tensor emb = flat(a[2], "emb", dev, t, t, {B, 2 * D});
    const Tensor mean = flat(a[3], "mean", dev, at::kFloat, at::kFloat, {B, S}),
                 rstd = flat(a[4], "rstd", dev, at::kFloat, at::kFloat, {B, S});
    const Tensor out = result(a[5], "out", dev, t, {B, S, D});
    if (t == at::kFloat)
        status("adaln_f32_out_again_ckpt8",
               lib.f32_again_ckpt8((const uint8_t *)ptr(ckpt), (const float *)ptr(emb), (const float *)ptr(mean),
                                   (const float *)ptr(rstd), (float *)ptr(out), size_of(B), size_of(S), size_of(D),
                                   stream_of(dev)));
    else
        status("adaln_out_again_ckpt8",
               lib.again_ckpt8((const uint8_t *)ptr(ckpt), (const adaln_bf16 *)ptr(emb), (const float *)ptr(mean),
                               (const float *)ptr(rstd), (adaln_bf16 *)ptr(out), size_of(B), size_of(S), size_of(D),
                               stream_of(dev)));
    return THPVariable_Wrap(out);
}

// ---- low-rank adapters -----------------------------------------------------------------

// Rows [B, S, C]: x itself where the C ABI takes its strides, else a copy (an
// input) or a refusal (an output).
struct TokenRows {
    Tensor x;
    adaln_rows r = {nullptr, 0, 0};
    TokenRows() = default;
    TokenRows(Tensor t, const char *name, bool copy, bool positive) : x(std::move(t)) {
        if (!usable(positive)) {
            if (!copy) refuse(PyExc_ValueError, "%s: channels must be dense and rows 16-byte aligned", name);
            x = x.clone(at::MemoryFormat::Contiguous);
        }
        r = adaln_rows{x.data_ptr(), x.stride(0), x.stride(1)};
    }
    // a tensor allocated here: what its size makes impossible the C ABI refuses by that size
    explicit TokenRows(Tensor t) : x(std::move(t)), r{x.data_ptr(), x.stride(0), x.stride(1)} {}
    bool usable(bool positive) const {
        if (x.numel() == 0) return true;
        const int64_t step = 16 / x.element_size();
        if ((x.stride(2) != 1 && x.size(2) > 1) || !aligned(x)) return false;
        for (int i = 0; i < 2; ++i)
            if (x.size(i) > 1 && (x.stride(i) % step != 0 || (positive && x.stride(i) == 0))) return false;
        return true;
    }
};
TokenRows token_rows(PyObject *o, const char *name, int dev, ScalarType t, at::IntArrayRef shape, bool input,
                     bool positive) {
    const Tensor &x = tensor(o, name, dev, t, t);
    shape_is(x, shape, name);
    return TokenRows(x, name, input, positive);
}

// what forward and backward share
struct Adapters {
    ScalarType t;
    int dev;
    int64_t b, s, k, n, r, na;
    int B, S, K, N, R, NA, is64;
    Tensor A, U, scale, ids, lens;

    Adapters(PyObject *of32, PyObject *ox, PyObject *oA, PyObject *oU, PyObject *oscale, PyObject *oids,
             PyObject *olens)
        : t(float_type(of32)), dev(device_of(ox, "x")) {
        const Tensor &x = of_dim(ox, "x", 3, 3, "[B, S, K]");
        b = x.size(0), s = x.size(1), k = x.size(2);
        const Tensor &a = of_dim(oA, "A", 3, 3, "[NA, R, K]"), &u = of_dim(oU, "U", 3, 3, "[NA, R, N]");
        na = a.size(0), r = a.size(1), n = u.size(2);
        A = flat(oA, "A", dev, t, t, {na, r, k});
        U = flat(oU, "U", dev, t, t, {na, r, n});
        scale = flat(oscale, "scale", dev, at::kFloat, at::kFloat, {na});
        ids = flat(oids, "ids", dev, at::kInt, at::kLong, {b});
        is64 = ids.scalar_type() == at::kLong;
        if (given(olens)) lens = flat(olens, "lens", dev, at::kInt, at::kInt, {b});
        B = size_of(b), S = size_of(s), K = size_of(k), N = size_of(n), R = size_of(r), NA = size_of(na);
    }
    // a new tensor of rows: those past the end of a sample are zero
    Tensor fresh(at::IntArrayRef shape) const {
        Tensor x = make(shape, t, dev);
        if (lens.defined()) x.zero_();
        return x;
    }
};

// lora_fwd(f32, x, A, U, scale, ids, y, lens, out, state)
PyObject *lora_fwd(PyObject *const *a) {
    const Adapters z(a[0], a[1], a[2], a[3], a[4], a[5], a[7]);
    const TokenRows x = token_rows(a[1], "x", z.dev, z.t, {z.b, z.s, z.k}, true, true);
    TokenRows y, out;
    if (given(a[6])) y = token_rows(a[6], "y", z.dev, z.t, {z.b, z.s, z.n}, a[6] != a[8], false);
    out = given(a[8]) ? token_rows(a[8], "out", z.dev, z.t, {z.b, z.s, z.n}, false, true)
                      : TokenRows(z.fresh({z.b, z.s, z.n}));
    const size_t need = lib.lora_state_bytes(z.B, z.S, z.R);
    Tensor state;
    if (given(a[9])) {
        state = tensor(a[9], "state", z.dev, at::kByte, at::kByte);
        if (!state.is_contiguous() || !aligned(state) || state.nbytes() < need)
            refuse(PyExc_ValueError, "state: %zu contiguous, 16-byte aligned bytes needed", need);
    } else {
        state = make({(int64_t)need}, at::kByte, z.dev);
    }
    const adaln_rows *yr = given(a[6]) ? &y.r : nullptr;
    const int32_t *lens = (const int32_t *)ptr(z.lens);
    const float *scale = (const float *)ptr(z.scale);
    if (z.t == at::kFloat)
        status("adaln_f32_lora_fwd",
               lib.f32_lora_fwd(&x.r, (const float *)ptr(z.A), (const float *)ptr(z.U), scale, ptr(z.ids), z.is64, lens,
                                yr, &out.r, ptr(state), need, z.B, z.S, z.K, z.N, z.R, z.NA, stream_of(z.dev)));
    else
        status("adaln_lora_fwd",
               lib.lora_fwd(&x.r, (const adaln_bf16 *)ptr(z.A), (const adaln_bf16 *)ptr(z.U), scale, ptr(z.ids), z.is64,
                            lens, yr, &out.r, ptr(state), need, z.B, z.S, z.K, z.N, z.R, z.NA, stream_of(z.dev)));
    return Py_BuildValue("(NN)", THPVariable_Wrap(out.x), THPVariable_Wrap(state));
}

// lora_bwd(f32, d_out, x, state, A, U, scale, ids, lens, dx_base, dx, dA_acc, dU_acc, accumulate, want_x, want_w,
//          workspace)
PyObject *lora_bwd(PyObject *const *a) {
    const Adapters z(a[0], a[2], a[4], a[5], a[6], a[7], a[8]);
    const bool accumulate = truth(a[13]), want_x = truth(a[14]), want_w = truth(a[15]);
    const TokenRows g = token_rows(a[1], "d_out", z.dev, z.t, {z.b, z.s, z.n}, true, true),
                    x = token_rows(a[2], "x", z.dev, z.t, {z.b, z.s, z.k}, true, true);
    const Tensor &state = tensor(a[3], "state", z.dev, at::kByte, at::kByte);
    if (!state.is_contiguous() || !aligned(state) || state.nbytes() < lib.lora_state_bytes(z.B, z.S, z.R))
        refuse(PyExc_ValueError, "state: not that of a forward of these sizes");
    TokenRows base, dx;
    if (given(a[9])) base = token_rows(a[9], "dx_base", z.dev, z.t, {z.b, z.s, z.k}, a[9] != a[10], false);
    if (given(a[10]))
        dx = token_rows(a[10], "dx", z.dev, z.t, {z.b, z.s, z.k}, false, true);
    else if (want_x)
        dx = TokenRows(z.fresh({z.b, z.s, z.k}));
    // given accumulators are filled; want_w allocates the missing ones
    Tensor dA, dU;
    if (want_w && accumulate && (!given(a[11]) || !given(a[12])))
        refuse(PyExc_ValueError, "accumulate: dA_acc and dU_acc must be given");
    if (want_w || given(a[11])) dA = result(a[11], "dA_acc", z.dev, at::kFloat, {z.na, z.r, z.k});
    if (want_w || given(a[12])) dU = result(a[12], "dU_acc", z.dev, at::kFloat, {z.na, z.r, z.n});
    const size_t need = z.t == at::kFloat ? lib.f32_lora_bwd_bytes(z.B, z.S, z.K, z.N, z.R)
                                          : lib.lora_bwd_bytes(z.B, z.S, z.K, z.N, z.R);
    const Tensor ws = scratch(a[16], need, z.dev);
    const adaln_rows *br = given(a[9]) ? &base.r : nullptr, *dr = dx.x.defined() ? &dx.r : nullptr;
    const int32_t *lens = (const int32_t *)ptr(z.lens);
    const float *scale = (const float *)ptr(z.scale);
    if (z.t == at::kFloat)
        status("adaln_f32_lora_bwd",
               lib.f32_lora_bwd(&g.r, &x.r, ptr(state), (const float *)ptr(z.A), (const float *)ptr(z.U), scale,
                                ptr(z.ids), z.is64, lens, br, dr, (float *)ptr(dA), (float *)ptr(dU), accumulate,
                                ptr(ws), need, z.B, z.S, z.K, z.N, z.R, z.NA, stream_of(z.dev)));
    else
        status("adaln_lora_bwd",
               lib.lora_bwd(&g.r, &x.r, ptr(state), (const adaln_bf16 *)ptr(z.A), (const adaln_bf16 *)ptr(z.U), scale,
                            ptr(z.ids), z.is64, lens, br, dr, (float *)ptr(dA), (float *)ptr(dU), accumulate, ptr(ws),
                            need, z.B, z.S, z.K, z.N, z.R, z.NA, stream_of(z.dev)));
    return Py_BuildValue("(NNN)", dx.x.defined() ? THPVariable_Wrap(dx.x) : Py_NewRef(Py_None),
                         dA.defined() ? THPVariable_Wrap(dA) : Py_NewRef(Py_None),
                         dU.defined() ? THPVariable_Wrap(dU) : Py_NewRef(Py_None));
}

// ---- module --------------------------------------------------------------------------

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments", N);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the 32 functions in the headers' order, raise_status)
constexpr int kBound = 32;
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != kBound + 1) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments", kBound + 1);
        return nullptr;
    }
    void *f[kBound];
    for (int i = 0; i < kBound; ++i) {
        f[i] = PyLong_AsVoidPtr(args[i]);
        if (!f[i]) return nullptr;
    }
    lib = Library{(decltype(lib.qk_fwd))f[0],         (decltype(lib.f32_qk_fwd))f[1],
                  (decltype(lib.qk_bwd_bytes))f[2],   (decltype(lib.qk_bwd))f[3],
                  (decltype(lib.f32_qk_bwd))f[4],     (decltype(lib.embed_fwd))f[5],
                  (decltype(lib.f32_embed_fwd))f[6],  (decltype(lib.embed_bwd_bytes))f[7],
                  (decltype(lib.embed_bwd))f[8],      (decltype(lib.f32_embed_bwd))f[9],
                  (decltype(lib.grad_bytes))f[10],    (decltype(lib.grad_norm))f[11],
                  (decltype(lib.grad_clip))f[12],
                  (decltype(lib.ckpt8_bytes))f[13],     (decltype(lib.ckpt8_pack))f[14],
                  (decltype(lib.f32_ckpt8_pack))f[15],  (decltype(lib.ckpt8_unpack))f[16],
                  (decltype(lib.f32_ckpt8_unpack))f[17], (decltype(lib.fwd_ckpt8))f[18],
                  (decltype(lib.f32_fwd_ckpt8))f[19],   (decltype(lib.bwd_ckpt8_bytes))f[20],
                  (decltype(lib.bwd_ckpt8))f[21],       (decltype(lib.f32_bwd_ckpt8))f[22],
                  (decltype(lib.again_ckpt8))f[23],     (decltype(lib.f32_again_ckpt8))f[24],
                  (decltype(lib.lora_state_bytes))f[25], (decltype(lib.lora_fwd))f[26],
                  (decltype(lib.f32_lora_fwd))f[27],    (decltype(lib.lora_bwd_bytes))f[28],
                  (decltype(lib.f32_lora_bwd_bytes))f[29], (decltype(lib.lora_bwd))f[30],
                  (decltype(lib.f32_lora_bwd))f[31]};
    Py_XSETREF(raise_status, Py_NewRef(args[kBound]));
    Py_RETURN_NONE;
}

#define CALL(f, n) {#f, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(qk_fwd, 12),
                         CALL(qk_bwd, 19),
                         CALL(embed_fwd, 5),
                         CALL(embed_bwd, 9),
                         CALL(grad_workspace_bytes, 1),
                         CALL(grad_norm, 3),
                         CALL(grad_clip, 5),
                         CALL(ckpt8_pack, 3),
                         CALL(ckpt8_unpack, 4),
                         CALL(out_fwd_ckpt8, 8),
                         CALL(out_bwd_ckpt8, 9),
                         CALL(out_again_ckpt8, 6),
                         CALL(lora_fwd, 10),
                         CALL(lora_bwd, 17),
                         {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "adaln_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_adaln_marshal() { return PyModule_Create(&module); }
