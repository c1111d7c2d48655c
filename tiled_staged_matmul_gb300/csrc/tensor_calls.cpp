// tensor_calls.cpp -- torch tensors to the pointers and sizes of the C ABI
// (include/tsm_gemm.h), for the calls whose work on the GPU is so short that the
// host's share counts: the choice of experts and the 4-bit operators.  A Python
// extension module; binding.py holds the calls' signatures and documentation and
// passes their arguments on, in order.
//
// Checks of types and shapes, outputs and the stream, nothing else: what the
// library checks itself (pointers, spans, alignment, sizes) is left to it.  (From
// Python, through ctypes, a decode step's calls took three to four times as long: one
// token's product 14.4 us of host time, 3.4 so; quantising 18.2, 5.4; the choice 15.2,
// 4.2; its gradient 13.6, 3.4.)
//
// A function returns its results, or the library's status where that is not
// GEMM_OK, for the caller to raise.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/tsm_gemm.h"

namespace {

// An argument that is not what it has to be.
struct Refused : std::exception {
    PyObject *type;
    std::string text;
    Refused(PyObject *type_, std::string text_) : type(type_), text(std::move(text_)) {}
};
[[noreturn]] void refuse(const std::string &text) { throw Refused(PyExc_ValueError, text); }
[[noreturn]] void refuse_type(const std::string &text) { throw Refused(PyExc_TypeError, text); }

template <typename F>
PyObject *guarded(F &&fn)
{
    HANDLE_TH_ERRORS
    try {
        return fn();
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        refuse_type(std::string(name) + " must be a torch tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}

int32_t integer32(PyObject *o)
{
    const int64_t v = integer(o);
    if (v != int32_t(v))
        refuse(std::to_string(v) + " does not fit 32 bits");
    return int32_t(v);
}

float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return float(v);
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();
    return v != 0;
}

int32_t elem_type(const at::Tensor &t)
{
    switch (t.scalar_type()) {
    case at::kFloat: return GEMM_OUT_F32;
    case at::kHalf: return GEMM_OUT_F16;
    case at::kBFloat16: return GEMM_OUT_BF16;
    default: refuse_type("rows must be torch.float32, torch.float16 or torch.bfloat16");
    }
}

gemm_stream_t stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// The library's call without the interpreter's lock (a full launch queue can hold
// it up), and its status.  The lock is back before an exception (of a tensor whose
// address may not be taken, say) goes on.
template <typename F>
gemm_status_t call(F &&fn)
{
    struct Unlocked {
        PyThreadState *state = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(state); }
    } unlocked;
    return fn();
}

std::string sizes(at::IntArrayRef s)
{
    std::string text;
    for (size_t i = 0; i < s.size(); ++i)
        text += (i ? " x " : "") + std::to_string(s[i]);
    return text;
}

// A new tensor beside another (dense, or with these strides), without the way
// through the dispatcher that at::empty takes (three of them: quantising 8.3 us of
// host time so, 5.4 without).
at::Tensor fresh(const at::Tensor &like, at::IntArrayRef shape, at::ScalarType type)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
at::Tensor fresh(const at::Tensor &like, at::IntArrayRef shape, at::IntArrayRef strides, at::ScalarType type)
{
    return at::Tensor(at::detail::empty_strided_cuda(shape, strides, type, like.device()));
}

// The row pitch of a matrix of rows with a unit last stride.
int64_t pitch(const at::Tensor &t, const char *name)
{
    if (!t.is_cuda())
        refuse(std::string(name) + " must be a CUDA tensor");
    if (t.size(1) > 1 && t.numel() && t.stride(1) != 1)
        refuse(std::string(name) + " must have a unit last stride");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// A contiguous CUDA tensor of one type and shape.
const at::Tensor &dense(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape, const char *name)
{
    if (t.scalar_type() != type || !t.is_cuda() || t.sizes() != shape || !t.is_contiguous())
        refuse(std::string(name) + " must be a contiguous CUDA tensor of " + sizes(shape) + " " + c10::toString(type) + " values");
    return t;
}

// One count per matrix, or none.
const int32_t *counts_of(PyObject *o, int64_t batch)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = tensor(o, "group_rows");
    if (t.scalar_type() != at::kInt || !t.is_cuda() || t.numel() != batch || !t.is_contiguous())
        refuse("group_rows must be a contiguous CUDA int32 tensor of one count per matrix");
    return static_cast<const int32_t *>(t.data_ptr());
}

void want(Py_ssize_t n, Py_ssize_t count)
{
    if (n != count)
        refuse_type("wrong number of arguments");
}

// ------------------------------------------------------------- choice of experts

// (logits, topk, score, bias, groups, keep_groups, group_best, renormalize, scale)
PyObject *moe_choose(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        want(n, 9);
        const at::Tensor &x = tensor(a[0], "logits");
        const int32_t type = elem_type(x);
        if (x.dim() != 2)
            refuse("logits must be a tokens x experts tensor");
        const int64_t T = x.size(0), E = x.size(1), topk = integer(a[1]), ld = pitch(x, "logits");
        const float *bias = nullptr;
        if (a[3] != Py_None)
            bias = static_cast<const float *>(dense(tensor(a[3], "bias"), at::kFloat, {E}, "bias").data_ptr());
        const int64_t groups = integer(a[4]), keep = integer(a[5]);
        const int32_t score = integer32(a[2]), best = integer32(a[6]);
        const bool renormalize = truth(a[7]);
        const float scale = real(a[8]);
        if (topk < 0)
            refuse("topk must not be negative");
        const at::Tensor ids = fresh(x, {T, topk}, at::kInt), weights = fresh(x, {T, topk}, at::kFloat);
        const gemm_status_t st = call([&] {
            return choose_experts(x.data_ptr(), type, bias, static_cast<int32_t *>(ids.data_ptr()),
                                  static_cast<float *>(weights.data_ptr()), T, E, topk, ld, score, groups, keep, best,
                                  renormalize, scale, stream());
        });
        if (st != GEMM_OK)
            return PyLong_FromLong(st);
        PyObject *pair = PyTuple_New(2);
        PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(ids));
        PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(weights));
        return pair;
    });
}

// (dweights, logits, ids, out, score, renormalize, scale)
PyObject *moe_choose_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        want(n, 7);
        const at::Tensor &dw = tensor(a[0], "dweights"), &x = tensor(a[1], "logits"), &ids = tensor(a[2], "ids");
        const int32_t type = elem_type(x);
        if (x.dim() != 2)
            refuse("logits must be a tokens x experts tensor");
        const int64_t T = x.size(0), E = x.size(1), ld = pitch(x, "logits");
        if (ids.dim() != 2)
            refuse("ids must be a tokens x topk tensor");
        const int64_t topk = ids.size(1);
        dense(ids, at::kInt, {T, topk}, "ids");
        dense(dw, at::kFloat, {T, topk}, "dweights");
        at::Tensor out;
        int64_t ldo = E;
        if (a[3] == Py_None) {
            out = fresh(x, {T, E}, x.scalar_type());
        } else {
            out = tensor(a[3], "out");
            if (out.dim() != 2 || out.sizes() != x.sizes() || out.scalar_type() != x.scalar_type())
                refuse("out must be a tensor of the logits' shape and type");
            ldo = pitch(out, "out");
        }
        const int32_t score = integer32(a[4]);
        const bool renormalize = truth(a[5]);
        const float scale = real(a[6]);
        const gemm_status_t st = call([&] {
            return choose_experts_grad(static_cast<const float *>(dw.data_ptr()), x.data_ptr(), type,
                                       static_cast<const int32_t *>(ids.data_ptr()), out.data_ptr(), T, E, topk, ld, ldo,
                                       score, renormalize, scale, stream());
        });
        if (st != GEMM_OK)
            return PyLong_FromLong(st);
        return THPVariable_Wrap(out);
    });
}

// ------------------------------------------------------------- 4-bit rows

// (X, group_rows, block): codes, block scales and row scales (or None)
PyObject *quantize_fp4(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        want(n, 3);
        const at::Tensor &x = tensor(a[0], "X");
        const int32_t type = elem_type(x);
        const int64_t block = integer(a[2]);
        if (block != 16 && block != 32)
            refuse("block must be 16 or 32");
        const int64_t dim = x.dim();
        const bool three = dim == 3;
        if ((dim != 2 && dim != 3) || !x.is_cuda() || (x.size(-1) > 1 && x.numel() && x.stride(-1) != 1))
            refuse("X must be a 2-D or 3-D CUDA tensor with a unit last stride");
        const int64_t batch = three ? x.size(0) : 1, M = x.size(-2), K = x.size(-1);
        const int64_t sX = three ? x.stride(0) : 0, ldx = M > 1 ? x.stride(-2) : K;
        const int32_t *counts = counts_of(a[1], batch);
        const int64_t width = (K + 1) / 2, ldq = (width + 15) / 16 * 16, sQ = M * ldq;
        const int64_t rows = (M + 127) / 128, cols = (K + 4 * block - 1) / (4 * block);
        const at::Tensor q = three ? fresh(x, {batch, M, width}, {sQ, ldq, 1}, at::kByte) : fresh(x, {M, width}, {ldq, 1}, at::kByte);
        const at::Tensor s = three ? fresh(x, {batch, rows, cols, 512}, at::kByte) : fresh(x, {rows, cols, 512}, at::kByte);
        at::Tensor r;
        if (block == 16)
            r = three ? fresh(x, {batch, M}, at::kFloat) : fresh(x, {M}, at::kFloat);
        const gemm_status_t st = call([&] {
            return fp4_quantize_rows(x.data_ptr(), type, int32_t(block), static_cast<uint8_t *>(q.data_ptr()),
                                     static_cast<uint8_t *>(s.data_ptr()), r.defined() ? static_cast<float *>(r.data_ptr()) : nullptr,
                                     counts, M, K, ldx, ldq, sX, sQ, M, batch, stream());
        });
        if (st != GEMM_OK)
            return PyLong_FromLong(st);
        PyObject *all = PyTuple_New(3);
        PyTuple_SET_ITEM(all, 0, THPVariable_Wrap(q));
        PyTuple_SET_ITEM(all, 1, THPVariable_Wrap(s));
        PyTuple_SET_ITEM(all, 2, r.defined() ? THPVariable_Wrap(r) : Py_NewRef(Py_None));
        return all;
    });
}

// One operand of a product.
struct Rows {
    const at::Tensor &codes, &tiles;
    int64_t batch, rows, width, ld, stride;

    Rows(PyObject *codes_, PyObject *tiles_, int64_t block, const std::string &name)
        : codes(tensor(codes_, "codes")), tiles(tensor(tiles_, "block scales"))
    {
        if (codes.scalar_type() != at::kByte || tiles.scalar_type() != at::kByte)
            refuse_type(name + "'s codes and block scales must be torch.uint8");
        const int64_t dim = codes.dim();
        if (dim != 2 && dim != 3)
            refuse(name + "'s codes must be 2-D or 3-D");
        batch = dim == 3 ? codes.size(0) : -1;
        rows = codes.size(-2);
        width = codes.size(-1);
        if (!codes.is_cuda() || (width > 1 && codes.numel() && codes.stride(-1) != 1))
            refuse(name + "'s codes must be a CUDA tensor with a unit last stride");
        ld = rows > 1 ? codes.stride(-2) : std::max<int64_t>(width, 1);
        stride = dim == 3 ? codes.stride(0) : 0;
        const int64_t shape[4] = {batch, (rows + 127) / 128, (width + 2 * block - 1) / (2 * block), 512};
        const at::IntArrayRef wanted(shape + (dim == 2), shape + 4);
        if (tiles.sizes() != wanted || !tiles.is_cuda() || !tiles.is_contiguous())
            refuse(name + "'s block scales must be a contiguous " + sizes(wanted) + " CUDA tensor");
    }
    const uint8_t *code_ptr() const { return static_cast<const uint8_t *>(codes.data_ptr()); }
    const uint8_t *tile_ptr() const { return static_cast<const uint8_t *>(tiles.data_ptr()); }
};

// A vector of n values, or (batch >= 0) one per matrix.
struct Vector {
    const float *at = nullptr;
    int64_t stride = 0;

    Vector(PyObject *o, int64_t n, int64_t batch, const char *name)
    {
        if (o == Py_None)
            return;
        const at::Tensor &t = tensor(o, name);
        const int64_t dim = t.dim();
        if (t.scalar_type() != at::kFloat || !t.is_cuda() || dim < 1 || dim > (batch >= 0 ? 2 : 1) || t.size(-1) != n ||
            (n > 1 && t.stride(-1) != 1) || (dim == 2 && t.size(0) != batch))
            refuse(std::string(name) + " must be a CUDA float32 tensor of " + std::to_string(n) + " values" +
                   (batch >= 0 ? " (or " + std::to_string(batch) + " x " + std::to_string(n) + ")" : ""));
        at = static_cast<const float *>(t.data_ptr());
        if (dim == 2 && batch > 1)
            stride = t.stride(0);
    }
};

// (codes, block scales, scales of a, the same of b, block, group_rows, out, alpha, bias, activation, slope, out_dtype)
PyObject *gemm_fp4(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        want(n, 14);
        const int64_t block = integer(p[6]);
        if (block != 16 && block != 32)
            refuse("blocks must be 16 or 32");
        const Rows a(p[0], p[1], block, "a"), b(p[3], p[4], block, "b");
        if (a.batch != b.batch)
            refuse("batch sizes differ");
        if (a.width != b.width)
            refuse("inner sizes differ: " + std::to_string(2 * a.width) + " vs " + std::to_string(2 * b.width));
        const bool three = a.batch >= 0;
        const int64_t batch = three ? a.batch : 1, M = a.rows, N = b.rows;
        const int32_t *counts = counts_of(p[7], batch);
        const int64_t shape[3] = {batch, M, N};
        const at::IntArrayRef wanted(shape + !three, shape + 3);
        at::Tensor out;
        if (p[8] == Py_None) {
            at::ScalarType type = at::kFloat;
            if (p[13] != Py_None) {
                if (!THPDtype_Check(p[13]))
                    refuse_type("out_dtype must be a torch dtype");
                type = reinterpret_cast<THPDtype *>(p[13])->scalar_type;
            }
            out = counts ? at::zeros(wanted, at::TensorOptions().device(a.codes.device()).dtype(type)) : fresh(a.codes, wanted, type);
        } else {
            out = tensor(p[8], "out");
        }
        if (out.sizes() != wanted)
            refuse("out must be a " + sizes(wanted) + " tensor");
        if (!out.is_cuda() || (N > 1 && out.numel() && out.stride(-1) != 1))
            refuse("out must be a CUDA tensor with a unit last stride");
        const Vector sa(p[2], M, a.batch, "a.scales"), sb(p[5], N, a.batch, "b.scales"), bias(p[10], N, a.batch, "bias");
        gemm_epilogue_t epi = {};
        epi.alpha = real(p[9]);
        epi.bias = bias.at;
        epi.bias_stride = bias.stride;
        epi.activation = integer32(p[11]);
        epi.slope = real(p[12]);
        epi.out_type = elem_type(out);
        const int64_t ldc = M > 1 ? out.stride(-2) : std::max<int64_t>(N, 1), sC = three ? out.stride(0) : 0;
        const gemm_status_t st = call([&] {
            return counts ? gemm_fp4_grouped_scaled(a.code_ptr(), b.code_ptr(), out.data_ptr(), a.tile_ptr(), b.tile_ptr(), sa.at,
                                                    sb.at, int32_t(block), counts, batch, M, N, 2 * a.width, a.ld, b.ld, ldc,
                                                    a.stride, b.stride, sC, sa.stride, sb.stride, &epi, stream())
                          : gemm_fp4_scaled(a.code_ptr(), b.code_ptr(), out.data_ptr(), a.tile_ptr(), b.tile_ptr(), sa.at, sb.at,
                                            int32_t(block), M, N, 2 * a.width, a.ld, b.ld, ldc, a.stride, b.stride, sC, sa.stride,
                                            sb.stride, batch, &epi, stream());
        });
        if (st != GEMM_OK)
            return PyLong_FromLong(st);
        return p[8] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(p[8]);
    });
}

PyMethodDef methods[] = {
    {"moe_choose", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(moe_choose)), METH_FASTCALL, nullptr},
    {"moe_choose_grad", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(moe_choose_grad)), METH_FASTCALL, nullptr},
    {"quantize_fp4", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(quantize_fp4)), METH_FASTCALL, nullptr},
    {"gemm_fp4", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(gemm_fp4)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "tsm_tensor_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tsm_tensor_calls()
{
    return PyModule_Create(&module);
}
