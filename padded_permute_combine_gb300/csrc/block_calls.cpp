// The block operators' calls from Python, without ctypes: checks of the
// tensors, outputs and workspace, and the C ABI call, for the plain case of
// every one (tensors that are right, outputs to be allocated). Anything else
// returns None, and block.py takes the call step by step, with its messages;
// a call that failed once work may have been enqueued raises MoeError here.
//
// A call of these operators on a few rows runs for 3 to 14 us on the GPU. On the
// host the whole call takes 5.1 to 7.4 us (it varies from process to process) for
// a layer norm forward of four rows, 8.1 to 10.7 backward, 14 to 16.2 for an MoE
// layer of one token, some 2.2 for each launch and the rest for three to five
// allocations; in Python the same steps took 14, 22 and 29.
#include "calls.h"
#include "moe_block.h"

namespace {

using namespace moe_calls;

// x, weight, bias, eps -> (y, mean, rstd)
PyObject* layer_norm_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[3];
    int64_t stride;
    if (n != 4 || !tensors(args, 3, t, 6) || !PyFloat_Check(args[3]) || !rows_ok(t[0], &stride)) return nullptr;
    const Tensor &x = t[0], &w = t[1], &b = t[2];
    const CUDAGuard current(x.device());
    const int64_t M = x.size(0), H = x.size(1);
    const float eps = (float)PyFloat_AS_DOUBLE(args[3]);
    const at::ScalarType wt = w.defined() ? w.scalar_type() : b.defined() ? b.scalar_type() : at::kFloat;
    if ((wt != at::kFloat && wt != at::kBFloat16) || (w.defined() && !plain(w, x, wt, {H})) || (b.defined() && !plain(b, x, wt, {H})))
      return nullptr;
    const Tensor y = make(x, x.scalar_type(), {M, H}), mean = make(x, at::kFloat, {M}), rstd = make(x, at::kFloat, {M});
    const int rc = unlocked([&] {
      return moe_layer_norm_fwd(x.const_data_ptr(), dtype_of(x), stride, at_or_null(w), at_or_null(b),
                                wt == at::kFloat ? MOE_F32 : MOE_BF16, M, H, eps, y.data_ptr(), mean.data_ptr<float>(),
                                rstd.data_ptr<float>(), stream_of(x));
    });
    return rc == MOE_OK ? wrapped({y, mean, rstd}) : failed("moe_layer_norm_fwd", rc);
  });
}

// dy, x, weight, mean, rstd, need_cols -> (dx, dweight, dbias)
PyObject* layer_norm_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[5];
    int64_t stride, dy_stride;
    if (n != 6 || !tensors(args, 5, t, 4) || !rows_ok(t[1], &stride) || !rows_ok(t[0], &dy_stride)) return nullptr;
    const Tensor &dy = t[0], &x = t[1], &w = t[2], &mean = t[3], &rstd = t[4];
    const CUDAGuard current(x.device());
    const int64_t M = x.size(0), H = x.size(1);
    const at::ScalarType wt = w.defined() ? w.scalar_type() : at::kFloat;
    if (dy.scalar_type() != x.scalar_type() || dy.device() != x.device() || dy.sizes() != x.sizes() || !plain(mean, x, at::kFloat, {M}) ||
        !plain(rstd, x, at::kFloat, {M}) || (wt != at::kFloat && wt != at::kBFloat16) || (w.defined() && !plain(w, x, wt, {H})))
      return nullptr;
    const Tensor dx = make(x, x.scalar_type(), {M, H});
    Tensor dw, db, ws;
    size_t bytes = 0;
    if (args[5] == Py_True) {
      bytes = moe_layer_norm_bwd_workspace_size(M, H);
      dw = make(x, wt, {H});
      db = make(x, wt, {H});
      ws = make(x, at::kByte, {(int64_t)bytes});
    }
    const int rc = unlocked([&] {
      return moe_layer_norm_bwd(dy.const_data_ptr(), dy_stride, x.const_data_ptr(), dtype_of(x), stride, at_or_null(w),
                                wt == at::kFloat ? MOE_F32 : MOE_BF16, mean.const_data_ptr<float>(), rstd.const_data_ptr<float>(), M, H,
                                dx.data_ptr(), dw.defined() ? dw.data_ptr() : nullptr, db.defined() ? db.data_ptr() : nullptr,
                                ws.defined() ? ws.data_ptr() : nullptr, bytes, stream_of(x));
    });
    return rc == MOE_OK ? wrapped({dx, dw, db}) : failed("moe_layer_norm_bwd", rc);
  });
}

// The experts' matrices: [E, 2F, H] and [E, H, F] beside x [T, H].
bool experts_ok(const Tensor& x, const Tensor& gate_up, const Tensor& down, int64_t* E, int64_t* F) {
  if (down.dim() != 3 || down.size(1) != x.size(1)) return false;
  *E = down.size(0);
  *F = down.size(2);
  return *E <= INT32_MAX && plain(down, x, x.scalar_type(), {*E, x.size(1), *F}) &&
         plain(gate_up, x, x.scalar_type(), {*E, 2 * *F, x.size(1)});
}

// x, router, w_gate_up, w_down, top_k, mode, normalize -> (y, top_expert, weights)
PyObject* layer(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[4];
    int64_t stride, E, F;
    if (n != 7 || !tensors(args, 4, t) || !PyLong_Check(args[4]) || !rows_ok(t[0], &stride)) return nullptr;
    const Tensor &x = t[0], &router = t[1], &gate_up = t[2], &down = t[3];
    const CUDAGuard current(x.device());
    const int64_t T = x.size(0), H = x.size(1), K = PyLong_AsLongLong(args[4]);
    if (!experts_ok(x, gate_up, down, &E, &F) || !plain(router, x, x.scalar_type(), {E, H}) || K < 1 || K > E) return nullptr;
    const int32_t mode = (int32_t)PyLong_AsLong(args[5]), normalize = PyObject_IsTrue(args[6]);
    const size_t bytes = moe_layer_workspace_size(T, H, F, (int32_t)E, (int32_t)K);
    if (bytes == 0) return nullptr;
    const Tensor y = make(x, x.scalar_type(), {T, H}), top = make(x, at::kInt, {T, K}), w = make(x, at::kFloat, {T, K}),
                 ws = make(x, at::kByte, {(int64_t)bytes});
    const int rc = unlocked([&] {
      return moe_layer(x.const_data_ptr(), dtype_of(x), stride, router.const_data_ptr(), gate_up.const_data_ptr(), down.const_data_ptr(), T,
                       H, F, (int32_t)E, (int32_t)K, mode, normalize, top.data_ptr<int32_t>(), w.data_ptr<float>(), y.data_ptr(),
                       ws.data_ptr(), bytes, nullptr, stream_of(x));
    });
    return rc == MOE_OK ? wrapped({y, top, w}) : failed("moe_layer", rc);
  });
}

// x, top_expert, weights, w_gate_up, w_down -> (y,)
PyObject* experts(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[5];
    int64_t stride, E, F;
    if (n != 5 || !tensors(args, 5, t) || !rows_ok(t[0], &stride)) return nullptr;
    const Tensor &x = t[0], &top = t[1], &w = t[2], &gate_up = t[3], &down = t[4];
    const CUDAGuard current(x.device());
    if (top.dim() != 2) return nullptr;
    const int64_t T = x.size(0), H = x.size(1), K = top.size(1);
    if (!experts_ok(x, gate_up, down, &E, &F) || !plain(top, x, at::kInt, {T, K}) || !plain(w, x, at::kFloat, {T, K}) || K < 1 || K > E)
      return nullptr;
    const size_t bytes = moe_layer_workspace_size(T, H, F, (int32_t)E, (int32_t)K);
    if (bytes == 0) return nullptr;
    const Tensor y = make(x, x.scalar_type(), {T, H}), ws = make(x, at::kByte, {(int64_t)bytes});
    const int rc = unlocked([&] {
      return moe_experts(x.const_data_ptr(), dtype_of(x), stride, top.const_data_ptr<int32_t>(), w.const_data_ptr<float>(),
                         gate_up.const_data_ptr(), down.const_data_ptr(), T, H, F, (int32_t)E, (int32_t)K, y.data_ptr(), ws.data_ptr(),
                         bytes, nullptr, stream_of(x));
    });
    return rc == MOE_OK ? wrapped({y}) : failed("moe_experts", rc);
  });
}

// A set's table, pieces and workspace (and max_norm) -> (norm,)
PyObject* grads(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[2];
    if ((n != 3 && n != 4) || !tensors(args, 2, t) || !PyLong_Check(args[2]) || (n == 4 && !PyFloat_Check(args[3]))) return nullptr;
    const Tensor &table = t[0], &ws = t[1];
    if (!table.is_cuda()) return nullptr;
    const CUDAGuard current(table.device());
    const int64_t pieces = PyLong_AsLongLong(args[2]);
    const Tensor norm = make(table, at::kFloat, {});
    const auto* p = static_cast<const moe_grad_piece*>(table.const_data_ptr());
    const float max_norm = n == 3 ? 0.0f : (float)PyFloat_AS_DOUBLE(args[3]);
    const int rc = unlocked([&] {
      return n == 3 ? moe_grad_norm(p, pieces, norm.data_ptr<float>(), ws.data_ptr(), ws.numel(), stream_of(table))
                    : moe_clip_grads(p, pieces, max_norm, norm.data_ptr<float>(), ws.data_ptr(), ws.numel(), stream_of(table));
    });
    return rc == MOE_OK ? wrapped({norm}) : failed(n == 3 ? "moe_grad_norm" : "moe_clip_grads", rc);
  });
}

PyMethodDef methods[] = {CALL(layer_norm_fwd), CALL(layer_norm_bwd), CALL(layer), CALL(experts), CALL(grads),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__block_calls() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddFunctions(m, moe_calls::decode_methods()) != 0) Py_CLEAR(m);
  return m;
}
