// The decode operators' calls from Python, as block_calls.cpp has them for the
// block's: the plain case of every one is checked, given its outputs and
// workspace, and called; anything else returns None, and decode.py takes the
// call step by step, with its messages.
#include <algorithm>
#include <array>

#include "calls.h"
#include "moe_decode.h"

namespace moe_calls {
namespace {

bool ints(PyObject* const* args, int n, int64_t* out) {
  for (int i = 0; i < n; ++i) {
    if (!PyLong_Check(args[i])) return false;
    out[i] = PyLong_AsLongLong(args[i]);
    if (out[i] == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return false;
    }
  }
  return true;
}
bool fits32(int64_t v) { return v >= INT32_MIN && v <= INT32_MAX; }
bool on(const Tensor& t, at::ScalarType type, int64_t dims, c10::Device device) {
  return t.defined() && t.is_cuda() && t.device() == device && t.scalar_type() == type && t.dim() == dims;
}
bool ints_of(const Tensor& t, c10::Device device, at::IntArrayRef sizes) {
  return on(t, at::kInt, (int64_t)sizes.size(), device) && t.is_contiguous() && t.sizes() == sizes;
}

// Several small outputs as parts of one allocation (an allocation costs the
// host 0.7 us or more, a part 0.2): each on 16 bytes, contiguous.
template <int N> void parts_of(const Tensor& like, const at::ScalarType (&types)[N], const std::initializer_list<int64_t> (&sizes)[N], Tensor (&out)[N]) {
  int64_t bytes = 0, at[N];
  for (int i = 0; i < N; ++i) {
    int64_t n = (int64_t)c10::elementSize(types[i]);
    for (const int64_t d : sizes[i]) n *= d;
    at[i] = bytes;
    bytes += (n + 15) / 16 * 16;
  }
  const Tensor whole = make(like, at::kByte, {bytes});
  for (int i = 0; i < N; ++i) {
    out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                      c10::scalarTypeToTypeMeta(types[i]));
    c10::TensorImpl* impl = out[i].unsafeGetTensorImpl();
    impl->set_storage_offset(at[i] / (int64_t)c10::elementSize(types[i]));
    impl->set_sizes_contiguous(sizes[i]);
  }
}

// The stride of dimension i, 0 where it has one element.
int64_t step(const Tensor& t, int64_t i) { return t.size(i) <= 1 ? 0 : t.stride(i); }

// Keys and values [pages, page_size, kv_heads, head_dim], alike, none overlapping itself.
bool cache_of(const Tensor& k, const Tensor& v, moe_kv_cache* c) {
  if (!k.is_cuda() || dtype_of(k) < 0 || k.dim() != 4 || !on(v, k.scalar_type(), 4, k.device()) || v.sizes() != k.sizes()) return false;
  std::array<std::pair<int64_t, int64_t>, 3> dims;
  for (int i = 0; i < 3; ++i) {
    dims[i] = {step(k, i), k.size(i)};
    if (step(v, i) != dims[i].first) return false;
  }
  if (k.size(3) > 1 && (k.stride(3) != 1 || v.stride(3) != 1)) return false;
  for (int i = 1; i < 4; ++i)
    if (!fits32(k.size(i))) return false;
  *c = {k.data_ptr(), v.data_ptr(), k.size(0), dims[0].first, dims[1].first, dims[2].first, dtype_of(k), (int32_t)k.size(1),
        (int32_t)k.size(2), (int32_t)k.size(3)};
  if (k.numel() == 0) return true;
  std::sort(dims.begin(), dims.end());
  int64_t reach = k.size(3);
  for (const auto& [stride, n] : dims) {
    if (n <= 1) continue;
    if (stride < reach) return false;
    reach += stride * (n - 1);
  }
  return true;
}
bool heads_of(const Tensor& t, const Tensor& like, int64_t rows, int64_t heads, moe_heads* h) {
  if (!on(t, like.scalar_type(), 3, like.device()) || t.size(0) != rows || t.size(1) != heads || t.size(2) != like.size(3)) return false;
  if (t.size(2) > 1 && t.stride(2) != 1) return false;
  *h = {t.const_data_ptr(), step(t, 0), step(t, 1)};
  return true;
}
// A table of rows that do not overlap, with the rows' lengths.
bool table_of(const Tensor& table, const Tensor& lengths, c10::Device device, int64_t* stride) {
  if (!on(table, at::kInt, 2, device) || !ints_of(lengths, device, {table.size(0)})) return false;
  *stride = step(table, 0);
  return (table.size(1) <= 1 || table.stride(1) == 1) && (table.size(0) <= 1 || *stride >= table.size(1));
}

// q, k_cache, v_cache, page_table, lengths, k_new, v_new, scale, window -> (out, lse)
PyObject* attention_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[7];
    int64_t window, stride;
    if (n != 9 || !tensors(args, 7, t, 0x60) || !ints(args + 8, 1, &window) || (args[7] != Py_None && !PyFloat_Check(args[7]))) return nullptr;
    const Tensor &q = t[0], &k = t[1], &table = t[3], &lengths = t[4];
    moe_kv_cache cache;
    moe_heads qs, kn, vn;
    if (!cache_of(k, t[2], &cache) || q.dim() != 3) return nullptr;
    const int64_t B = q.size(0), H = q.size(1), D = q.size(2);
    const bool fresh = t[5].defined();
    if (fresh != t[6].defined() || !fits32(H) || !heads_of(q, k, B, H, &qs) || !table_of(table, lengths, k.device(), &stride) || table.size(0) != B ||
        (fresh && !(heads_of(t[5], k, B, k.size(2), &kn) && heads_of(t[6], k, B, k.size(2), &vn))) || D < 1)
      return nullptr;
    const c10::cuda::CUDAGuard current(k.device());
    const size_t bytes = moe_attention_decode_workspace_size(B, (int32_t)H, cache.num_kv_heads, (int32_t)D);
    if (bytes == 0) return nullptr;
    Tensor o[2];
    parts_of(k, {k.scalar_type(), at::kFloat}, {{B, H, D}, {B, H}}, o);
    const Tensor &out = o[0], &lse = o[1], ws = make(k, at::kByte, {(int64_t)bytes});
    const float scale = args[7] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)PyFloat_AS_DOUBLE(args[7]);
    const int rc = unlocked([&] {
      return moe_attention_decode(&cache, &qs, (int32_t)H, table.const_data_ptr<int32_t>(), stride, table.size(1), lengths.const_data_ptr<int32_t>(), B,
                                  fresh ? &kn : nullptr, fresh ? &vn : nullptr, scale, window, out.data_ptr(), lse.data_ptr<float>(), ws.data_ptr(),
                                  bytes, nullptr, stream_of(k));
    });
    return rc == MOE_OK ? wrapped({out, lse}) : failed("moe_attention_decode", rc);
  });
}

// k, v, k_cache, v_cache, page_table, offsets, lengths -> ()
PyObject* cache_write(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[7];
    int64_t stride;
    moe_kv_cache cache;
    moe_heads k, v;
    if (n != 7 || !tensors(args, 7, t) || !cache_of(t[2], t[3], &cache) || t[0].dim() != 3) return nullptr;
    const Tensor &table = t[4], &offsets = t[5], &lengths = t[6];
    const int64_t T = t[0].size(0);
    if (!heads_of(t[0], t[2], T, t[2].size(2), &k) || !heads_of(t[1], t[2], T, t[2].size(2), &v) || !table_of(table, lengths, t[2].device(), &stride) ||
        !ints_of(offsets, t[2].device(), {table.size(0) + 1}))
      return nullptr;
    const c10::cuda::CUDAGuard current(t[2].device());
    const int rc = unlocked([&] {
      return moe_cache_write(&cache, &k, &v, T, offsets.const_data_ptr<int32_t>(), table.const_data_ptr<int32_t>(), stride, table.size(1),
                             lengths.const_data_ptr<int32_t>(), table.size(0), nullptr, stream_of(t[2]));
    });
    return rc == MOE_OK ? wrapped({}) : failed("moe_cache_write", rc);
  });
}

// page_table, lengths, parents, page_size, num_pages, grow, width -> (page_table, lengths, src, dst)
PyObject* cache_fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[3];
    int64_t v[4], stride;
    const bool same = n == 7 && args[6] == Py_None;
    if (n != 7 || !tensors(args, 3, t) || !ints(args + 3, same ? 3 : 4, v) || !fits32(v[0]) || !t[0].is_cuda()) return nullptr;
    const Tensor &table = t[0], &lengths = t[1], &parents = t[2];
    if (same) v[3] = table.dim() == 2 ? table.size(1) : -1;
    if (!table_of(table, lengths, table.device(), &stride) || parents.dim() != 1 || !ints_of(parents, table.device(), {parents.size(0)}) || v[3] < 0)
      return nullptr;
    const c10::cuda::CUDAGuard current(table.device());
    const int64_t R = parents.size(0);
    Tensor o[4];
    parts_of(table, {at::kInt, at::kInt, at::kInt, at::kInt}, {{R, v[3]}, {R}, {R}, {R}}, o);
    const Tensor &next = o[0], &len = o[1], &src = o[2], &dst = o[3];
    const int rc = unlocked([&] {
      return moe_cache_fork(table.const_data_ptr<int32_t>(), stride, table.size(1), lengths.const_data_ptr<int32_t>(), table.size(0),
                            parents.const_data_ptr<int32_t>(), R, (int32_t)v[0], v[1], v[2], next.data_ptr<int32_t>(), v[3], len.data_ptr<int32_t>(),
                            src.data_ptr<int32_t>(), dst.data_ptr<int32_t>(), nullptr, stream_of(table));
    });
    return rc == MOE_OK ? wrapped({next, len, src, dst}) : failed("moe_cache_fork", rc);
  });
}

// page_table, lengths, page_size, num_pages -> (page_table, src, dst, count)
PyObject* cache_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[2];
    int64_t v[2], stride;
    if (n != 4 || !tensors(args, 2, t) || !ints(args + 2, 2, v) || !fits32(v[0]) || v[1] < 0 || !t[0].is_cuda()) return nullptr;
    const Tensor &table = t[0], &lengths = t[1];
    if (!table_of(table, lengths, table.device(), &stride) || v[1] > MOE_CACHE_MAX_PAGES) return nullptr;
    const c10::cuda::CUDAGuard current(table.device());
    Tensor o[4];
    parts_of(table, {at::kInt, at::kInt, at::kInt, at::kInt}, {{table.size(0), table.size(1)}, {v[1] / 2}, {v[1] / 2}, {1}}, o);
    const Tensor &next = o[0], &src = o[1], &dst = o[2], &count = o[3];
    const int rc = unlocked([&] {
      return moe_cache_compact(table.const_data_ptr<int32_t>(), stride, table.size(1), lengths.const_data_ptr<int32_t>(), table.size(0), (int32_t)v[0],
                               v[1], next.data_ptr<int32_t>(), src.data_ptr<int32_t>(), dst.data_ptr<int32_t>(), count.data_ptr<int32_t>(), nullptr,
                               stream_of(table));
    });
    return rc == MOE_OK ? wrapped({next, src, dst, count}) : failed("moe_cache_compact", rc);
  });
}

// A page is one block of memory, and pages do not overlap.
bool pages_of(const Tensor& t, int64_t num_pages, c10::Device device, moe_cache_pages* p) {
  if (!t.is_cuda() || t.device() != device || t.dim() < 1 || t.size(0) != num_pages || t.dim() > 8) return false;
  std::array<std::pair<int64_t, int64_t>, 8> dims;
  int n = 0;
  for (int64_t i = 1; i < t.dim(); ++i)
    if (t.size(i) != 1) dims[n++] = {t.stride(i), t.size(i)};
  std::sort(dims.begin(), dims.begin() + n);
  int64_t size = 1;
  for (int i = 0; i < n; ++i) {
    if (dims[i].first != size || dims[i].second == 0) return false;
    size *= dims[i].second;
  }
  const int64_t stride = num_pages > 1 ? t.stride(0) : size, e = t.element_size();
  *p = {t.data_ptr(), stride * e, size * e};
  return stride >= size;
}

// caches (a list), src, dst, count -> ()
PyObject* cache_copy(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[3];
    if (n != 4 || !PyList_Check(args[0]) || !tensors(args + 1, 3, t, 4)) return nullptr;
    const Py_ssize_t num = PyList_GET_SIZE(args[0]);
    const Tensor &src = t[0], &dst = t[1], &count = t[2];
    if (num < 1 || num > MOE_CACHE_MAX_CACHES || !src.is_cuda()) return nullptr;
    const int64_t pairs = src.numel();
    if (!ints_of(src, src.device(), {pairs}) || !ints_of(dst, src.device(), {pairs}) || (count.defined() && !ints_of(count, src.device(), {1}))) return nullptr;
    std::array<moe_cache_pages, MOE_CACHE_MAX_CACHES> entries;
    int64_t pages = 0;
    for (Py_ssize_t i = 0; i < num; ++i) {
      PyObject* o = PyList_GET_ITEM(args[0], i);
      if (!THPVariable_Check(o)) return nullptr;
      const Tensor& c = THPVariable_Unpack(o);
      if (i == 0) pages = c.dim() < 1 ? 0 : c.size(0);
      if (!pages_of(c, pages, src.device(), &entries[i])) return nullptr;
    }
    const c10::cuda::CUDAGuard current(src.device());
    const int rc = unlocked([&] {
      return moe_cache_copy(entries.data(), num, pages, src.const_data_ptr<int32_t>(), dst.const_data_ptr<int32_t>(), pairs,
                            count.defined() ? count.const_data_ptr<int32_t>() : nullptr, nullptr, stream_of(src));
    });
    return rc == MOE_OK ? wrapped({}) : failed("moe_cache_copy", rc);
  });
}

// logits, scores, num_out, ended, end_token -> (scores, parents, tokens)
PyObject* beam_select(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Tensor t[2], ended;
    int64_t num_out, end_token;
    if (n != 5 || !tensors(args, 2, t) || !tensors(args + 3, 1, &ended, 1) || !ints(args + 2, 1, &num_out) || !ints(args + 4, 1, &end_token)) return nullptr;
    const Tensor &x = t[0], &scores = t[1];
    if (!x.is_cuda() || dtype_of(x) < 0 || x.dim() != 3 || num_out < 1 || num_out > MOE_BEAM_MAX_OUT || !fits32(end_token)) return nullptr;
    const int64_t B = x.size(0), W = x.size(1), V = x.size(2), stride = W == 1 ? step(x, 0) : step(x, 1);
    if ((V > 1 && x.stride(2) != 1) || (B > 1 && W > 1 && x.stride(0) != W * stride) || (B * W > 1 && stride < V) || !plain(scores, x, at::kFloat, {B, W}) ||
        (ended.defined() && !plain(ended, x, at::kBool, {B, W}) && !plain(ended, x, at::kByte, {B, W})) || !fits32(W))
      return nullptr;
    const c10::cuda::CUDAGuard current(x.device());
    const size_t bytes = moe_beam_select_workspace_size(B, (int32_t)W, V);
    if (bytes == 0) return nullptr;
    Tensor o[3];
    parts_of(x, {at::kFloat, at::kInt, at::kInt}, {{B, num_out}, {B, num_out}, {B, num_out}}, o);
    const Tensor &best = o[0], &from = o[1], &token = o[2], ws = make(x, at::kByte, {(int64_t)bytes});
    const int rc = unlocked([&] {
      return moe_beam_select(x.const_data_ptr(), dtype_of(x), stride, scores.const_data_ptr<float>(),
                             static_cast<const uint8_t*>(ended.defined() ? ended.const_data_ptr() : nullptr), B, (int32_t)W, V, (int32_t)num_out,
                             (int32_t)end_token, best.data_ptr<float>(), from.data_ptr<int32_t>(), token.data_ptr<int32_t>(), ws.data_ptr(), bytes,
                             stream_of(x));
    });
    return rc == MOE_OK ? wrapped({best, from, token}) : failed("moe_beam_select", rc);
  });
}

PyMethodDef methods[] = {CALL(attention_decode), CALL(cache_write), CALL(cache_fork), CALL(cache_compact), CALL(cache_copy), CALL(beam_select),
                         {nullptr, nullptr, 0, nullptr}};

}  // namespace

PyMethodDef* decode_methods() { return methods; }

}  // namespace moe_calls
