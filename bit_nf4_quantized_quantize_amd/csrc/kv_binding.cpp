// The Python side of the 8-bit and the shared key-value cache
// (include/qlora_kvcache.h): a CPython module that checks tensors, allocates what
// a call returns and calls the C ABI, for kvcache.py.  Host code only.
//
// Every function returns a tuple of its results; or an int, the non-zero status
// of the ABI call; or None when the tensors' device is not the current one (the
// caller makes it current and calls again).
#include "binding_args.h"

#include <cmath>

#include "qlora_kvcache.h"

namespace {

using namespace qlora_py;

// The four tensors of a cache.
struct Cache {
  const Tensor &k, &v;
  const Tensor *ks, *vs;
  qlora_kv_cache c = {};
  explicit Cache(PyObject* const* a)
      : k(need(a[0], "cache.k")), v(need(a[1], "cache.v")), ks(opt(a[2], "cache.k_scale")), vs(opt(a[3], "cache.v_scale")) {
    TORCH_CHECK_VALUE(k.dim() == 4, "cache.k must be [num_pages, kv_heads, page_size, head_dim]");
    const auto t = k.scalar_type();
    TORCH_CHECK_VALUE(t == at::kBFloat16 || t == at::kChar || t == at::kFloat8_e4m3fn,
                      "cache.k must be bfloat16, int8 or float8_e4m3fn");
    dense(&k, "cache.k", k.sizes(), t);
    dense(&v, "cache.v", k.sizes(), t);
    const bool coded = t != at::kBFloat16;
    TORCH_CHECK_VALUE(coded == (ks != nullptr) && coded == (vs != nullptr),
                      "a cache of 8 bits needs cache.k_scale and cache.v_scale, one of bfloat16 has none");
    const at::IntArrayRef rows = k.sizes().slice(0, 3);
    dense(ks, "cache.k_scale", rows, at::kFloat);
    dense(vs, "cache.v_scale", rows, at::kFloat);
    for (int i = 1; i < 4; ++i) TORCH_CHECK_VALUE(k.size(i) <= INT32_MAX, "the cache is too large");
    c.num_pages = k.size(0);
    c.kv_heads = (int32_t)k.size(1), c.page_size = (int32_t)k.size(2), c.head_dim = (int32_t)k.size(3);
    c.type = t == at::kChar ? QLORA_CACHE_INT8 : coded ? QLORA_CACHE_E4M3 : QLORA_CACHE_BF16;
  }
  // The buffers, once the device is known to be the right one.
  const qlora_kv_cache* on_device() {
    c.k = ptr(k), c.v = ptr(v), c.k_scale = as<float>(ks), c.v_scale = as<float>(vs);
    return &c;
  }
};

// (q, k, v, positions, turns or None, rot_dim, mscale, interleaved, slots,
// cache (4), q_out) -> (q_out,)
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 14);
  const Tensor *q0 = opt(a[0], "q"), *turns = opt(a[4], "turns"), *positions = turns ? &need(a[3], "positions") : nullptr;
  const Tensor &k = need(a[1], "k"), &v = need(a[2], "v"), &slots = need(a[8], "slots");
  const int64_t rot = turns ? integer(a[5]) : 0;
  const float mscale = (float)real(a[6]);
  const int inter = flag(a[7]);
  Cache cache(a + 9);
  const int64_t d = cache.c.head_dim;
  TORCH_CHECK_VALUE(k.dim() == 3, "k must be [tokens, kv_heads, head_dim]");
  const int64_t T = k.size(0);
  dense(&slots, "slots", {T}, at::kInt);
  dense(positions, "positions", {T}, at::kInt);
  dense(turns, "the table", {rot / 2}, at::kDouble);
  const Heads kh = heads_of(k, "k", T, d, at::kBFloat16), vh = heads_of(v, "v", T, d, at::kBFloat16);
  TORCH_CHECK_VALUE(kh.heads == cache.c.kv_heads && vh.heads == cache.c.kv_heads, "k and v must have the cache's heads");
  Turned q(q0, opt(a[13], "q_out"), "q", "q_out", T, d, at::kBFloat16);
  const Device dev({&k, &v, q0, turns, positions, &slots, &cache.k, &cache.v, cache.ks, cache.vs, q.out.given});
  if (!dev.current) Py_RETURN_NONE;
  q.make();
  const qlora_kv_cache* c = cache.on_device();
  int st;
  {
    pybind11::gil_scoped_release no_gil;
    st = qlora_kv_write(ptr(q0), q.from.stride, (int32_t)q.from.heads, ptr(q.out.get()), q.to.stride, ptr(k), kh.stride,
                        ptr(v), vh.stride, T, (int32_t)rot, as<const int32_t>(positions), as<const double>(turns),
                        mscale, inter, (const int32_t*)ptr(slots), c, dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({&cache.k, &cache.v, cache.ks, cache.vs, q.out.given});
  return results({q.out.get()});
  END_HANDLE_TH_ERRORS
}

// (cache (4), slots, dtype code, k_out, v_out) -> (k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 8);
  Cache cache(a);
  const Tensor& slots = need(a[4], "slots");
  const int code = (int)integer(a[5]);
  Out k(opt(a[6], "k_out")), v(opt(a[7], "v_out"));
  TORCH_CHECK_VALUE(slots.dim() == 1, "slots must be [tokens]");
  const int64_t T = slots.size(0), shape[3] = {T, cache.c.kv_heads, cache.c.head_dim};
  const auto type = scalar_of(code);
  dense(&slots, "slots", {T}, at::kInt);
  dense(k.given, "k_out", shape, type);
  dense(v.given, "v_out", shape, type);
  const Device dev({&cache.k, &cache.v, cache.ks, cache.vs, &slots, k.given, v.given});
  if (!dev.current) Py_RETURN_NONE;
  if (!k.given) k.made = at::empty(shape, cache.k.options().dtype(type));
  if (!v.given) v.made = at::empty(shape, cache.k.options().dtype(type));
  const qlora_kv_cache* c = cache.on_device();
  int st;
  {
    pybind11::gil_scoped_release no_gil;
    st = qlora_kv_read(c, (const int32_t*)ptr(slots), T, code, ptr(k.get()), ptr(v.get()), dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({k.given, v.given});
  return results({k.get(), v.get()});
  END_HANDLE_TH_ERRORS
}

// (q, cache (4), prefix_table or None, prefix_len or None, block_table, lengths,
// scale or None, out, lse) -> (out,)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 12);
  const Tensor& q = need(a[0], "q");
  Cache cache(a + 1);
  const bool shared = a[5] != Py_None || a[6] != Py_None;
  const Tensor *ptable = shared ? &need(a[5], "prefix_table") : nullptr, *plen = shared ? &need(a[6], "prefix_len") : nullptr;
  const Tensor &table = need(a[7], "block_table"), &lengths = need(a[8], "lengths");
  Out out(opt(a[10], "out"));
  const Tensor* lse = opt(a[11], "lse");
  const int64_t d = cache.c.head_dim;
  TORCH_CHECK_VALUE(q.dim() == 3 && table.dim() == 2, "q must be [sequences, heads, head_dim], block_table [sequences, "
                    "columns]");
  const int64_t S = q.size(0), cols = table.size(1);
  const Heads qh = heads_of(q, "q", S, d, at::kBFloat16);
  dense(&lengths, "lengths", {S}, at::kInt);
  dense(&table, "block_table", {S, cols}, at::kInt);
  TORCH_CHECK_VALUE(!shared || ptable->dim() == 1, "prefix_table must be [columns]");
  const int64_t pcols = shared ? ptable->size(0) : 0;
  dense(ptable, "prefix_table", {pcols}, at::kInt);
  dense(plen, "prefix_len", {1}, at::kInt);
  dense(out.given, "out", q.sizes(), at::kBFloat16);
  dense(lse, "lse", {S, qh.heads}, at::kFloat);
  const float scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)real(a[9]);
  const Device dev({&q, &cache.k, &cache.v, cache.ks, cache.vs, ptable, plen, &table, &lengths, out.given, lse});
  if (!dev.current) Py_RETURN_NONE;
  const qlora_kv_cache* c = cache.on_device();
  const int32_t heads = (int32_t)qh.heads;
  int64_t bytes = 0;
  int st = shared ? qlora_prefix_attention_workspace(c, S, heads, pcols, cols, &bytes)
                  : qlora_kv_attention_workspace(c, S, heads, cols, &bytes);
  if (st) return PyLong_FromLong(st);
  if (!out.given) out.made = new_like(q);
  Tensor ws;
  if (bytes) ws = at::empty({bytes}, q.options().dtype(at::kByte));
  void* const scratch = bytes ? ws.data_ptr() : nullptr;
  const auto* t = (const int32_t*)ptr(table);
  const auto* n = (const int32_t*)ptr(lengths);
  {
    pybind11::gil_scoped_release no_gil;
    if (shared)
      st = qlora_prefix_attention(ptr(q), qh.stride, S, heads, c, as<const int32_t>(ptable), pcols,
                                  as<const int32_t>(plen), t, cols, n, scale, ptr(out.get()), as<float>(lse), scratch,
                                  bytes, dev.stream());
    else
      st = qlora_kv_attention(ptr(q), qh.stride, S, heads, c, t, cols, n, scale, ptr(out.get()), as<float>(lse),
                              scratch, bytes, dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({out.given, lse});
  return results({out.get()});
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {method<write>("write"), method<read>("read"), method<attention>("attention"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvcache", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvcache() { return PyModule_Create(&module); }
