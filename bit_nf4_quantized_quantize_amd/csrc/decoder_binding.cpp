// The Python side of the decoder-block operators (include/qlora_decoder.h): a
// CPython module that checks tensors, allocates what a call returns and calls
// the C ABI, for decoder.py.  Host code only.
//
// Decoding calls these operators many times per token with little work in
// each, so the host side counts: through Python and ctypes a small call took 8.5
// to 10 us, through this 4 to 5.5, of which the launch itself is 3.3.
//
// Every function returns a tuple of its results; or an int, the non-zero status
// of the ABI call; or None when the tensors' device is not the current one (the
// caller makes it current and calls again).
#include "binding_args.h"

#include <cmath>

#include "qlora_decoder.h"

namespace {

using namespace qlora_py;

// --------------------------------------------- norm, gate and residual

// (x, h, w_pre, w_post, gate, alpha, eps, n_dtype or -1, xo, n) -> (xo, n)
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 10);
  const Tensor& x = need(a[0], "x");
  const Tensor *h = opt(a[1], "h"), *w_pre = opt(a[2], "w_pre"), *w_post = opt(a[3], "w_post"), *gate = opt(a[4], "gate");
  const float alpha = (float)real(a[5]), eps = (float)real(a[6]);
  int nc = (int)integer(a[7]);
  Out xo(opt(a[8], "xo")), n(opt(a[9], "n"));
  TORCH_CHECK_VALUE(x.dim() >= 1, "x must have a last dimension");
  const int xc = dtype_code(x.scalar_type(), "x");
  const auto shape = x.sizes();
  const int64_t D = shape.back(), T = D ? x.numel() / D : 0;
  dense(&x, "x", shape, x.scalar_type());
  if (h) {
    const int hc = dtype_code(h->scalar_type(), "h");
    dense(h, "h", shape, h->scalar_type());
    TORCH_CHECK_VALUE(nc < 0 || nc == hc, "n has the type of h");
    nc = hc;
  } else if (nc < 0) {
    nc = xc;
  }
  for (const auto& g : {std::make_pair(w_pre, "w_pre"), std::make_pair(w_post, "w_post"), std::make_pair(gate, "gate")})
    dense(g.first, g.second, {D}, at::kFloat);
  dense(xo.given, "xo", shape, x.scalar_type());
  dense(n.given, "n", shape, scalar_of(nc));
  const Device dev({&x, h, w_pre, w_post, gate, xo.given, n.given});
  if (!dev.current) Py_RETURN_NONE;
  if (!xo.given && h) xo.made = at::empty_like(x);
  if (!n.given && w_pre) n.made = nc == xc ? at::empty_like(x) : at::empty(shape, x.options().dtype(scalar_of(nc)));
  int st;
  {
    pybind11::gil_scoped_release no_gil;
    st = qlora_norm_residual_fwd(ptr(x), xc, ptr(h), nc, T, D, as<float>(w_post), as<float>(gate), alpha,
                                 as<float>(w_pre), eps, ptr(xo.get()), ptr(n.get()), dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({xo.given, n.given});
  return results({xo.get() ? xo.get() : &x, n.get()});
  END_HANDLE_TH_ERRORS
}

// (dxo, dn, xo, h, w_pre, w_post, gate, alpha, eps, need_dh, wanted, dx, dh) ->
// (dx, dh, dw_pre, dw_post, dgate); wanted: 1 w_pre, 2 w_post, 4 gate
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 13);
  const Tensor *dxo = opt(a[0], "dxo"), *dn = opt(a[1], "dn"), *h = opt(a[3], "h"), *w_pre = opt(a[4], "w_pre"),
               *w_post = opt(a[5], "w_post"), *gate = opt(a[6], "gate");
  const Tensor& xo = need(a[2], "xo");
  const float alpha = (float)real(a[7]), eps = (float)real(a[8]);
  const bool need_dh = flag(a[9]);
  const int64_t wanted = integer(a[10]);
  Out dx(opt(a[11], "dx")), dh(opt(a[12], "dh"));
  TORCH_CHECK_VALUE(xo.dim() >= 1, "xo must have a last dimension");
  const auto xt = xo.scalar_type();
  const auto ht = h ? h->scalar_type() : dn ? dn->scalar_type() : dh.given ? dh.given->scalar_type() : xt;
  const int xc = dtype_code(xt, "xo"), hc = dtype_code(ht, "h, dn and dh");
  const auto shape = xo.sizes();
  const int64_t D = shape.back(), T = D ? xo.numel() / D : 0;
  dense(&xo, "xo", shape, xt);
  dense(dxo, "dxo", shape, xt);
  dense(dx.given, "dx", shape, xt);
  dense(dn, "dn", shape, ht);
  dense(h, "h", shape, ht);
  dense(dh.given, "dh", shape, ht);
  dense(w_pre, "w_pre", {D}, at::kFloat);
  dense(w_post, "w_post", {D}, at::kFloat);
  dense(gate, "gate", {D}, at::kFloat);
  const Device dev({&xo, dxo, dn, h, w_pre, w_post, gate, dx.given, dh.given});
  if (!dev.current) Py_RETURN_NONE;
  if (!dx.given) dx.made = at::empty_like(xo);
  if (!dh.given && need_dh) dh.made = at::empty(shape, xo.options().dtype(ht));
  const auto f32 = xo.options().dtype(at::kFloat);
  Tensor dw_pre, dw_post, dgate, ws;
  if (dn && (wanted & 1)) dw_pre = at::empty({D}, f32);
  if (w_post && (wanted & 2)) dw_post = at::empty({D}, f32);
  if (gate && (wanted & 4)) dgate = at::empty({D}, f32);
  const int sums = dw_pre.defined() + dw_post.defined() + dgate.defined();
  int64_t bytes = 0;
  if (sums) {
    if (const int st = qlora_norm_residual_bwd_workspace(T, D, xc, hc, sums, &bytes)) return PyLong_FromLong(st);
    ws = at::empty({bytes}, xo.options().dtype(at::kByte));
  }
  const auto made = [](const Tensor& t) { return t.defined() ? (float*)t.data_ptr() : nullptr; };
  int st;
  {
    pybind11::gil_scoped_release no_gil;
    st = qlora_norm_residual_bwd(ptr(dxo), ptr(xo), xc, ptr(dn), ptr(h), hc, T, D, as<float>(w_post), as<float>(gate),
                                 alpha, as<float>(w_pre), eps, ptr(dx.get()), ptr(dh.get()), made(dw_post), made(dgate),
                                 made(dw_pre), made(ws), bytes, dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({dx.given, dh.given});
  return results({dx.get(), dh.get(), &dw_pre, &dw_post, &dgate});
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------ rotary positions

// (q, k, positions, turns, rot_dim, mscale, interleaved, inverse, q_out, k_out)
// -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 10);
  const Tensor *q0 = opt(a[0], "q"), *k0 = opt(a[1], "k"), *t = q0 ? q0 : k0;
  TORCH_CHECK_VALUE(t && t->dim() == 3, "q or k must be given, as [T, heads, head_dim]");
  const Tensor &positions = need(a[2], "positions"), &turns = need(a[3], "turns");
  const int64_t rot = integer(a[4]), T = t->size(0), d = t->size(2);
  const float mscale = (float)real(a[5]);
  const int inter = flag(a[6]), inverse = flag(a[7]);
  const auto type = t->scalar_type();
  const int code = dtype_code(type, "q and k");
  dense(&positions, "positions", {T}, at::kInt);
  dense(&turns, "the table", {rot / 2}, at::kDouble);
  Turned q(q0, opt(a[8], "q_out"), "q", "q_out", T, d, type), k(k0, opt(a[9], "k_out"), "k", "k_out", T, d, type);
  const Device dev({q0, k0, &positions, &turns, q.out.given, k.out.given});
  if (!dev.current) Py_RETURN_NONE;
  q.make();
  k.make();
  int st;
  {
    pybind11::gil_scoped_release no_gil;
    st = qlora_rope(ptr(q0), q.from.stride, (int32_t)q.from.heads, ptr(q.out.get()), q.to.stride, ptr(k0),
                    k.from.stride, (int32_t)k.from.heads, ptr(k.out.get()), k.to.stride, T, (int32_t)d, (int32_t)rot,
                    code, (const int32_t*)ptr(positions), (const double*)ptr(turns), mscale, inter, inverse,
                    dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({q.out.given, k.out.given});
  return results({q.out.get(), k.out.get()});
  END_HANDLE_TH_ERRORS
}

// ----------------------------------------------------------- paged cache

void check_cache(const Tensor& k, const Tensor& v) {
  TORCH_CHECK_VALUE(k.dim() == 4, "the caches must be [num_pages, kv_heads, page_size, head_dim]");
  dense(&k, "k_cache", k.sizes(), at::kBFloat16);
  dense(&v, "v_cache", k.sizes(), at::kBFloat16);
}

// (q, k, v, positions, turns or None, rot_dim, mscale, interleaved, slots,
// k_cache, v_cache, q_out) -> (q_out,)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 12);
  const Tensor *q0 = opt(a[0], "q"), *turns = opt(a[4], "turns"), *positions = turns ? &need(a[3], "positions") : nullptr;
  const Tensor &k = need(a[1], "k"), &v = need(a[2], "v"), &slots = need(a[8], "slots"), &kc = need(a[9], "k_cache"),
               &vc = need(a[10], "v_cache");
  const int64_t rot = turns ? integer(a[5]) : 0;
  const float mscale = (float)real(a[6]);
  const int inter = flag(a[7]);
  check_cache(kc, vc);
  const int64_t kvh = kc.size(1), page = kc.size(2), d = kc.size(3);
  TORCH_CHECK_VALUE(k.dim() == 3, "k must be [tokens, kv_heads, head_dim]");
  const int64_t T = k.size(0);
  dense(&slots, "slots", {T}, at::kInt);
  dense(positions, "positions", {T}, at::kInt);
  dense(turns, "the table", {rot / 2}, at::kDouble);
  const Heads kh = heads_of(k, "k", T, d, at::kBFloat16), vh = heads_of(v, "v", T, d, at::kBFloat16);
  TORCH_CHECK_VALUE(kh.heads == kvh && vh.heads == kvh, "k and v must have the cache's heads");
  Turned q(q0, opt(a[11], "q_out"), "q", "q_out", T, d, at::kBFloat16);
  const Device dev({&k, &v, q0, turns, positions, &slots, &kc, &vc, q.out.given});
  if (!dev.current) Py_RETURN_NONE;
  q.make();
  TORCH_CHECK_VALUE(page <= INT32_MAX && d <= INT32_MAX && kvh <= INT32_MAX, "the cache is too large");
  int st;
  {
    pybind11::gil_scoped_release no_gil;
    st = qlora_rope_cache_write(ptr(q0), q.from.stride, (int32_t)q.from.heads, ptr(q.out.get()), q.to.stride, ptr(k),
                                kh.stride, ptr(v), vh.stride, (int32_t)kvh, T, (int32_t)d, (int32_t)rot,
                                as<const int32_t>(positions), as<const double>(turns), mscale, inter,
                                (const int32_t*)ptr(slots), ptr(kc), ptr(vc), kc.size(0), (int32_t)page, dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({&kc, &vc, q.out.given});
  return results({q.out.get()});
  END_HANDLE_TH_ERRORS
}

// (cached_lens, new_lens, free_pages, block_table, page_size, tokens, out or
// None) -> (total_lens, starts, slots, positions, pages_needed)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 7);
  const Tensor &cached = need(a[0], "cached_lens"), &fresh = need(a[1], "new_lens"), &free_pages = need(a[2], "free_pages"),
               &table = need(a[3], "block_table");
  const int64_t page = integer(a[4]), tokens = integer(a[5]);
  TORCH_CHECK_VALUE(page > 0 && page <= INT32_MAX && tokens >= 0 && tokens <= INT32_MAX,
                    "page_size must be positive and tokens not negative");
  TORCH_CHECK_VALUE(cached.dim() == 1 && table.dim() == 2, "cached_lens must be [sequences], block_table [sequences, "
                    "columns]");
  const int64_t S = cached.size(0), cols = table.size(1), nfree = free_pages.numel();
  dense(&cached, "cached_lens", {S}, at::kInt);
  dense(&fresh, "new_lens", {S}, at::kInt);
  dense(&free_pages, "free_pages", {nfree}, at::kInt);
  dense(&table, "block_table", {S, cols}, at::kInt);
  const int64_t sizes[5] = {S, S + 1, tokens, tokens, 1};
  static const char* const names[5] = {"total_lens", "starts", "slots", "positions", "pages_needed"};
  Tensor out[5];
  if (a[6] != Py_None) {
    TORCH_CHECK_VALUE(PyTuple_Check(a[6]) && PyTuple_GET_SIZE(a[6]) == 5, "out must be a PagedPlan");
    for (int i = 0; i < 5; ++i) {
      out[i] = need(PyTuple_GET_ITEM(a[6], i), names[i]);
      dense(&out[i], names[i], {sizes[i]}, at::kInt);
    }
  }
  const auto given = [&](int i) { return a[6] != Py_None ? &out[i] : nullptr; };
  const Device dev({&cached, &fresh, &free_pages, &table, given(0), given(1), given(2), given(3), given(4)});
  if (!dev.current) Py_RETURN_NONE;
  if (a[6] == Py_None) {
    // one allocation, five parts
    auto parts = at::empty({2 * (S + tokens + 1)}, cached.options()).split_with_sizes(at::IntArrayRef(sizes, 5));
    for (int i = 0; i < 5; ++i) out[i] = std::move(parts[i]);
  }
  const auto i32 = [](const Tensor& t) { return (int32_t*)t.data_ptr(); };
  int st;
  {
    pybind11::gil_scoped_release no_gil;
    st = qlora_paged_plan(i32(cached), i32(fresh), S, (int32_t)page, i32(free_pages), nfree, i32(table), cols, tokens,
                          i32(out[0]), i32(out[1]), i32(out[2]), i32(out[3]), i32(out[4]), dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({&table, given(0), given(1), given(2), given(3), given(4)});
  return results({&out[0], &out[1], &out[2], &out[3], &out[4]});
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, block_table, lengths, scale or None, out, lse) -> (out,)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  count(n_args, 8);
  const Tensor &q = need(a[0], "q"), &kc = need(a[1], "k_cache"), &vc = need(a[2], "v_cache"),
               &table = need(a[3], "block_table"), &lengths = need(a[4], "lengths");
  Out out(opt(a[6], "out"));
  const Tensor* lse = opt(a[7], "lse");
  check_cache(kc, vc);
  const int64_t kvh = kc.size(1), page = kc.size(2), d = kc.size(3);
  TORCH_CHECK_VALUE(q.dim() == 3 && table.dim() == 2, "q must be [sequences, heads, head_dim], block_table [sequences, "
                    "columns]");
  const int64_t S = q.size(0), cols = table.size(1);
  const Heads qh = heads_of(q, "q", S, d, at::kBFloat16);
  dense(&lengths, "lengths", {S}, at::kInt);
  dense(&table, "block_table", {S, cols}, at::kInt);
  dense(out.given, "out", q.sizes(), at::kBFloat16);
  dense(lse, "lse", {S, qh.heads}, at::kFloat);
  const float scale = a[5] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)real(a[5]);
  const Device dev({&q, &kc, &vc, &table, &lengths, out.given, lse});
  if (!dev.current) Py_RETURN_NONE;
  TORCH_CHECK_VALUE(page <= INT32_MAX && d <= INT32_MAX && kvh <= INT32_MAX && qh.heads <= INT32_MAX,
                    "the cache is too large");
  int64_t bytes = 0;
  int st = qlora_paged_attention_workspace(S, (int32_t)qh.heads, (int32_t)kvh, (int32_t)d, cols, (int32_t)page, &bytes);
  if (st) return PyLong_FromLong(st);
  if (!out.given) out.made = new_like(q);
  Tensor ws;
  if (bytes) ws = at::empty({bytes}, q.options().dtype(at::kByte));
  {
    pybind11::gil_scoped_release no_gil;
    st = qlora_paged_attention(ptr(q), qh.stride, S, (int32_t)qh.heads, (int32_t)kvh, (int32_t)d, ptr(kc), ptr(vc),
                               kc.size(0), (int32_t)page, (const int32_t*)ptr(table), cols, (const int32_t*)ptr(lengths),
                               scale, ptr(out.get()), as<float>(lse), bytes ? ws.data_ptr() : nullptr, bytes,
                               dev.stream());
  }
  if (st) return PyLong_FromLong(st);
  wrote({out.given, lse});
  return results({out.get()});
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {method<norm_fwd>("norm_fwd"), method<norm_bwd>("norm_bwd"), method<rope>("rope"),
                         method<cache_write>("cache_write"), method<plan>("plan"),
                         method<attention>("attention"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_decoder", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decoder() { return PyModule_Create(&module); }
