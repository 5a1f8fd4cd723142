"""Writes of the decoder-block operators into tensors they are given, as autograd
sees them: the version of such a tensor rises, so a backward that saved it raises
instead of using what it became."""

import pytest
import torch

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def D():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_nf4_quantized_quantize_amd import decoder
    decoder.native()
    return decoder


def _calls(D):
    """name -> (function, arguments, names of the arguments it writes)."""
    b = lambda *s: torch.randn(*s, device="cuda").to(BF)  # noqa: E731
    x, h, w = b(5, 64), b(5, 64), torch.ones(64, device="cuda")
    q, k, v, tab = b(3, 4, 32), b(3, 2, 32), b(3, 2, 32), D.RopeTable(32, device="cuda")
    lens, cols = torch.tensor([5, 17, 0], **I32), torch.arange(6, **I32).view(3, 2)
    kc, vc = b(6, 2, 16, 32), b(6, 2, 16, 32)
    e = lambda *s: torch.empty(*s, **I32)  # noqa: E731
    plan = D.PagedPlan(e(3), e(4), e(3), e(3), e(1))
    return {
        "norm_fwd": (D.qlora_norm_residual_fwd, dict(x=x, h=h, w_pre=w, w_post=w, gate=w, xo=x, n=b(5, 64)), ("xo", "n")),
        "norm_bwd": (D.qlora_norm_residual_bwd, dict(dxo=x, dn=h, xo=b(5, 64), h=b(5, 64), w_pre=w, w_post=w, gate=w,
                                                     need_gains=True, dx=x, dh=h), ("dx", "dh")),
        "rope": (D.qlora_rope, dict(q=q, k=k, table=tab, positions=lens, q_out=q, k_out=b(3, 2, 32)),
                 ("q_out", "k_out")),
        "write": (D.qlora_rope_cache_write, dict(q=q, k=k, v=v, table=tab, positions=lens, slots=lens, k_cache=kc,
                                                 v_cache=vc, q_out=b(3, 4, 32)), ("k_cache", "v_cache", "q_out")),
        "plan": (D.qlora_paged_plan, dict(cached_lens=lens, new_lens=torch.ones(3, **I32), free_pages=torch.arange(6, **I32),
                                          block_table=cols, page_size=16, tokens=3, out=plan),
                 ("block_table", *plan._fields)),
        "attention": (D.qlora_paged_attention, dict(q=q, k_cache=kc, v_cache=vc, block_table=cols, lengths=lens,
                                                    out=b(3, 4, 32), lse=torch.empty(3, 4, device="cuda")),
                      ("out", "lse")),
    }


NAMES = ("norm_fwd", "norm_bwd", "rope", "write", "plan", "attention")


def _tensors(kw):
    named = {k: v for k, v in kw.items() if isinstance(v, torch.Tensor)}
    if "tokens" in kw:
        named.update(kw["out"]._asdict())
    return named


@pytest.mark.parametrize("with_stream", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_versions_rise_where_a_call_writes(D, name, with_stream):
    f, kw, written = _calls(D)[name]
    tensors = _tensors(kw)
    before = {k: t._version for k, t in tensors.items()}
    mine = {id(tensors[k]) for k in written}
    f(**kw, stream=torch.cuda.Stream() if with_stream else None)
    torch.cuda.synchronize()
    for k, t in tensors.items():
        assert (t._version > before[k]) == (id(t) in mine), k


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_call_leaves_the_versions(D, name):
    f, kw, _ = _calls(D)[name]
    tensors = _tensors(kw)
    before = {k: t._version for k, t in tensors.items()}
    first = next(k for k, v in kw.items() if isinstance(v, torch.Tensor))
    with pytest.raises((TypeError, ValueError)):
        f(**{**kw, first: kw[first].cpu()})
    assert {k: t._version for k, t in tensors.items()} == before


@pytest.mark.parametrize("name", NAMES)
def test_inference_tensors_are_taken(D, name):
    """Tensors made under inference mode have no version."""
    with torch.inference_mode():
        f, kw, _ = _calls(D)[name]
        f(**kw)
    f(**kw)
    torch.cuda.synchronize()


def test_positions_planned_anew_under_a_rotation_are_noticed(D):
    from bit_nf4_quantized_quantize_amd import block
    _, kw, _ = _calls(D)["plan"]
    plan = D.qlora_paged_plan(**kw)
    q = torch.randn(3, 4, 32, device="cuda", requires_grad=True)
    out, _ = block.rope(q, None, D.RopeTable(32, device="cuda"), plan.positions)
    D.qlora_paged_plan(**kw)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_a_stream_updated_under_its_norm_is_noticed(D):
    """The library's own update in place of a stream that a norm saved, and one of a
    view of it."""
    from bit_nf4_quantized_quantize_amd import block
    w, h = torch.ones(64, device="cuda"), torch.randn(5, 64, device="cuda").to(BF)
    for view in (False, True):
        x = torch.randn(5, 64, device="cuda")
        leaf = h.clone().requires_grad_(True)
        xo, n = block.norm_residual(x, leaf, w)
        to = xo.detach()[:] if view else xo.detach()
        D.qlora_norm_residual_fwd(to, h, xo=to)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            n.float().sum().backward()


def test_a_queries_buffer_rotated_under_a_product_is_noticed(D):
    """A torch operation's saved input, rotated where it lies."""
    q, w = torch.randn(3, 4, 32, device="cuda"), torch.ones(3, 4, 32, device="cuda", requires_grad=True)
    y = (q * w).sum()
    D.qlora_rope(q, None, D.RopeTable(32, device="cuda"), torch.arange(3, **I32), q_out=q)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
