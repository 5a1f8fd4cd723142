"""A LLaMA-shaped decoder block with QLoRA adapters on all seven linear
layers, for measuring what a whole layer costs in memory and time.

QLoRA (Dettmers et al., arXiv 2305.14314) puts adapters on every network
layer (introduction). Section 2 "Memory Requirement of Parameter-Efficient
Finetuning" finds that activation gradients, not LoRA parameters, dominate
training memory, and that gradient checkpointing shrinks them. Appendix G
"Memory Footprint" (Figure 6) measures with batch 1, sequence length 512 and
checkpointing.

The block is the pre-norm LLaMA layer without rotary encoding:
    n1 = rmsnorm(x) g1;  h = x + L_o(attn(L_q(n1), L_k(n1), L_v(n1)))
    n2 = rmsnorm(h) g2;  y = h + L_down(silu(L_gate(n2)) * L_up(n2))
Every L is the library's frozen-NF4 linear with a LoRA adapter, run through
qlora_linear_fwd / qlora_linear_bwd on bf16 operands. The glue around them
(rmsnorm, causal attention, SiLU, residuals) is the surrounding model, not
part of the layer, and runs as plain fp32 torch ops. Only the adapters and
the block input receive gradients. With checkpoint=True the forward keeps
only the block input for the backward and runs again inside it.

With `fused` the glue runs on the library's kernels instead: the norms and
the residual update as qlora_norm_residual_fwd / _bwd, 16-bit between the
linears. That form also takes what the plain one lacks: rotary positions
(qlora_rope), norms behind the branches, gates and a residual scale
    h = x + c * t1 * post1(L_o(...)),  y = h + c * t2 * post2(L_down(...)),
gradients for the norm gains and gates that require them, and decoding from
a paged key-value cache (prefill, decode), which may hold its rows in 8 bits and
a prefix that all sequences share (prefill_shared). The attention core and SiLU
stay fp32 torch ops. Blocks of this form may run on several streams at once, and
their forward be captured into a graph (prefill and decode not: the cache takes
counts from the host); the plain one shares the binding's workspace of the
device, so its calls belong on one stream.
"""

import math

import torch
import torch.utils.checkpoint
from torch.autograd.function import once_differentiable

from . import binding as B
from . import decoder as D
from . import kvcache as K

LINEARS = ("q", "k", "v", "o", "gate", "up", "down")
EPS = 1e-6


def linear_shapes(hidden, mlp):
    """[out, in] weight shape of each linear."""
    return {"q": (hidden, hidden), "k": (hidden, hidden), "v": (hidden, hidden), "o": (hidden, hidden),
            "gate": (mlp, hidden), "up": (mlp, hidden), "down": (hidden, mlp)}


class _CallWorkspace:
    """Scratch of one linear call from the allocator, on the call's stream. The
    binding's own is one per device: calls on other streams and captured graphs
    would share it."""

    @staticmethod
    def get(nbytes, device):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


class _QLoraLinearFn(torch.autograd.Function):
    """Y = X W_bf16^T + s (X A) B on the library's kernels; the backward
    returns dX, dA, dB (no dW)."""

    @staticmethod
    def forward(ctx, X, A, Bm, lin, workspace):
        Y, XA = B.qlora_linear_fwd(X, lin.qw, A, Bm, lin.s, workspace=workspace)
        ctx.save_for_backward(X, XA, A, Bm)
        ctx.lin, ctx.workspace = lin, workspace
        return Y

    @staticmethod
    def backward(ctx, dY):
        X, XA, A, Bm = ctx.saved_tensors
        lin = ctx.lin
        dX, dA, dB = B.qlora_linear_bwd(dY.contiguous(), X, XA, lin.qw, A, Bm, lin.s, workspace=ctx.workspace)
        return dX, dA, dB, None, None


class QLoraLinear:
    """One frozen NF4 (+ double quantisation) weight with a bf16 LoRA adapter
    (A [in, r], B [r, out], both leaves with requires_grad)."""

    def __init__(self, W, A, Bm, s):
        self.qw = B.qlora_nf4_quantize(W.contiguous(), double_quant=True)
        self.out_features, self.in_features = W.shape
        self.A = A.to(torch.bfloat16).contiguous().requires_grad_(True)
        self.B = Bm.to(torch.bfloat16).contiguous().requires_grad_(True)
        self.s = float(s)

    def __call__(self, z):
        """z: fp32 [..., in] -> fp32 [..., out] (bf16 at the layer boundary)."""
        lead = z.shape[:-1]
        X = z.reshape(-1, self.in_features).to(torch.bfloat16).contiguous()
        Y = _QLoraLinearFn.apply(X, self.A, self.B, self, None)
        return Y.float().reshape(*lead, self.out_features)

    def bf16(self, X):
        """X: bf16 [tokens, in] -> bf16 [tokens, out]."""
        return _QLoraLinearFn.apply(X.contiguous(), self.A, self.B, self, _CallWorkspace)

    def storage_bytes(self):
        return sum(self.qw.sizes.values())


def _dense16(t):
    """t (or None) contiguous and on a 16-byte boundary, as the library takes it
    (a contiguous slice of a larger tensor may start off one)."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _NormResidualFn(torch.autograd.Function):
    """qlora_norm_residual_fwd with its backward."""

    @staticmethod
    def forward(ctx, x, h, w_pre, w_post, gate, alpha, eps, n_dtype):
        xo, n = D.qlora_norm_residual_fwd(x, h, w_pre, w_post, gate, alpha, eps, n_dtype if h is None else None)
        need_h = w_post is not None or ctx.needs_input_grad[4]
        ctx.save_for_backward(xo if w_pre is not None else None, h if need_h else None, w_pre, w_post, gate)
        ctx.args = (None if h is None else h.dtype, alpha, eps)
        ctx.set_materialize_grads(False)
        return xo, n

    @staticmethod
    @once_differentiable
    def backward(ctx, dxo, dn):
        if dxo is None and dn is None:
            return (None,) * 8
        xo, h, w_pre, w_post, gate = ctx.saved_tensors
        ht, alpha, eps = ctx.args
        dxo, dn = _dense16(dxo), _dense16(dn)
        need = ctx.needs_input_grad
        gains = [name for i, name in ((2, "w_pre"), (3, "w_post"), (4, "gate")) if need[i]]
        if xo is None:
            xo = dxo      # no norm of the stream: its values do not matter
        dh = torch.empty(xo.shape, dtype=ht, device=xo.device) if ht is not None and need[1] else None
        gr = D.qlora_norm_residual_bwd(dxo, dn, xo, h, w_pre if dn is not None else None, w_post, gate, alpha, eps,
                                       need_dh=dh is not None, need_gains=gains, dh=dh)
        return gr.dx, gr.dh, gr.dw_pre, gr.dw_post, gr.dgate, None, None, None


def norm_residual(x, h=None, w_pre=None, w_post=None, gate=None, alpha=1.0, eps=EPS, n_dtype=torch.bfloat16):
    """Differentiable qlora_norm_residual_fwd: (xo, n).  Without h, xo is x and n
    has n_dtype; without w_pre, n is None."""
    return _NormResidualFn.apply(_dense16(x), _dense16(h), w_pre, w_post, gate, alpha, eps, n_dtype)


class _RopeFn(torch.autograd.Function):
    """qlora_rope; the backward turns the other way."""

    @staticmethod
    def forward(ctx, q, k, table, positions):
        ctx.table = table
        ctx.save_for_backward(positions, table.turns)   # as they are now: a later change is noticed
        ctx.set_materialize_grads(False)
        return D.qlora_rope(q, k, table, positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        if dq is not None or dk is not None:
            dq, dk = D.qlora_rope(_dense16(dq), _dense16(dk), ctx.table, ctx.saved_tensors[0], inverse=True)
        return dq, dk, None, None


def rope(q, k, table, positions):
    """Differentiable qlora_rope of q and k [T, heads, head_dim] (either may be
    None)."""
    return _RopeFn.apply(q, k, table, positions)


class PagedCache:
    """The paged key-value cache of one block for up to `max_seqs` sequences of
    up to `max_len` tokens: pages [num_pages, heads, page_size, head_dim] of keys
    and values, the block table, and the pages not in use. dtype is bfloat16, or
    int8 or float8_e4m3fn for rows of codes with a scale each (`rows` is the
    KVCache). With max_prefix the sequences may share up to that many tokens, which
    come before their own and lie in pages of their own, once.
    The lengths are known to the host too, so running out of room raises
    before anything is enqueued.  page_size is a power of two from 16 to 1024,
    head_dim a multiple of 8 (of 16 for codes) up to 256, as the attention takes
    them, max_seqs at most 4096, as the plan does."""

    def __init__(self, num_pages, page_size, heads, head_dim, max_seqs, max_len, device=None, dtype=torch.bfloat16,
                 max_prefix=0):
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        if dtype not in K.CACHE_TYPES:
            raise ValueError("a cache is bfloat16, int8 or float8_e4m3fn")
        unit = 8 if dtype == torch.bfloat16 else 16
        if page_size not in (16, 32, 64, 128, 256, 512, 1024) or head_dim % unit or not unit <= head_dim <= 256:
            raise ValueError(f"page_size must be a power of two in [16, 1024], head_dim a multiple of {unit} in [{unit}, "
                             "256]")
        if not 1 <= max_seqs <= D.PLAN_MAX_SEQS or heads < 1:
            raise ValueError(f"max_seqs must be in [1, {D.PLAN_MAX_SEQS}], heads at least 1")
        if not 1 <= num_pages * page_size < 2 ** 31 or not 1 <= max_len <= 2 ** 31 - page_size:
            raise ValueError("num_pages and max_len must be at least 1, num_pages * page_size and max_len in whole pages "
                             "below 2^31")
        if not 0 <= max_prefix <= 2 ** 31 - 4097 - page_size or max_prefix + max_len > 2 ** 31 - page_size:
            raise ValueError("max_prefix must be at least 0, max_prefix + max_len in whole pages below 2^31")
        self.rows = K.KVCache.zeros(num_pages, heads, page_size, head_dim, dtype, dev)
        self.k, self.v = self.rows.k, self.rows.v
        self.page_size, self.max_len, self.max_prefix = int(page_size), int(max_len), int(max_prefix)
        self.free = torch.arange(num_pages, dtype=torch.int32, device=dev)
        self.table = torch.full((max_seqs, -(-self.max_len // page_size)), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(max_seqs, dtype=torch.int32, device=dev)
        self.host_lens = [0] * max_seqs
        self.prefix_table = torch.full((-(-self.max_prefix // page_size),), -1, dtype=torch.int32, device=dev)
        self.prefix_len = torch.zeros(1, dtype=torch.int32, device=dev)
        self.prefix_pages, self.prefix_slots = self.prefix_table[:0], torch.zeros(0, dtype=torch.int32, device=dev)
        self.host_prefix = 0
        self.used = 0

    def state(self):
        """What the cache counts; set_state takes it back to that."""
        return (self.lens, self.host_lens, self.prefix_len, self.prefix_pages, self.prefix_slots, self.host_prefix,
                self.used)

    def set_state(self, state):
        (self.lens, self.host_lens, self.prefix_len, self.prefix_pages, self.prefix_slots, self.host_prefix,
         self.used) = state

    def _take(self, need):
        """Refuses what cannot be had before anything is enqueued."""
        if self.used + need > self.free.numel():
            raise ValueError(f"{need} pages needed, {self.free.numel() - self.used} left")
        if self.lens.is_cuda and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("PagedCache.add cannot be captured into a graph: its counts come from the host")

    def add(self, new_lens):
        """Room for new_lens[s] more tokens of each sequence: the PagedPlan of
        their rows, in order of the sequences (positions count from the end of the
        prefix). The counts are copied from the host, so a graph cannot hold this
        call (or prefill and decode, which make it)."""
        if len(new_lens) != len(self.host_lens) or any(n < 0 for n in new_lens):
            raise ValueError(f"new_lens must be {len(self.host_lens)} counts")
        total = [c + n for c, n in zip(self.host_lens, new_lens)]
        if max(total) > self.max_len:
            raise ValueError(f"a sequence would pass max_len = {self.max_len} tokens")
        p = self.page_size
        need = sum(-(-t // p) - -(-c // p) for t, c in zip(total, self.host_lens))
        self._take(need)
        new = torch.tensor(new_lens, dtype=torch.int32).to(self.lens.device)
        plan = D.qlora_paged_plan(self.lens, new, self.free[self.used:], self.table, p, sum(new_lens))
        self.lens, self.host_lens, self.used = plan.total_lens, total, self.used + need
        return plan

    def add_prefix(self, n):
        """Room for a prefix of n tokens, before any others: the PagedPlan of its
        rows."""
        if self.host_prefix or any(self.host_lens):
            raise ValueError("a prefix comes once, before the sequences' own tokens")
        if not 1 <= n <= self.max_prefix:
            raise ValueError(f"a prefix must have 1 to max_prefix = {self.max_prefix} tokens")
        need = -(-n // self.page_size)
        self._take(need)
        dev = self.lens.device
        plan = D.qlora_paged_plan(torch.zeros(1, dtype=torch.int32, device=dev),
                                  torch.tensor([n], dtype=torch.int32).to(dev), self.free[self.used:],
                                  self.prefix_table[None], self.page_size, n)
        self.prefix_len, self.prefix_slots, self.host_prefix = plan.total_lens, plan.slots, int(n)
        # the kernels are chosen by the room of the table they are given
        self.prefix_pages = self.prefix_table[:need]
        self.used += need
        return plan


def rms_norm(z, g):
    return z * torch.rsqrt(torch.mean(z * z, dim=-1, keepdim=True) + EPS) * g


# Scores that a call without gradients has in memory at a time (with their masked,
# exponential and weighted copies some 5 GB).
MOST_SCORES = 2 ** 28


def causal_attention(q, k, v, heads, prefix=None):
    """softmax(q k^T / sqrt(d)) v per sequence and head, causal; fp32.
    q, k, v: [batch, seq, hidden]. prefix: keys and values [tokens, heads, d]
    that come before every sequence. Where no gradient is wanted and the scores are
    more than MOST_SCORES, sequences or rows of one are taken in turns."""
    b, t, hd = q.shape
    d = hd // heads

    def split(z):
        return z.reshape(b, t, heads, d).permute(0, 2, 1, 3).contiguous()

    qh, kh, vh = split(q), split(k), split(v)
    if prefix is not None:
        pk, pv = (z.float().transpose(0, 1).contiguous() for z in prefix)
        pk = pk.transpose(-1, -2).contiguous()

    def rows(qr, first, kt, vr):
        """The rows from the first one on, over the keys up to their last."""
        scores = torch.matmul(qr, kt) / math.sqrt(d)
        future = torch.triu(torch.ones(scores.shape[-2:], dtype=torch.bool, device=q.device), diagonal=1 + first)
        scores = scores.masked_fill(future, float("-inf"))
        if prefix is None:
            return torch.matmul(torch.softmax(scores, dim=-1), vr)
        before = torch.matmul(qr, pk) / math.sqrt(d)
        p = torch.softmax(torch.cat((before, scores), -1), dim=-1)
        n = pv.shape[1]
        return torch.matmul(p[..., :n].contiguous(), pv) + torch.matmul(p[..., n:].contiguous(), vr)

    of_row = heads * (t + (0 if prefix is None else pv.shape[1]))
    if torch.is_grad_enabled() or b * t * of_row <= MOST_SCORES:
        o = rows(qh, 0, kh.transpose(-1, -2).contiguous(), vh)
    else:
        # whole sequences as far as they fit, else rows of one
        o, step = torch.empty_like(qh), max(1, min(t, MOST_SCORES // of_row))
        seqs = max(1, MOST_SCORES // (t * of_row))
        for s in range(0, b, seqs):
            qs, ks, vs = (z[s:s + seqs] for z in (qh, kh, vh))
            for i in range(0, t, step):
                j = min(i + step, t)
                o[s:s + seqs, :, i:j] = rows(qs[:, :, i:j].contiguous(), i,
                                             ks[:, :, :j].transpose(-1, -2).contiguous(), vs[:, :, :j].contiguous())
    return o.permute(0, 2, 1, 3).reshape(b, t, hd)


class QLoraBlock:
    """The decoder block above.  `W`, `A`, `Bm`: dicts by linear name of fp32
    device tensors (W [out, in]); g1, g2: fp32 [hidden] norm gains; s =
    alpha / r.  The rest belongs to the fused form: rope a decoder.RopeTable,
    post1 / post2 and gate1 / gate2 fp32 [hidden] gains and gates of the two
    branches, residual_scale c; giving any of them implies `fused`."""

    def __init__(self, W, A, Bm, g1, g2, s, heads, rope=None, post1=None, post2=None, gate1=None, gate2=None,
                 residual_scale=1.0, fused=None):
        self.lin = {n: QLoraLinear(W[n], A[n], Bm[n], s) for n in LINEARS}
        self.g1, self.g2 = g1.float(), g2.float()
        self.heads = int(heads)
        self.hidden = W["q"].shape[1]
        self.rope = rope
        self.post1, self.post2, self.gate1, self.gate2 = post1, post2, gate1, gate2
        self.residual_scale = float(residual_scale)
        extras = self.residual_scale != 1.0 or any(v is not None for v in (rope, post1, post2, gate1, gate2))
        self.fused = extras if fused is None else bool(fused)
        if extras and not self.fused:
            raise ValueError("rope, post norms, gates and a residual scale need the fused form")

    def parameters(self):
        """The trainable tensors: every adapter's A and B."""
        out = []
        for n in LINEARS:
            out += [self.lin[n].A, self.lin[n].B]
        return out

    def _forward(self, x):
        L = self.lin
        n1 = rms_norm(x, self.g1)
        a = causal_attention(L["q"](n1), L["k"](n1), L["v"](n1), self.heads)
        h = x + L["o"](a)
        n2 = rms_norm(h, self.g2)
        return h + L["down"](torch.nn.functional.silu(L["gate"](n2)) * L["up"](n2))

    def _fused(self, x, attend):
        """The fused form on [..., hidden]: `attend` maps the linears' bf16 q, k,
        v [tokens, heads, head_dim] to the attention's bf16 [tokens, hidden]."""
        L, c, T = self.lin, self.residual_scale, x.numel() // self.hidden
        x, n1 = norm_residual(x, None, self.g1)
        n1 = n1.reshape(T, self.hidden)
        q, k, v = (L[n].bf16(n1).view(T, self.heads, self.hidden // self.heads) for n in ("q", "k", "v"))
        o = L["o"].bf16(attend(q, k, v)).view(x.shape)
        h, n2 = norm_residual(x, o, self.g2, self.post1, self.gate1, c)
        n2 = n2.reshape(T, self.hidden)
        m = torch.nn.functional.silu(L["gate"].bf16(n2).float()) * L["up"].bf16(n2).float()
        d = L["down"].bf16(m.to(torch.bfloat16)).view(x.shape)
        return norm_residual(h, d, None, self.post2, self.gate2, c)[0]

    def _fused_forward(self, x):
        b, t, _ = x.shape

        def attend(q, k, v):
            if self.rope is not None:
                pos = torch.arange(t, dtype=torch.int32, device=x.device).repeat(b)
                q, k = rope(q, k, self.rope, pos)
            q, k, v = (z.float().view(b, t, self.hidden) for z in (q, k, v))
            return causal_attention(q, k, v, self.heads).reshape(b * t, self.hidden).to(torch.bfloat16)

        return self._fused(x, attend)

    def cache(self, num_pages, page_size, max_seqs, max_len, dtype=torch.bfloat16, max_prefix=0):
        """A PagedCache for this block."""
        return PagedCache(num_pages, page_size, self.heads, self.hidden // self.heads, max_seqs, max_len,
                          self.lin["q"].A.device, dtype, max_prefix)

    def _check_cached(self, x, cache):
        """What a cached call needs of x, the cache and the rotary table."""
        d = self.hidden // self.heads
        if not self.fused:
            raise ValueError("the cache needs a block in the fused form")
        if x.dtype not in (torch.float32, torch.bfloat16) or x.device != cache.k.device:
            raise ValueError("x must be float32 or bfloat16 and on the cache's device")
        if cache.k.shape[1] != self.heads or cache.k.shape[3] != d:
            raise ValueError(f"the cache must hold {self.heads} heads of {d}")
        if self.rope is not None and (self.rope.rot_dim > d or self.rope.turns.device != cache.k.device):
            raise ValueError(f"the rotary table must be of at most {d} elements and on the cache's device")

    def _cached(self, x, cache, add, attend):
        """_fused on the rows of the plan that add() makes, attend(plan, q, k, v).
        If that fails the cache counts the tokens it had before: what was stored
        lies behind them and is not used."""
        before = cache.state()
        plan = add()
        try:
            return self._fused(x, lambda q, k, v: attend(plan, q, k, v))
        except BaseException:
            cache.set_state(before)
            raise

    def _prompt(self, x, cache, positions, slots, q, k, v, prefix=None):
        """The attention of prompts x [batch, seq, hidden], causal and behind the
        prefix, with their keys and values stored."""
        b, t, _ = x.shape
        if self.rope is not None:
            q, k = D.qlora_rope(q, k, self.rope, positions)
        K.qlora_kv_write(None, k, v, None, None, slots, cache.rows)
        q, k, v = (z.float().view(b, t, self.hidden) for z in (q, k, v))
        return causal_attention(q, k, v, self.heads, prefix).reshape(b * t, self.hidden).to(torch.bfloat16)

    @torch.no_grad()
    def prefill_shared(self, x, cache):
        """The tokens x [seq, hidden] that all sequences of the cache share, before
        any of their own: the block's output, with their keys and values stored
        once."""
        self._check_cached(x, cache)
        if x.dim() != 2 or x.shape[1] != self.hidden:
            raise ValueError(f"prefill_shared needs x [seq, {self.hidden}]")

        def attend(plan, q, k, v):
            return self._prompt(x[None], cache, plan.positions, plan.slots, q, k, v)

        return self._cached(x, cache, lambda: cache.add_prefix(x.shape[0]), attend)

    @torch.no_grad()
    def prefill(self, x, cache):
        """The first tokens x [batch, seq, hidden] of the cache's sequences 0 ..
        batch - 1, behind the prefix if there is one: the block's output, with their
        keys and values stored."""
        self._check_cached(x, cache)
        if x.dim() != 3 or x.shape[2] != self.hidden or x.shape[0] > len(cache.host_lens) or any(cache.host_lens):
            raise ValueError(f"prefill needs x [batch, seq, {self.hidden}] and an empty cache of at least batch "
                             "sequences")
        b, t, _ = x.shape

        def attend(plan, q, k, v):
            prefix = None
            if cache.host_prefix:
                prefix = K.qlora_kv_read(cache.rows, cache.prefix_slots, dtype=torch.float32)
            return self._prompt(x, cache, self._behind(plan.positions, cache), plan.slots, q, k, v, prefix)

        new_lens = [t if s < b else 0 for s in range(len(cache.host_lens))]
        return self._cached(x, cache, lambda: cache.add(new_lens), attend)

    @staticmethod
    def _behind(positions, cache):
        """Positions counted from the prefix's first token."""
        return positions + cache.host_prefix if cache.host_prefix else positions

    @torch.no_grad()
    def decode(self, x, cache):
        """One more token x [sequences, hidden] for every sequence of the cache:
        the block's output."""
        S = len(cache.host_lens)
        self._check_cached(x, cache)
        if tuple(x.shape) != (S, self.hidden):
            raise ValueError(f"decode needs x [{S}, {self.hidden}]")

        def attend(plan, q, k, v):
            q = K.qlora_kv_write(q, k, v, self.rope, self._behind(plan.positions, cache), plan.slots, cache.rows)
            if cache.host_prefix:
                o = K.qlora_prefix_attention(q, cache.rows, cache.prefix_pages, cache.prefix_len, cache.table, cache.lens)
            elif cache.rows.k_scale is not None:
                o = K.qlora_kv_attention(q, cache.rows, cache.table, cache.lens)
            else:
                o = D.qlora_paged_attention(q, cache.k, cache.v, cache.table, cache.lens)
            return o.view(S, self.hidden)

        return self._cached(x, cache, lambda: cache.add([1] * S), attend)

    def __call__(self, x, checkpoint=False):
        """x: fp32 [batch, seq, hidden] -> y (same shape)."""
        if x.shape[-1] != self.hidden:
            raise ValueError(f"x must end in the hidden size {self.hidden}")
        if self.fused:
            if checkpoint:
                return torch.utils.checkpoint.checkpoint(self._fused_forward, x, use_reentrant=False)
            return self._fused_forward(x)
        if checkpoint:
            return torch.utils.checkpoint.checkpoint(self._forward, x, use_reentrant=False)
        return self._forward(x)

    def weight_bytes(self):
        """HBM bytes of the seven quantised weights (codes and constants)."""
        return sum(self.lin[n].storage_bytes() for n in LINEARS)

    def adapter_bytes(self):
        """HBM bytes of the bf16 adapters."""
        return sum(p.numel() * p.element_size() for p in self.parameters())
