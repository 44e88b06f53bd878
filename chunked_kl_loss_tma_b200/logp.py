"""Torch-facing calls of the operators on token log-probabilities: scoring, the
clipped policy loss and the preference loss, with their gradients (see
include/chunked_kl.h for what each computes and which rows take part).

    r = logp_fwd(H, W, ids, want_entropy=True)            # r["logp"], r["entropy"]
    out = policy_fwd_bwd(H, W, ids, adv, old_logp=old, ref_logp=ref, kl_coef=0.02)
    out["loss"], out["dH"], out["dW"]

    loss = fused_preference_loss(H, W, ids, cu_seqlens, ref_logp=ref)   # autograd
    loss.backward()                                                     # H.grad, W.grad

H [N, d] (its rows may lie apart, as in a slice) and W [V, d] are bfloat16.  ids [N]
are int32 or int64.  A row takes no part when mask is 0 there, its id is negative
(-1, -100) or it lies outside the packed sequences of cu_seqlens; its outputs and
gradients are 0 and it costs no work.  A NaN in a row that takes part reaches the loss
and the gradients.  Everything is enqueued on the current stream of H's device; an id >= V
or a bad offset shows in status(out["workspace"])."""
from __future__ import annotations

import torch
from torch.autograd.graph import increment_version

from . import _lib as L
from .ops import _need, _ptr, _workspace, on_device


def _rows(t, name, dev, n):
    return _need(t, name, torch.float32, dev, shape=(n,))


def _row_distance(H):
    """Values from one row of H to the next, 0 where it is contiguous."""
    if H.is_contiguous():
        return 0
    ldH = H.stride(0)  # rows at a distance: a slice of a wider tensor, say
    if H.stride(1) != 1 or ldH < H.shape[1] or ldH % 8:
        raise ValueError("the rows of H must be contiguous, a multiple of 8 values apart")
    return ldH


def make_logp_problem(H, W, ids, *, T=1.0, mask=None, chunk_tokens=0, want_entropy=False,
                      keep_chunk=False, cu_seqlens=None, dW_dtype=torch.float32):
    """Fill a kl_logp_problem from tensors.  Returns (problem, tensors kept alive)."""
    if not isinstance(H, torch.Tensor) or not H.is_cuda:
        raise ValueError("H must be a CUDA tensor")
    dev = H.device
    if H.dtype != torch.bfloat16:
        raise TypeError("H must be bfloat16")
    _need(W, "W", H.dtype, dev)
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1]:
        raise ValueError("H must be [N, d] and W [V, d]")
    ldH = _row_distance(H)
    N = H.shape[0]
    _need(ids, "ids", None, dev, shape=(N,))
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64")
    if mask is not None and mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    _need(mask, "mask", torch.uint8, dev, shape=(N,))
    if dW_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dW_dtype must be float32 or bfloat16")
    T_row, n_seqs = None, 0
    if isinstance(T, torch.Tensor):
        T_row, T = _rows(T, "T", dev, N), 1.0
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [n_seqs + 1]")
        n_seqs = cu_seqlens.numel() - 1
    p = L.KLLogpProblem(
        N, H.shape[1], W.shape[0], L.KL_DTYPE_BF16,
        L.KL_DTYPE_F32 if dW_dtype == torch.float32 else L.KL_DTYPE_BF16, H.data_ptr(),
        W.data_ptr(), ids.data_ptr(), ids.dtype == torch.int64, bool(want_entropy), _ptr(mask), T,
        bool(keep_chunk), _ptr(T_row), chunk_tokens, _ptr(cu_seqlens), n_seqs, ldH)
    return p, [H, W, ids, mask, T_row, cu_seqlens]


class _Call:
    """Problem, workspace and stream of one call (or of a forward and its backward)."""

    def __init__(self, entry, workspace, H, W, ids, **kw):
        self.p, self.keep = make_logp_problem(H, W, ids, **kw)
        self.dev, self.N = H.device, H.shape[0]
        if workspace is None:
            n = L.kl_logp_workspace_bytes(self.p, entry)
            if n == 0:
                raise ValueError("invalid problem (kl_logp_workspace_bytes returned 0)")
            workspace = torch.empty(n, dtype=torch.uint8, device=self.dev)
            self.head = (workspace.data_ptr(), n)
        else:
            self.head = (workspace.data_ptr(), _workspace(workspace, self.dev))
        self.ws = workspace

    def rebind(self, H, W, ids, mask, T_row, cu_seqlens):
        """The same problem with its tensors where they are now: saved tensors may have come
        back at other addresses (a head that was freed and gathered again, hooks that keep
        them on the host)."""
        p = self.p
        p.ldH = _row_distance(H)
        p.H, p.W, p.ids, p.mask, p.T_row, p.cu_seqlens = map(
            _ptr, (H, W, ids, mask, T_row, cu_seqlens))
        self.keep = H, W, ids, mask, T_row, cu_seqlens

    def new(self, *shape):
        return torch.empty(shape, dtype=torch.float32, device=self.dev)

    def rows(self, n):
        """n tensors [N] of one allocation."""
        return self.new(n, self.N).unbind(0)

    def run(self, name, *args):
        """Enqueue on the current stream of H's device, with that device current."""
        on_device(self.dev, name, self.p, *args)


def _grads(c, H, W, dW, dW_dtype, accumulate, need_dH, need_dW):
    """dH and dW to write, None for one that is not wanted."""
    if not (need_dH or need_dW):
        raise ValueError("neither dH nor dW is wanted")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate_dW: pass the dW to add to")
        if need_dW:
            dW = torch.empty(W.shape, dtype=dW_dtype, device=c.dev)
    elif not need_dW:
        raise ValueError("a dW to write, but need_dW is False")
    else:
        _need(dW, "dW", dW_dtype, c.dev, shape=W.shape)
        increment_version(dW)  # written through its address: autograd is told
    return torch.empty(H.shape, dtype=H.dtype, device=c.dev) if need_dH else None, dW


def _dW_type(dW, dW_dtype):
    return dW_dtype if dW_dtype is not None else torch.float32 if dW is None else dW.dtype


def logp_fwd(H, W, ids, *, want_entropy=False, workspace=None, **kw):
    """Log-probabilities (and entropies) of the rows' tokens.  Options: T (number or
    float32 [N]), mask, cu_seqlens, chunk_tokens, keep_chunk.  Returns dict(logp,
    entropy, lse, workspace)."""
    return _logp(_Call(L.KL_ENTRY_FWD, workspace, H, W, ids, want_entropy=want_entropy, **kw))


def _logp(c):
    # each with storage of its own: autograd refuses in-place changes of an output that
    # is a view
    logp, lse, ent = c.new(c.N), c.new(c.N), c.new(c.N) if c.p.entropy else None
    c.run("kl_logp_fwd", *c.head, logp.data_ptr(), _ptr(ent), lse.data_ptr())
    return dict(logp=logp, entropy=ent, lse=lse, workspace=c.ws)


def logp_bwd(H, W, ids, lse, g_logp, *, g_entropy=None, entropy=None, grad_loss=None, dW=None,
             accumulate_dW=False, dW_dtype=None, need_dH=True, need_dW=True, workspace=None, **kw):
    """Gradients for dL/dlogp = g_logp [N] (and dL/dentropy = g_entropy [N], with the
    forward's entropy), times the device scalar grad_loss (default 1).  dW: float32
    by default, or bfloat16 rounded once.  need_dH, need_dW False: that gradient is
    not computed (None).  keep_chunk: pass the workspace of the forward, once.
    Returns dict(dH, dW, workspace)."""
    if kw.get("keep_chunk") and workspace is None:
        raise ValueError("keep_chunk: pass the workspace of the forward call")
    dW_dtype = _dW_type(dW, dW_dtype)
    c = _Call(L.KL_ENTRY_BWD, workspace, H, W, ids, dW_dtype=dW_dtype, **kw)
    for t, name in ((lse, "lse"), (g_logp, "g_logp")):
        if t is None:
            raise ValueError(f"{name} is required")
        _rows(t, name, c.dev, c.N)
    _rows(g_entropy, "g_entropy", c.dev, c.N)
    _rows(entropy, "entropy", c.dev, c.N)
    if g_entropy is not None and entropy is None:
        raise ValueError("g_entropy needs the forward's entropy")
    dH, dW = _grads(c, H, W, dW, dW_dtype, accumulate_dW, need_dH, need_dW)
    _backward(c, lse, entropy, g_logp, g_entropy, grad_loss, dH, dW, accumulate_dW)
    return dict(dH=dH, dW=dW, workspace=c.ws)


def _backward(c, lse, entropy, g_logp, g_entropy, grad_loss, dH, dW, accumulate=False):
    if grad_loss is not None:
        if grad_loss.dtype != torch.float32:
            grad_loss = grad_loss.to(torch.float32)
        if grad_loss.numel() != 1 or grad_loss.device != c.dev:
            raise ValueError(f"grad_loss must be a scalar on {c.dev}")
    c.run("kl_logp_bwd", *c.head, lse.data_ptr(), _ptr(entropy), g_logp.data_ptr(),
          _ptr(g_entropy), _ptr(grad_loss), _ptr(dH), _ptr(dW), accumulate)


def _policy(c, advantage, old_logp, ref_logp, row_weight, clip_low, clip_high, dual_clip, kl_coef,
            entropy_coef, normalizer):
    if advantage is None:
        raise ValueError("advantage is required")
    if kl_coef and ref_logp is None:
        raise ValueError("kl_coef needs ref_logp")
    dev, n = c.dev, c.N
    c.keep += (advantage, old_logp, ref_logp, row_weight)
    return L.KLPolicy(_ptr(_rows(advantage, "advantage", dev, n)),
                      _ptr(_rows(old_logp, "old_logp", dev, n)),
                      _ptr(_rows(ref_logp, "ref_logp", dev, n)),
                      _ptr(_rows(row_weight, "row_weight", dev, n)), clip_low, clip_high,
                      dual_clip, kl_coef, entropy_coef, normalizer)


def policy_fwd(H, W, ids, advantage, *, old_logp=None, ref_logp=None, row_weight=None,
               clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0,
               normalizer=0.0, want_entropy=False, workspace=None, **kw):
    """Clipped policy loss, forward only.  Returns dict(loss, row_loss, logp, entropy,
    lse, g_logp, g_entropy, workspace): g_* are the loss's derivatives for logp_bwd."""
    c = _Call(L.KL_ENTRY_FWD, workspace, H, W, ids,
              want_entropy=want_entropy or entropy_coef != 0, **kw)
    return _policy_fwd(c, _policy(c, advantage, old_logp, ref_logp, row_weight, clip_low,
                                  clip_high, dual_clip, kl_coef, entropy_coef, normalizer))


def _policy_fwd(c, q):
    o = dict(loss=c.new(), row_loss=c.new(c.N), logp=c.new(c.N),
             entropy=c.new(c.N) if c.p.entropy else None, lse=c.new(c.N), g_logp=c.new(c.N),
             g_entropy=c.new(c.N) if q.entropy_coef != 0 else None)
    c.run("kl_policy_fwd", q, *c.head, *(_ptr(t) for t in o.values()))
    return dict(o, workspace=c.ws)


def policy_fwd_bwd(H, W, ids, advantage, *, old_logp=None, ref_logp=None, row_weight=None,
                   clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0,
                   normalizer=0.0, want_entropy=False, grad_loss=1.0, dW=None,
                   accumulate_dW=False, dW_dtype=None, need_dH=True, need_dW=True, workspace=None,
                   **kw):
    """Clipped policy loss, forward and backward in one pass (no logits recomputed).
    dW, need_dH, need_dW as logp_bwd.  Returns dict(loss, row_loss, logp, entropy, dH,
    dW, workspace)."""
    dW_dtype = _dW_type(dW, dW_dtype)
    c = _Call(L.KL_ENTRY_FWD_BWD, workspace, H, W, ids,
              want_entropy=want_entropy or entropy_coef != 0, dW_dtype=dW_dtype, **kw)
    q = _policy(c, advantage, old_logp, ref_logp, row_weight, clip_low, clip_high, dual_clip,
                kl_coef, entropy_coef, normalizer)
    dH, dW = _grads(c, H, W, dW, dW_dtype, accumulate_dW, need_dH, need_dW)
    loss = c.new()
    row_loss, logp, ent = c.rows(3) if c.p.entropy else (*c.rows(2), None)
    c.run("kl_policy_fwd_bwd", q, *c.head, grad_loss, loss.data_ptr(), row_loss.data_ptr(),
          logp.data_ptr(), _ptr(ent), _ptr(dH), _ptr(dW), accumulate_dW)
    return dict(loss=loss, row_loss=row_loss, logp=logp, entropy=ent, dH=dH, dW=dW,
                workspace=c.ws)


def _preference(c, pairs, ref_logp=None, beta=0.1, loss="sigmoid", label_smoothing=0.0, margin=0.0,
                average=False, normalizer=0.0):
    if loss not in L.KL_PREFERENCE:
        raise ValueError(f"unknown loss {loss!r}")
    S = int(c.p.n_seqs)
    if pairs is not None:
        _need(pairs, "pairs", torch.int32, c.dev)
        if pairs.dim() != 2 or pairs.shape[1] != 2:
            raise ValueError("pairs must be [P, 2]")
        P = pairs.shape[0]
    else:
        if S % 2:
            raise ValueError("without pairs the number of sequences must be even")
        P = S // 2
    _need(ref_logp, "ref_logp", torch.float32, c.dev, shape=(S,))
    c.keep += (pairs, ref_logp)
    at = _ptr(pairs)
    if at == 0:  # no pairs: an address that is not read, since NULL asks for the default ones
        at = c.p.cu_seqlens
    return L.KLPreference(at, P, _ptr(ref_logp), L.KL_PREFERENCE[loss],
                          int(bool(average)), beta, label_smoothing, margin, normalizer)


def _preference_fwd(c, q):
    logp, lse, g_logp = c.rows(3)
    o = dict(loss=c.new(), pair_loss=c.new(q.n_pairs), seq_logp=c.new(c.p.n_seqs), logp=logp,
             lse=lse, g_logp=g_logp)
    c.run("kl_preference_fwd", q, *c.head, *(t.data_ptr() for t in o.values()))
    return dict(o, workspace=c.ws)


def preference_fwd(H, W, ids, cu_seqlens, pairs=None, *, workspace=None, T=1.0, mask=None,
                   chunk_tokens=0, keep_chunk=False, dW_dtype=torch.float32, **options):
    """Preference loss over packed sequences.  cu_seqlens int32 [S + 1]; pairs int32
    [P, 2] of (chosen, rejected) sequences, or None: the first half of the sequences
    is chosen, the second rejected.  Options: ref_logp float32 [S], beta (0.1), loss
    "sigmoid", "squared" (or "ipo") or "hinge", label_smoothing, margin, average,
    normalizer.  Returns dict(loss, pair_loss, seq_logp, logp, lse, g_logp,
    workspace)."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    c = _Call(L.KL_ENTRY_FWD, workspace, H, W, ids, cu_seqlens=cu_seqlens, T=T, mask=mask,
              chunk_tokens=chunk_tokens, keep_chunk=keep_chunk, dW_dtype=dW_dtype)
    return _preference_fwd(c, _preference(c, pairs, **options))


def preference_fwd_bwd(H, W, ids, cu_seqlens, pairs=None, *, grad_loss=None, dW=None,
                       accumulate_dW=False, dW_dtype=None, need_dH=True, need_dW=True,
                       workspace=None, T=1.0, mask=None, chunk_tokens=0, **options):
    """Preference loss, forward and backward (options as preference_fwd; dW, grad_loss,
    need_dH, need_dW as logp_bwd).  Every sequence's score is needed before any
    gradient, so rows beyond the first chunk (8192 by default) are projected twice; a
    chunk_tokens of N or more avoids that.  Returns dict(loss, pair_loss, seq_logp,
    logp, dH, dW, workspace)."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    dW_dtype = _dW_type(dW, dW_dtype)
    c = _Call(L.KL_ENTRY_FWD_BWD, workspace, H, W, ids, cu_seqlens=cu_seqlens, T=T, mask=mask,
              chunk_tokens=chunk_tokens, keep_chunk=True, dW_dtype=dW_dtype)
    q = _preference(c, pairs, **options)
    dH, dW = _grads(c, H, W, dW, dW_dtype, accumulate_dW, need_dH, need_dW)
    f = _preference_fwd(c, q)
    _backward(c, f["lse"], None, f["g_logp"], None, grad_loss, dH, dW, accumulate_dW)
    return dict(loss=f["loss"], pair_loss=f["pair_loss"], seq_logp=f["seq_logp"], logp=f["logp"],
                dH=dH, dW=dW, workspace=c.ws)


# ---------------------------------------------------------------- autograd
class _Once(torch.autograd.Function):
    """A gradient under create_graph: it depends on H and W, but not differentiably."""

    @staticmethod
    def forward(ctx, grad, *inputs):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("the fused losses have no second derivatives")


def _kinds(ts):
    return [None if t is None else (t.shape, t.get_device(), t.dtype) for t in ts]


def _check_saved(ts, kinds):
    """Saved tensors are what they were, wherever they are now (hooks may have moved them)."""
    if _kinds(ts) != kinds:
        for t, k in zip(ts, kinds):
            if t is not None and t.dtype != k[2]:
                raise TypeError(f"a saved tensor came back as {t.dtype}, not {k[2]}")
        raise ValueError("a saved tensor came back with another shape or on another device")
    for t in ts[1:]:  # rows of H may lie apart
        if t is not None and not t.is_contiguous():
            raise ValueError("a saved tensor came back with gaps")


class _Fused(torch.autograd.Function):
    """Forward run(call) with the row gradients of a scalar loss (or, without "loss",
    logp and entropy themselves); backward kl_logp_bwd, from the kept chunk the first
    time and recomputing every chunk when called again.  Both may be captured into a CUDA
    graph.  As for any operator of PyTorch, no eager graph of the same leaves that began on
    the default stream may live then: autograd would wait on that stream, and the
    capture ends with an error (policy_fwd_bwd and preference_fwd_bwd have no such rule)."""

    @staticmethod
    def forward(ctx, H, W, call, run):
        f = run(call)
        ctx.call, ctx.kept = call, bool(call.p.keep_chunk)
        ctx.captured = torch.cuda.is_current_stream_capturing()
        ctx.scalar = "loss" in f
        ctx.set_materialize_grads(False)  # an entropy that no loss uses costs no pass
        # ids, mask, T and cu_seqlens too: the backward reads them again
        saved = (H, W, f["lse"], f.get("entropy"), f.get("g_logp"), f.get("g_entropy"),
                 *call.keep[2:6])
        ctx.save_for_backward(*saved)
        ctx.kinds = _kinds(saved)
        call.keep = None  # from here on autograd's saved tensors are what is held and read
        if not ctx.kept:
            call.ws = call.head = None
        if ctx.scalar:
            return f["loss"]
        return (f["logp"], f["entropy"]) if f["entropy"] is not None else f["logp"]

    @staticmethod
    def backward(ctx, g, g_ent=None):
        # refuses inputs that changed in place since the forward
        saved = ctx.saved_tensors
        _check_saved(saved, ctx.kinds)
        H, W, lse, ent, g_logp, g_entropy, *rest = saved
        c, scale = ctx.call, g
        c.rebind(H, W, *rest)
        if not ctx.scalar:
            scale = None
            g_logp, g_entropy = (t if t is None else t.to(torch.float32).contiguous()
                                 for t in (g, g_ent))
            if g_logp is None:
                g_logp = c.new(c.N).zero_()
        # No kept chunk (any more).  A backward captured apart from its forward is replayed
        # without it, and may not use up what the forward left.
        if not ctx.kept or torch.cuda.is_current_stream_capturing() != ctx.captured:
            c.p.keep_chunk = 0
            n = L.kl_logp_workspace_bytes(c.p, L.KL_ENTRY_BWD)
            c.ws = torch.empty(n, dtype=torch.uint8, device=c.dev)
            c.head = (c.ws.data_ptr(), n)
        need_dH, need_dW = ctx.needs_input_grad[:2]
        dH, dW = _grads(c, H, W, None, W.dtype, False, need_dH, need_dW)
        _backward(c, lse, ent, g_logp, g_entropy, scale, dH, dW)
        ctx.kept = False
        c.ws, c.head, c.keep = None, None, None  # freed now; a second backward takes a new one
        if torch.is_grad_enabled():
            dH, dW = (t if t is None else _Once.apply(t, H, W, g, g_ent) for t in (dH, dW))
        return dH, dW, None, None


def _constants(**rows):
    """Refuses row inputs that require grad: the losses differentiate H and W alone."""
    if torch.is_grad_enabled():
        for name, t in rows.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{name} requires grad, but gradients reach H and W alone: pass "
                                 f"{name}.detach()")


def _fused(run, H, W, ids, keep_chunk, **kw):
    _constants(T=kw["T"])
    keep = keep_chunk and torch.is_grad_enabled() and (H.requires_grad or W.requires_grad)
    entry = L.KL_ENTRY_FWD_BWD if keep else L.KL_ENTRY_FWD
    c = _Call(entry, None, H.detach(), W.detach(), ids, keep_chunk=keep, dW_dtype=W.dtype, **kw)
    return c, lambda: _Fused.apply(H, W, c, run)


def fused_logp(H, W, ids, *, want_entropy=False, keep_chunk=True, T=1.0, mask=None,
               chunk_tokens=0, cu_seqlens=None):
    """Differentiable log-probabilities [N] (with want_entropy: and entropies [N]) with
    respect to H and W.  keep_chunk: the workspace of both passes
    (kl_logp_workspace_bytes, KL_ENTRY_FWD_BWD) stays allocated until the backward, which
    takes the first chunk's logits from it and recomputes the other chunks only.  False:
    nothing stays but a few numbers per row, and every chunk is recomputed.  A T that
    requires grad is refused."""
    _, apply = _fused(_logp, H, W, ids, keep_chunk, want_entropy=want_entropy, T=T, mask=mask,
                      chunk_tokens=chunk_tokens, cu_seqlens=cu_seqlens)
    return apply()


def fused_policy_loss(H, W, ids, advantage, *, old_logp=None, ref_logp=None, row_weight=None,
                      clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0,
                      normalizer=0.0, keep_chunk=True, T=1.0, mask=None, chunk_tokens=0,
                      cu_seqlens=None):
    """Differentiable clipped policy loss (options as policy_fwd; keep_chunk as fused_logp).
    Row inputs that require grad are refused."""
    _constants(advantage=advantage, old_logp=old_logp, ref_logp=ref_logp, row_weight=row_weight)
    c, apply = _fused(lambda c: _policy_fwd(c, q), H, W, ids, keep_chunk,
                      want_entropy=entropy_coef != 0, T=T, mask=mask, chunk_tokens=chunk_tokens,
                      cu_seqlens=cu_seqlens)
    q = _policy(c, advantage, old_logp, ref_logp, row_weight, clip_low, clip_high, dual_clip,
                kl_coef, entropy_coef, normalizer)
    return apply()


def fused_preference_loss(H, W, ids, cu_seqlens, pairs=None, *, keep_chunk=True, T=1.0,
                          mask=None, chunk_tokens=0, **options):
    """Differentiable preference loss (options as preference_fwd; keep_chunk as fused_logp).
    Reference scores that require grad are refused."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    _constants(ref_logp=options.get("ref_logp"))
    c, apply = _fused(lambda c: _preference_fwd(c, q), H, W, ids, keep_chunk, T=T, mask=mask,
                      chunk_tokens=chunk_tokens, cu_seqlens=cu_seqlens)
    q = _preference(c, pairs, **options)
    return apply()
