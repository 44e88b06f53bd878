"""Token data-parallel form of the loss, and host-side helpers for multi-rank runs.

The loss partitions over tokens: each rank evaluates its own shard of rows
against the shared head with no collective on the data path.  Combining the
shards takes two exchanges.  The global count of valid tokens is summed first
and passed as `normalizer`, so every rank scales its loss and gradients by the
same mean.  Then the ranks' head gradients dW and their loss shares are summed
(all-reduce), or dW is reduce-scattered into row shards, as a sharded
optimizer keeps them.  dH stays with the rank that owns the tokens.

NCCL reduces device tensors in place, also in a group of one rank (so a one-GPU
run takes the multi-GPU path); another backend (gloo) stages them through host
memory, and a group of one gloo rank exchanges nothing."""
from __future__ import annotations

import torch
import torch.distributed as dist


def shard_range(n_tokens: int, world: int, rank: int):
    """Contiguous, balanced [start, stop) token range of `rank` (sizes differ by
    at most one; together the ranges cover [0, n_tokens) exactly once)."""
    if world < 1 or not 0 <= rank < world or n_tokens < 0:
        raise ValueError("bad shard request")
    base, extra = divmod(n_tokens, world)
    start = rank * base + min(rank, extra)
    return start, start + base + (1 if rank < extra else 0)


def _world(group):
    return dist.get_world_size(group) if dist.is_initialized() else 1


def _nccl(group):
    return dist.is_initialized() and dist.get_backend(group) == "nccl"


def global_valid_count(local_count: int, group=None) -> int:
    """Sum of the ranks' valid-token counts (one all-reduce of an int64)."""
    t = torch.tensor([int(local_count)], dtype=torch.int64)
    if _nccl(group):
        t = t.cuda()
    dist.all_reduce(t, op=dist.ReduceOp.SUM, group=group)
    return int(t.item())


def max_over_ranks(value: float, group=None) -> float:
    """Max of a per-rank scalar (e.g. the elapsed time of the timed region)."""
    t = torch.tensor([float(value)], dtype=torch.float64)
    if _nccl(group):
        t = t.cuda()
    dist.all_reduce(t, op=dist.ReduceOp.MAX, group=group)
    return float(t.item())


def dW_shard_rows(V: int, world: int, rank: int):
    """Rows [start, stop) of dW that `rank` holds after a reduce-scatter: V
    padded up to a multiple of `world`, equal blocks in rank order (the last
    block may hold fewer real rows)."""
    per = -(-V // world)
    start = min(rank * per, V)
    return start, min(start + per, V)


def sum_over_ranks(t: torch.Tensor, group=None, async_op: bool = False):
    """In-place sum of `t` over the ranks.  With NCCL and async_op, returns the
    work handle to wait on; otherwise the sum is complete on return."""
    if not dist.is_initialized() or (dist.get_world_size(group) == 1 and not _nccl(group)):
        return None
    if _nccl(group):
        return dist.all_reduce(t, op=dist.ReduceOp.SUM, group=group, async_op=async_op)
    h = t.detach().to("cpu")
    dist.all_reduce(h, op=dist.ReduceOp.SUM, group=group)
    t.copy_(h)
    return None


def reduce_scatter_rows(t: torch.Tensor, group=None) -> torch.Tensor:
    """Sum of `t` [V, ...] over the ranks, returning this rank's block of rows
    (dW_shard_rows); a copy padded to the block size."""
    world = dist.get_world_size(group) if dist.is_initialized() else 1
    rank = dist.get_rank(group) if dist.is_initialized() else 0
    if world == 1 and not _nccl(group):
        return t
    V = t.shape[0]
    per = -(-V // world)
    if per * world != V:
        pad = torch.zeros((per * world - V,) + tuple(t.shape[1:]), dtype=t.dtype, device=t.device)
        t = torch.cat([t, pad])
    if _nccl(group):
        out = torch.empty((per,) + tuple(t.shape[1:]), dtype=t.dtype, device=t.device)
        dist.reduce_scatter_tensor(out, t.contiguous(), op=dist.ReduceOp.SUM, group=group)
        a, b = dW_shard_rows(V, world, rank)
        return out[: b - a]
    h = t.detach().to("cpu").contiguous()
    dist.all_reduce(h, op=dist.ReduceOp.SUM, group=group)
    a, b = dW_shard_rows(V, world, rank)
    return h[a:b].to(t.device)


def dp_kl_fwd_bwd(H, W, *, group=None, grad_loss=1.0, mask=None, reduce="all_reduce",
                  dW=None, workspace=None, **kw):
    """Fused forward + backward of this rank's token shard H [n_r, d] against
    the shared head W, combined over the ranks of `group`.

    The normaliser is the global count of valid tokens (mask = 1 rows over all
    ranks), so the sum over ranks of the shard losses is the loss of the whole
    batch.  Returns dict(loss = the whole batch's loss, dH = this shard's rows,
    dW = the summed head gradient (reduce="all_reduce"), this rank's block of
    rows of it (reduce="reduce_scatter", rows dW_shard_rows(V, world, rank)) or
    the local gradient (reduce="none"), n_valid = the global count, workspace).
    accumulate_dW adds this rank's share to dW before the exchange: dW has to hold this
    rank's own sums then (of calls with reduce="none"), not the ranks'."""
    from . import ops

    if reduce not in ("all_reduce", "reduce_scatter", "none"):
        raise ValueError(f"unknown reduce {reduce!r}")
    local = int(H.shape[0]) if mask is None else int(mask.sum().item())
    n_all = global_valid_count(local, group) if dist.is_initialized() else local
    out = ops.kl_fwd_bwd(H, W, grad_loss=grad_loss, mask=mask, normalizer=float(n_all), dW=dW,
                         workspace=workspace, **kw)
    return _combine(out, reduce, n_all, group)


def _combine(out, reduce, n_all, group):
    """The ranks' shares of loss and dW joined."""
    loss = out["loss"].reshape(1)
    if out["dW"] is None:  # need_dW=False
        pass
    elif reduce == "all_reduce":
        sum_over_ranks(out["dW"], group)
    elif reduce == "reduce_scatter":
        out["dW"] = reduce_scatter_rows(out["dW"], group)
    sum_over_ranks(loss, group)
    out["loss"] = loss.reshape(())
    out["n_valid"] = n_all
    return out


def _dp(fn, n_local, H, W, args, group, reduce, normalizer, kw):
    if reduce not in ("all_reduce", "reduce_scatter", "none"):
        raise ValueError(f"unknown reduce {reduce!r}")
    if kw.get("accumulate_dW") and reduce != "none" and _world(group) > 1:
        # the exchange would sum what dW held before over the ranks again
        raise ValueError("accumulate_dW over several ranks needs reduce='none': add up every "
                         "call's share, then exchange dW once (sum_over_ranks, "
                         "reduce_scatter_rows)")
    n_all = global_valid_count(n_local, group) if dist.is_initialized() else n_local
    # a count of 0 over all ranks: no loss and no gradient, whatever the divisor
    out = fn(H, W, *args, normalizer=float(normalizer or n_all or 1), **kw)
    return _combine(out, reduce, n_all, group)


def dp_policy_fwd_bwd(H, W, ids, advantage, *, group=None, mask=None, reduce="all_reduce",
                      normalizer=None, cu_seqlens=None, **kw):
    """Policy loss, forward and backward, of this rank's token shard, combined over the
    ranks as dp_kl_fwd_bwd does.  normalizer: the whole batch's divisor; by default
    the number of rows that take part on all ranks.  reduce="all_reduce" sums dW in its
    own type (pass dW_dtype float32, the default, for fp32 sums).  Several calls into one
    dW: accumulate_dW with reduce="none", then sum_over_ranks(dW) or
    reduce_scatter_rows(dW) once."""
    from . import logp

    # the rows that the device lets take part
    N = ids.shape[0]
    keep = (ids >= 0) & (ids < W.shape[0])
    if mask is not None:
        keep &= mask.bool()
    if cu_seqlens is not None:
        row = torch.arange(N, device=ids.device)
        good = (cu_seqlens >= 0).all() & (cu_seqlens <= N).all() & (cu_seqlens.diff() >= 0).all()
        keep &= (row >= cu_seqlens[0]) & (row < cu_seqlens[-1]) & good
    return _dp(logp.policy_fwd_bwd, int(keep.sum().item()), H, W, (ids, advantage), group, reduce,
               normalizer, dict(kw, mask=mask, cu_seqlens=cu_seqlens))


def dp_preference_fwd_bwd(H, W, ids, cu_seqlens, pairs=None, *, group=None, reduce="all_reduce",
                          normalizer=None, **kw):
    """Preference loss, forward and backward, of this rank's pairs (both sequences of a
    pair on one rank), combined over the ranks.  normalizer: by default the number of
    pairs on all ranks (n_valid of the result).  A rank without pairs passes an empty
    tensor [0, 2]."""
    from . import logp

    n = pairs.shape[0] if pairs is not None else (cu_seqlens.numel() - 1) // 2
    return _dp(logp.preference_fwd_bwd, n, H, W, (ids, cu_seqlens, pairs), group, reduce,
               normalizer, kw)


def dp_clip_grad_norm_(grads, max_norm, *, sharded=(), group=None, norm_type=2.0, out=None):
    """clip_grad_norm_ where the ranks hold different parts of some gradients: `sharded`
    lists this rank's parts (its rows of a reduce-scattered dW, say), `grads` the
    tensors that are the same on every rank.  A rank that holds no part passes an empty
    tensor.  One all-reduce of 8 bytes; no synchronisation with NCCL.  out: destinations
    for grads, then for sharded.  Returns the norm over all ranks."""
    from . import clip

    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    sharded = [sharded] if isinstance(sharded, torch.Tensor) else list(sharded)
    total = None
    if sharded:
        total = clip.grad_total(sharded, norm_type=norm_type)
        if dist.is_initialized():
            part = total if _nccl(group) else total.cpu()
            if norm_type == 2:
                dist.all_reduce(part, op=dist.ReduceOp.SUM, group=group)
            else:  # magnitudes order as their bits do, with NaN, which a maximum of
                # floats may drop, above all of them
                dist.all_reduce(part.view(torch.int64), op=dist.ReduceOp.MAX, group=group)
            total = part.to(total.device)
        if grads:
            mine = clip.grad_total(grads, norm_type=norm_type)
            total = total + mine if norm_type == 2 else torch.maximum(total, mine)
    return clip.clip_grad_norm_(grads + sharded, max_norm, norm_type=norm_type, out=out,
                                total=total)
