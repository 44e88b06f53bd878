"""Host logic of the data-parallel losses on two gloo ranks without a GPU: the local
call is the 64-bit oracle, the combination around it is the package's."""
import os
import socket

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

N, D, V = 26, 6, 11


def _free_port():
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    p = s.getsockname()[1]
    s.close()
    return p


def _batch(seed):
    g = torch.Generator().manual_seed(seed)
    H = torch.randn(N, D, generator=g, dtype=torch.float64)
    ids = torch.randint(V, (N,), generator=g)
    return H, ids, torch.randn(N, generator=g, dtype=torch.float64)


def _head():
    return torch.randn(V, D, generator=torch.Generator().manual_seed(99), dtype=torch.float64)


def _oracle_call(H, W, ids, adv, *, normalizer=0.0, mask=None, cu_seqlens=None, dW=None,
                 accumulate_dW=False, need_dW=True, need_dH=True):
    from oracle import logp_oracle as lo

    r = lo.Rows(H, W, ids, 1.0, mask, cu_seqlens)
    o = lo.policy(r, adv, normalizer=normalizer)
    dH, g, _, _ = r.grads(o["g"], o["h"])
    g = torch.tensor(g)
    if dW is not None:
        g = dW.add_(g) if accumulate_dW else dW.copy_(g)
    return dict(loss=torch.tensor(o["loss"]), dH=torch.tensor(dH) if need_dH else None,
                dW=g if need_dW else None)


def _whole(H, W, ids, adv):
    return _oracle_call(H, W, ids, adv)


def _accumulate(kd, rank, world):
    """Two microbatches: refused where each would be exchanged, right with one exchange of
    the sums."""
    W, dW, want, n = _head(), torch.zeros(V, D, dtype=torch.float64), 0, 2 * N
    for reduce in ("all_reduce", "reduce_scatter"):
        H, ids, adv = _batch(0)
        a, b = kd.shard_range(N, world, rank)
        with pytest.raises(ValueError, match="none"):
            kd.dp_policy_fwd_bwd(H[a:b], W, ids[a:b], adv[a:b], reduce=reduce, dW=dW,
                                 accumulate_dW=True)
        assert (dW == 0).all()
    loss = 0
    for seed in (0, 1):
        H, ids, adv = _batch(seed)
        out = kd.dp_policy_fwd_bwd(H[a:b], W, ids[a:b], adv[a:b], reduce="none", dW=dW,
                                   accumulate_dW=seed > 0, normalizer=float(n))
        loss = loss + out["loss"]
        whole = _oracle_call(H, W, ids, adv, normalizer=float(n))
        want = want + whole["dW"]
        assert torch.allclose(out["loss"], whole["loss"])
    kd.sum_over_ranks(dW)
    assert torch.allclose(dW, want)


def _one_gradient(kd, rank, world):
    """A frozen head: no dW to exchange."""
    H, ids, adv = _batch(2)
    W = _head()
    a, b = kd.shard_range(N, world, rank)
    whole = _whole(H, W, ids, adv)
    for reduce in ("all_reduce", "reduce_scatter", "none"):
        out = kd.dp_policy_fwd_bwd(H[a:b], W, ids[a:b], adv[a:b], reduce=reduce, need_dW=False)
        assert out["dW"] is None
        assert torch.allclose(out["loss"], whole["loss"])
        assert torch.allclose(out["dH"], whole["dH"][a:b])


def _count(kd, rank, world):
    """The rows that the device leaves out are not counted: tokens outside the vocabulary,
    and every row of a rank whose offsets are bad."""
    H, ids, adv = _batch(3)
    W = _head()
    ids = ids.clone()
    ids[[1, 20]] = V
    ids[[2, 21]] = V + 7
    ids[5] = -100
    whole = _whole(H, W, ids, adv)
    a, b = kd.shard_range(N, world, rank)
    out = kd.dp_policy_fwd_bwd(H[a:b], W, ids[a:b], adv[a:b])
    assert out["n_valid"] == N - 5
    assert torch.allclose(out["loss"], whole["loss"]) and torch.allclose(out["dW"], whole["dW"])
    # offsets: good on rank 0 (rows 2 to 9), bad in one of three ways on rank 1
    H, ids, adv = _batch(4)
    for bad in ([0, 9, 4], [-1, 3, 9], [0, 9, 14]):
        cu = torch.tensor([2, 5, 9] if rank == 0 else bad, dtype=torch.int32)
        seen = kd.dp_policy_fwd_bwd(H[a:b], W, ids[a:b], adv[a:b], cu_seqlens=cu)["n_valid"]
        assert seen == 7, (bad, seen)


def _worker(rank, world, port, what, q):
    from chunked_kl_loss_tma_b200 import dist as kd
    from chunked_kl_loss_tma_b200 import logp

    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        logp.policy_fwd_bwd = _oracle_call
        globals()[what](kd, rank, world)
        q.put((rank, None))
    except BaseException as e:  # report instead of leaving the parent waiting
        q.put((rank, repr(e)))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("what,world", [("_accumulate", 2), ("_one_gradient", 1),
                                        ("_one_gradient", 2), ("_count", 2)])
def test_ranks(what, world):
    ctx = mp.get_context("spawn")
    q, port = ctx.Queue(), _free_port()
    procs = [ctx.Process(target=_worker, args=(r, world, port, what, q)) for r in range(world)]
    for p in procs:
        p.start()
    res = [q.get(timeout=120) for _ in procs]
    for p in procs:
        p.join(timeout=60)
    assert all(e is None for _, e in res), res


def test_one_process_accumulates_as_before(monkeypatch):
    """Without other ranks nothing is exchanged, and dW may be added to."""
    from chunked_kl_loss_tma_b200 import dist as kd
    from chunked_kl_loss_tma_b200 import logp

    monkeypatch.setattr(logp, "policy_fwd_bwd", _oracle_call)
    H, ids, adv = _batch(5)
    W, dW = _head(), torch.ones(V, D, dtype=torch.float64)
    out = kd.dp_policy_fwd_bwd(H, W, ids, adv, dW=dW, accumulate_dW=True)
    want = _whole(H, W, ids, adv)
    assert torch.allclose(out["dW"], 1 + want["dW"]) and torch.allclose(out["loss"], want["loss"])


def test_oracle_call_is_the_sum_of_shards():
    """The stand-in itself: shards with the whole batch's count add up."""
    H, ids, adv = _batch(6)
    W = _head()
    parts = [_oracle_call(H[s], W, ids[s], adv[s], normalizer=float(N))
             for s in (slice(0, 11), slice(11, N))]
    whole = _whole(H, W, ids, adv)
    assert np.isclose(sum(p["loss"] for p in parts), whole["loss"])
    assert torch.allclose(parts[0]["dW"] + parts[1]["dW"], whole["dW"])
