"""Data-parallel losses on ranks whose shares differ in kind: one without pairs, one
without rows, several calls into one dW, a frozen head.  Two processes share one GPU and
exchange over gloo on the host (no kernel waits on the other rank's); the results are
the whole batch's, against the fp64 oracle within its bounds."""
import os
import socket

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _free_port():
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    p = s.getsockname()[1]
    s.close()
    return p


def _within(got, want, tol):
    return bool((np.abs(got.detach().double().cpu().numpy() - want) <= tol).all())


def _batch(seed, N, d, V):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, d, generator=torch.Generator().manual_seed(1)) * d**-0.5).bfloat16()
    ids = torch.randint(V, (N,), generator=g)
    H = (torch.randn(N, d, generator=g) + 4 * W[ids].float()).bfloat16()
    return H.cuda(), W.cuda(), ids.cuda(), torch.randn(N, generator=g).cuda()


def _pairs(kd, lo, rank):
    """Two pairs on rank 0; rank 1 holds sequences without a pair, then no row at all."""
    H, W, ids, _ = _batch(0, 200, 136, 1203)
    cu = torch.tensor([0, 40, 90, 120, 200], dtype=torch.int32, device="cuda")
    pairs = torch.tensor([[0, 2], [3, 1]], dtype=torch.int32, device="cuda")
    r = lo.Rows(H, W, ids, 1.0, None, cu)
    o = lo.preference(r, cu, pairs)
    dH, dW, tH, tW = r.grads(o["g"], tol_g=o["tol_g"])
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    out = []
    for n, other in ((200, cu), (0, torch.zeros(2, dtype=torch.int32, device="cuda"))):
        mine = (H, W, ids, cu, pairs) if rank == 0 else (H[:n], W, ids[:n], other, none)
        for reduce in ("all_reduce", "reduce_scatter"):
            x = kd.dp_preference_fwd_bwd(*mine, reduce=reduce)
            v = slice(0, 1203) if reduce == "all_reduce" else slice(*kd.dW_shard_rows(1203, 2, rank))
            out += [x["n_valid"] == 2,
                    _within(x["loss"], o["loss"], o["tol_loss"] + 2.0**-22 * abs(o["loss"])),
                    _within(x["dW"], dW[v], tW[v] * 1.001),
                    _within(x["dH"], dH, tH) if rank == 0 else bool((x["dH"] == 0).all())]
    return out


def _microbatches(kd, lo, rank):
    """Two calls of 301 rows each into one dW, exchanged once, then clipped; and the same
    with a frozen head."""
    N, d, V, out = 301, 136, 1203, []
    dW, want, bound = torch.empty(V, d, device="cuda"), 0, 0
    for k in range(2):
        H, W, ids, adv = _batch(2 + k, N, d, V)
        r = lo.Rows(H, W, ids)
        o = lo.policy(r, adv, normalizer=2.0 * N)
        a, b = kd.shard_range(N, 2, rank)
        mine = (H[a:b], W, ids[a:b], adv[a:b])
        x = kd.dp_policy_fwd_bwd(*mine, normalizer=2.0 * N, reduce="none", dW=dW,
                                 accumulate_dW=k > 0)
        oH, oW, tH, tW = r.grads(o["g"], o["h"], tol_g=o["tol_g"])
        want, bound = want + oW, bound + tW
        y = kd.dp_policy_fwd_bwd(*mine, normalizer=2.0 * N, need_dW=False)
        out += [_within(x["loss"], o["loss"], o["tol_loss"] + 2.0**-22 * abs(o["loss"])),
                _within(x["dH"], oH[a:b], tH[a:b]), y["dW"] is None,
                torch.equal(x["dH"], y["dH"]), torch.equal(x["loss"], y["loss"])]
    kd.sum_over_ranks(dW)
    return out + [_within(dW, want, bound * 1.001)]


def _worker(rank, world, port, what, q):
    import torch.distributed as dist

    from chunked_kl_loss_tma_b200 import dist as kd
    from oracle import logp_oracle as lo

    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        torch.cuda.set_device(0)
        q.put((rank, globals()[what](kd, lo, rank)))
    except Exception as e:  # report instead of leaving the parent waiting
        q.put((rank, repr(e)))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("what", ["_pairs", "_microbatches"])
def test_two_ranks(what):
    import torch.multiprocessing as mp

    ctx = mp.get_context("spawn")
    q, port = ctx.Queue(), _free_port()
    procs = [ctx.Process(target=_worker, args=(r, 2, port, what, q)) for r in range(2)]
    for p in procs:
        p.start()
    res = [q.get(timeout=300) for _ in procs]
    for p in procs:
        p.join(timeout=120)
        assert p.exitcode == 0
    for rank, ok in res:
        assert isinstance(ok, list) and all(ok), (rank, ok)
