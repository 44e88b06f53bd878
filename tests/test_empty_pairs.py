"""An explicit list of no pairs: a tensor [0, 2] has no address of its own, and must not
read as "no pairs given" (the first half of the sequences against the second)."""
from types import SimpleNamespace

import pytest
import torch

from chunked_kl_loss_tma_b200 import logp as lp

EMPTY = torch.zeros(0, 2, dtype=torch.int32)


@pytest.mark.parametrize("S", [1, 2, 3, 8])
def test_the_library_is_given_an_address(S):
    assert EMPTY.data_ptr() == 0
    cu = torch.zeros(S + 1, dtype=torch.int32)
    c = SimpleNamespace(p=SimpleNamespace(n_seqs=S, cu_seqlens=cu.data_ptr()),
                        dev=EMPTY.device, keep=[])
    for pairs in (EMPTY, torch.zeros(4, 2, dtype=torch.int32)[2:2]):
        q = lp._preference(c, pairs)
        assert q.n_pairs == 0 and q.pairs is not None


@pytest.mark.gpu
@pytest.mark.parametrize("S", [1, 2, 3])
@pytest.mark.parametrize("N", [0, 40, 2000])
def test_no_pairs(N, S):
    """Scores as ever, loss 0 and no gradient."""
    import chunked_kl_loss_tma_b200 as ck
    from chunked_kl_loss_tma_b200 import ops

    g = torch.Generator().manual_seed(N + S)
    H = torch.randn(N, 64, generator=g).bfloat16().cuda()
    W = torch.randn(300, 64, generator=g).bfloat16().cuda()
    ids = torch.randint(300, (N,), generator=g).cuda()
    cu = (torch.arange(S + 1) * (N // S)).int().cuda()
    pairs = EMPTY.cuda()
    logp = ck.logp_fwd(H, W, ids)["logp"]
    for kw in (dict(), dict(normalizer=3.0), dict(average=True, loss="hinge")):
        for t in (torch.float32, torch.bfloat16):
            out = ck.preference_fwd_bwd(H, W, ids, cu, pairs, dW_dtype=t, **kw)
            assert ops.status(out["workspace"]) == 0
            assert out["loss"].item() == 0 and out["pair_loss"].numel() == 0
            assert (out["dH"] == 0).all() and (out["dW"] == 0).all()
        for s in range(S):
            part = logp[s * (N // S):(s + 1) * (N // S)].double()
            want = (part.mean() if kw.get("average") and len(part) else part.sum()).item()
            assert out["seq_logp"][s].item() == pytest.approx(want, rel=2.0**-22, abs=1e-30)
    if N:
        h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
        ck.fused_preference_loss(h, w, ids, cu, pairs).backward()
        assert (h.grad == 0).all() and (w.grad == 0).all()
