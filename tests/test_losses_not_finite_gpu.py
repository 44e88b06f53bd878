"""NaN in rows that take part: it reaches the loss, the row's own outputs and the
gradients, and leaves the other rows' outputs as they were.  (A NaN in a row that takes
no part is not read: test_logp_gpu.py.)"""
import pytest
import torch

import chunked_kl_loss_tma_b200 as ck

pytestmark = pytest.mark.gpu
NAN = float("nan")
N, D, V, ROW = 130, 64, 500, 70


def _inputs(seed=0):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, D, generator=g) * D**-0.5).bfloat16().cuda()
    H = torch.randn(N, D, generator=g).bfloat16().cuda()
    ids = torch.randint(V, (N,), generator=g).cuda()
    return H, W, ids


def _only_row(t, want):
    """t is NaN in ROW alone and `want` elsewhere."""
    rest = torch.arange(N, device="cuda") != ROW
    assert t[ROW].isnan().all()
    assert torch.equal(t[rest], want[rest])


@pytest.mark.parametrize("where", ["H", "old_logp", "ref_logp", "advantage", "row_weight"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kw", [dict(), dict(entropy_coef=0.01), dict(dual_clip=1.5),
                                dict(kl_coef=0.1), dict(chunk_tokens=64)])
def test_policy(where, sign, kw):
    if where == "ref_logp":
        kw = dict(kw, kl_coef=0.2)
    H, W, ids = _inputs()
    logp = ck.logp_fwd(H, W, ids)["logp"]
    x = dict(H=H, old_logp=logp - 0.03, ref_logp=logp + 0.1,
             advantage=torch.linspace(-1, 1.1, N, device="cuda"),
             row_weight=torch.ones(N, device="cuda"))
    x["advantage"][ROW] = sign

    def run(x, f=ck.policy_fwd_bwd):
        x = dict(x)
        return f(x.pop("H"), W, ids, x.pop("advantage"), **x, **kw)

    clean = run(x)
    assert clean["loss"].isfinite()
    x[where] = x[where].clone()
    x[where][ROW] = NAN
    out = run(x)
    assert out["loss"].isnan()
    _only_row(out["row_loss"], clean["row_loss"])
    _only_row(out["dH"], clean["dH"])
    assert out["dW"].isnan().all()
    f = run(x, ck.policy_fwd)
    assert f["loss"].isnan() and f["g_logp"][ROW].isnan()
    assert f["g_logp"].isnan().sum() == 1
    leaf = [x["H"].clone().requires_grad_(), W.clone().requires_grad_()]
    y = {k: v for k, v in x.items() if k not in ("H", "advantage")}
    loss = ck.fused_policy_loss(*leaf, ids, x["advantage"], **y, **kw)
    loss.backward()
    assert loss.isnan() and leaf[0].grad[ROW].isnan().all() and leaf[1].grad.isnan().all()


@pytest.mark.parametrize("advantage", [1.0, 0.0, -1.0])
def test_policy_without_old_logp(advantage):
    """The ratio is then 1 whatever the log-probability; a NaN one is not hidden by it,
    nor by an advantage of 0, whose row's gradients are NaN as well."""
    H, W, ids = _inputs(1)
    H[ROW, 3] = NAN
    adv = torch.ones(N, device="cuda")
    adv[ROW] = advantage
    out = ck.policy_fwd_bwd(H, W, ids, adv)
    assert out["loss"].isnan() and out["row_loss"][ROW].isnan()
    assert out["row_loss"].isnan().sum() == 1
    assert out["dH"][ROW].isnan().all() and out["dW"].isnan().all()


def test_infinite_ratios_are_clipped():
    """Not NaN: a ratio that overflows is an ordinary clipped one, and without an
    advantage there is no surrogate, whatever the ratio."""
    H, W, ids = _inputs(2)
    logp = ck.logp_fwd(H, W, ids)["logp"]
    old = logp.clone()
    old[ROW] = float("-inf")
    for a, want in ((2.0, -2.0 * 1.25), (0.0, 0.0)):
        adv = torch.ones(N, device="cuda")
        adv[ROW] = a
        out = ck.policy_fwd_bwd(H, W, ids, adv, old_logp=old, clip_high=0.25)
        assert out["row_loss"][ROW].item() == want and (out["dH"][ROW] == 0).all()
        assert out["loss"].isfinite() and out["dW"].isfinite().all()


PREF = [dict(), dict(loss="squared"), dict(loss="hinge"), dict(loss="hinge", margin=0.3, beta=2.0),
        dict(label_smoothing=0.1), dict(average=True)]


@pytest.mark.parametrize("kw", PREF)
@pytest.mark.parametrize("where", ["H", "ref_logp"])
@pytest.mark.parametrize("more", [0, 1000])
def test_preference(kw, where, more):
    """A NaN in one sequence: its pair's loss and both its sequences' gradients; more:
    rows beyond what one CTA scores."""
    n = N + more
    g = torch.Generator().manual_seed(3)
    _, W, _ = _inputs(3)
    H = torch.randn(n, D, generator=g).bfloat16().cuda()
    ids = torch.randint(V, (n,), generator=g).cuda()
    cu = torch.tensor([0, 30, 60, 90, n], dtype=torch.int32, device="cuda")
    ref = torch.zeros(4, device="cuda")
    clean = ck.preference_fwd_bwd(H, W, ids, cu, ref_logp=ref, **kw)
    assert clean["loss"].isfinite()
    H, ref = H.clone(), ref.clone()
    if where == "H":
        H[40] = NAN  # sequence 1, in pair (1, 3)
    else:
        ref[3] = NAN
    out = ck.preference_fwd_bwd(H, W, ids, cu, ref_logp=ref, **kw)
    assert out["loss"].isnan() and out["pair_loss"][1].isnan()
    assert torch.equal(out["pair_loss"][0], clean["pair_loss"][0])
    assert out["dH"][30:60].isnan().all() and out["dH"][90:].isnan().all()
    for s in (slice(0, 30), slice(60, 90)):
        assert torch.equal(out["dH"][s], clean["dH"][s])
    assert out["dW"].isnan().all()
    pairs = torch.tensor([[0, 2], [1, 3], [2, 0]], dtype=torch.int32, device="cuda")
    f = ck.preference_fwd(H, W, ids, cu, pairs, ref_logp=ref, **kw)
    assert f["loss"].isnan() and f["pair_loss"].isnan().tolist() == [False, True, False]
    assert f["g_logp"].isnan().sum() == 30 + n - 90


@pytest.mark.parametrize("chunk", [0, 64])
@pytest.mark.parametrize("kept", [True, False])
def test_entropy_gradient(chunk, kept):
    """With a gradient for the entropies, the row's probabilities are NaN in dW too, not
    its own token's alone."""
    H, W, ids = _inputs(4)
    H[ROW, 3] = NAN
    one = torch.ones(N, device="cuda")
    kw = dict(chunk_tokens=chunk, keep_chunk=kept)
    f = ck.logp_fwd(H, W, ids, want_entropy=True, **kw)
    b = ck.logp_bwd(H, W, ids, f["lse"], one, g_entropy=one, entropy=f["entropy"],
                    workspace=f["workspace"] if kept else None, **kw)
    assert b["dH"][ROW].isnan().all() and b["dW"].isnan().all()
    assert b["dH"].isnan().sum() == D
    q = ck.policy_fwd_bwd(H, W, ids, one, entropy_coef=0.1, chunk_tokens=chunk)
    assert q["dH"][ROW].isnan().all() and q["dW"].isnan().all()
