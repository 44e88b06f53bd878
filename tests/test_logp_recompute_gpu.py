"""Gradients whose logits are recomputed, where the token is likely: its own entry of
the logits' gradient is a (1 - p), which is formed from the other entries and keeps
its relative accuracy however near 1 the probability is."""
import numpy as np
import pytest
import torch

import chunked_kl_loss_tma_b200 as ck
from chunked_kl_loss_tma_b200 import ops
from oracle import logp_oracle as lo

pytestmark = pytest.mark.gpu


def _inputs(N, d, V, seed):
    """Log-probabilities from -1 down to -1e-6."""
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, d, generator=g) * d**-0.5).bfloat16()
    ids = torch.randint(V, (N,), generator=g)
    H = torch.randn(N, d, generator=g).bfloat16().float()
    H = (H + torch.linspace(7, 21, N)[:, None] * W[ids].float()).bfloat16()
    return H.cuda(), W.cuda(), ids.int().cuda()


def _grads(r, g, h):
    """dH, dW and bounds that are relative to 1 - p.  Every p_j of another token is off
    by tz of its value (the error of a difference of logits); the own entry is their sum,
    so it is off by tz of its value too; each entry is rounded to bf16 up to three
    times.  With an entropy term -p b (ln p + ent) beside it: ln p of the own token and
    the entropy are sums of the others' e and e x, off by tz + 2^-17 of their values (80
    fp32 roundings); ln p of another token, which is below -1, by tz, or by a rounding of
    e where it is taken from a stored one."""
    dH, dW, _, _ = r.grads(g, h)
    u, step, n = 2.0**-8, 2.0**-23, len(r.ids)
    a = g[r.keep] / r.T
    b = np.zeros(n) if h is None else h[r.keep] / r.T
    one = np.zeros_like(r.p)
    one[np.arange(n), r.ids] = 1
    tz = r.tol_logp_k[:, None]
    # |1 - p| without the cancellation of the oracle's own 64-bit difference
    share = np.where(one == 1, -np.expm1(r.lp), r.p)
    size = np.abs(a)[:, None] * share + np.abs(b)[:, None] * r.p * np.abs(
        r.lp + r.ent_k[:, None])
    off = (3 * u + 4 * u * u + 2 * tz) * size + np.abs(b)[:, None] * r.p * (
        u * (1 - one) + (tz + 2.0**-17) * (np.abs(r.lp) + r.ent_k[:, None]))
    tH = np.zeros_like(dH)
    tH[r.keep] = (off + (r.V / 16 + 40) * step * size) @ np.abs(r.W)
    tW = (off + (n / 16 + 40) * step * size).T @ np.abs(r.H)
    return dH, dW, tH + u * (np.abs(dH) + tH) + 1e-30, tW + 2.0**-24 * np.abs(dW) + 1e-30


def _near(got, want, tol, name):
    off = np.abs(got.double().cpu().numpy() - want) / tol
    assert (off <= 1).all(), f"{name}: {off.max():.2f} times its bound"


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("N,d,V", [(200, 128, 2000), (131, 520, 2051), (65, 64, 257)])
def test_likely_tokens(N, d, V, entropy):
    H, W, ids = _inputs(N, d, V, seed=N)
    mask = torch.ones(N, dtype=torch.bool, device="cuda")
    mask[3::7] = False
    r = lo.Rows(H, W, ids, 1.0, mask)
    assert r.logp_k.max() > -1e-4
    gen = torch.Generator().manual_seed(5)
    g = torch.rand(N, generator=gen) + 0.5
    h = torch.randn(N, generator=gen) if entropy else None
    want = _grads(r, g.double().numpy(), None if h is None else h.double().numpy())
    g, h = g.cuda(), None if h is None else h.cuda()
    for chunk, kept in ((0, True), (0, False), (64, True), (64, False)):
        kw = dict(mask=mask, chunk_tokens=chunk, keep_chunk=kept)
        f = ck.logp_fwd(H, W, ids, want_entropy=entropy, **kw)
        b = ck.logp_bwd(H, W, ids, f["lse"], g, g_entropy=h, entropy=f["entropy"],
                        workspace=f["workspace"] if kept else None, **kw)
        assert ops.status(b["workspace"]) == 0
        _near(b["dH"], want[0], want[2], f"dH, chunk {chunk}, kept {kept}")
        _near(b["dW"], want[1], want[3], f"dW, chunk {chunk}, kept {kept}")


def test_every_backward_of_one_forward():
    """The first backward starts from the kept chunk, the second recomputes it."""
    N, d, V = 200, 128, 2000
    H, W, ids = _inputs(N, d, V, seed=9)
    r = lo.Rows(H, W, ids)
    dH, _, tH, _ = _grads(r, np.ones(N), None)
    H.requires_grad_()
    lp = ck.fused_logp(H, W, ids)
    for k in range(2):
        got, = torch.autograd.grad(lp.sum(), H, retain_graph=True)
        _near(got, dH, tH, f"dH of backward {k}")


def test_likely_preferences():
    """Rows beyond the first chunk of a preference loss."""
    N, d, V = 200, 128, 2000
    H, W, ids = _inputs(N, d, V, seed=10)
    cu = torch.tensor([0, 50, 100, 150, 200], dtype=torch.int32, device="cuda")
    r = lo.Rows(H, W, ids, 1.0, None, cu)
    o = lo.preference(r, cu, None)
    dH, dW, tH, tW = _grads(r, o["g"], None)
    # the slopes' own errors, relative: tol_g of g
    more = np.max(o["tol_g"][r.keep] / np.abs(o["g"][r.keep]))
    out = ck.preference_fwd_bwd(H, W, ids, cu, chunk_tokens=64)
    one = np.zeros_like(r.p)
    one[np.arange(N), r.ids] = 1
    size = np.abs(o["g"])[:, None] * np.where(one == 1, -np.expm1(r.lp), r.p)
    _near(out["dH"], dH, tH + 1.01 * more * (size @ np.abs(r.W)), "dH")
    _near(out["dW"], dW, tW + 1.01 * more * (size.T @ np.abs(r.H)), "dW")
