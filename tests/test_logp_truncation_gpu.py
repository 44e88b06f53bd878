"""The logits' scale undoes what the tensor core's truncation takes off on average, for
products that add up evenly over the steps of 16.  Here they do not: all of a logit in
the first or the last step, and halves that cancel.

Bound.  A step truncates the accumulator towards zero, by less than 2^-23 of the largest
magnitude in it (the sum so far and the step's own products), and only where something
is added; the scale adds 1.62e-8 per step of the finished logit.  Each other token's
logit is off by at most both, the own token's (formed apart) by fp32 roundings, and the
log-probability by their average under p, beside 2^-20 for exponentials, logarithms and
sums in fp32 (as the oracle's bound)."""
import numpy as np
import pytest
import torch

import chunked_kl_loss_tma_b200 as ck

pytestmark = pytest.mark.gpu
N, V = 48, 600


def _pattern(name, d):
    g = torch.Generator().manual_seed(d)
    W = torch.randn(V, d, generator=g) * d**-0.5
    H = torch.randn(N, d, generator=g)
    ids = torch.randint(V, (N,), generator=g)
    if name in ("first step", "last step"):
        s = slice(0, 16) if name == "first step" else slice(d - 16, d)
        W[:, s] *= (d / 16)**0.5
        lean = H[:, s] + 12 * W[ids][:, s]
        H = torch.zeros(N, d)
        H[:, s] = lean
    elif name == "first step, then noise":
        W[:, :16] *= (d / 16)**0.5
        H[:, :16] += 12 * W[ids][:, :16]
        H[:, 16:] *= 0.05
    elif name == "cancelling":
        w = W[:, :d // 2]
        W = torch.cat([8 * w, -8 * w + W[:, d // 2:]], 1)
        h = H[:, :d // 2] + 3 * w[ids]
        H = torch.cat([h, h], 1)
    else:  # evenly
        H = H + 12 * W[ids]
    return H.bfloat16(), W.bfloat16(), ids


@pytest.mark.parametrize("d", [512, 4096])
@pytest.mark.parametrize("name", ["evenly", "first step", "last step", "first step, then noise",
                                  "cancelling"])
def test_log_probabilities(name, d):
    H, W, ids = _pattern(name, d)
    h, w = (x.double().numpy().reshape(len(x), d // 16, 16) for x in (H, W))
    size, so_far = np.zeros((N, V)), np.zeros((N, V))
    for k in range(d // 16):  # the steps of one accumulator
        size = np.maximum(size, np.abs(so_far) + np.abs(h[:, k]) @ np.abs(w[:, k]).T)
        so_far += h[:, k] @ w[:, k].T
    z, row = so_far, np.arange(N)
    lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
    logp, p = z[row, ids] - lse, np.exp(z - lse[:, None])
    off = d / 16 * (2.0**-23 * size + 1.62e-8 * np.abs(z))
    off[row, ids] = 0
    tol = (p * off).sum(1) * (1 + off.max(1)) + 2.0**-20 * (1 + np.abs(logp) + np.abs(lse))
    got = ck.logp_fwd(H.cuda(), W.cuda(), ids.cuda())["logp"].double().cpu().numpy()
    assert (np.abs(got - logp) <= tol).all(), (np.abs(got - logp) / tol).max()
