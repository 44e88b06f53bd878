"""The oracle of the losses on rows with NaN: it reaches the loss and the row's own
gradient, as in the definitions (no GPU)."""
import numpy as np
import pytest

from oracle import logp_oracle as lo

N, D, V, ROW = 9, 6, 11, 4


def _rows(bad=False, cu=None):
    r = np.random.default_rng(0)
    H, W, ids = r.standard_normal((N, D)), r.standard_normal((V, D)), r.integers(0, V, N)
    if bad:
        H[ROW] = np.nan
    return lo.Rows(H, W, ids, 1.0, None, cu)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("where", ["H", "old_logp"])
@pytest.mark.parametrize("kw", [dict(), dict(dual_clip=1.5), dict(kl_coef=0.1)])
def test_policy(where, sign, kw):
    clean = _rows()
    old = clean.logp - 0.03
    adv = np.linspace(-1, 1.1, N)
    adv[ROW] = sign
    if where == "old_logp":
        old[ROW] = np.nan
    o = lo.policy(_rows(where == "H"), adv, old_logp=old, ref_logp=clean.logp, **kw)
    assert np.isnan(o["loss"])
    for x in (o["row_loss"], o["g"]):
        assert np.flatnonzero(np.isnan(x)).tolist() == [ROW]


@pytest.mark.parametrize("where", ["H", "ref_logp"])
@pytest.mark.parametrize("kw", [dict(), dict(loss="squared"), dict(loss="hinge"),
                                dict(loss="hinge", margin=0.2, average=True)])
def test_preference(where, kw):
    cu, ref = np.array([0, 2, 6, 7, 9]), np.zeros(4)
    if where == "ref_logp":
        ref[1] = np.nan
    o = lo.preference(_rows(where == "H", cu), cu, None, ref, **kw)
    assert np.isnan(o["loss"]) and np.isnan(o["pair_loss"]).tolist() == [False, True]
    assert np.flatnonzero(np.isnan(o["g"])).tolist() == [2, 3, 4, 5, 7, 8]
