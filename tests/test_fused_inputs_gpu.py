"""What the differentiable calls keep and read between forward and backward: the
tensors that autograd saved, at the addresses they have then, and nothing beside them."""
import pytest
import torch

import chunked_kl_loss_tma_b200 as ck

pytestmark = pytest.mark.gpu
N, D, V = 300, 136, 1500


def _inputs(seed=0):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, D, generator=g) * D**-0.5).bfloat16().cuda()
    H = torch.randn(N, D, generator=g).bfloat16().cuda()
    ids = torch.randint(V, (N,), generator=g).cuda()
    return H, W, ids


def _calls():
    """name -> loss(H, W, ids, mask, T, cu, keep)"""
    adv = torch.linspace(-1, 1, N, device="cuda")
    return dict(
        logp=lambda H, W, ids, mask, T, cu, keep: sum(
            x.sum() for x in ck.fused_logp(H, W, ids, want_entropy=True, mask=mask, T=T,
                                           cu_seqlens=cu, chunk_tokens=128, keep_chunk=keep)),
        policy=lambda H, W, ids, mask, T, cu, keep: ck.fused_policy_loss(
            H, W, ids, adv, mask=mask, T=T, cu_seqlens=cu, chunk_tokens=128, keep_chunk=keep),
        preference=lambda H, W, ids, mask, T, cu, keep: ck.fused_preference_loss(
            H, W, ids, cu, mask=mask, T=T, chunk_tokens=128, keep_chunk=keep))


def _arguments(seed=0):
    H, W, ids = _inputs(seed)
    mask = torch.ones(N, dtype=torch.bool, device="cuda")
    mask[2::5] = False
    cu = torch.tensor([3, 150, 290], dtype=torch.int32, device="cuda")
    return H, W, ids, mask, torch.linspace(0.7, 1.5, N, device="cuda"), cu


@pytest.mark.parametrize("name", ["logp", "policy", "preference"])
@pytest.mark.parametrize("keep", [True, False])
def test_storage_that_moved(name, keep):
    """Tensors that get other storage between the passes (as a sharded parameter does that
    is freed and gathered again): the backward reads the storage they have by then."""
    call = _calls()[name]
    want = None
    for moved in (False, True):
        H, W, *rest = _arguments()
        H.requires_grad_(), W.requires_grad_()
        loss = call(H, W, *rest, keep)
        if moved:
            old = []
            for t in (H, W, rest[2]):  # hidden states, head, temperatures
                old.append(t.data)
                t.data = t.data.clone()
            for t in old:
                t.fill_(float("nan"))
        got = torch.autograd.grad(loss, (H, W))
        if want is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
        assert all(g.isfinite().all() for g in got)


@pytest.mark.parametrize("name", ["logp", "policy", "preference"])
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("sliced", [False, True])
def test_saved_on_the_host(name, keep, sliced):
    """Saved tensors that hooks move away and back (H as a slice comes back contiguous):
    the originals may be reused."""
    call = _calls()[name]
    H, W, ids, mask, T, cu = _arguments(1)
    wide = torch.zeros(N, D + 24, device="cuda", dtype=torch.bfloat16)
    wide[:, 8:8 + D] = H

    def leaves():
        base = wide.clone().requires_grad_() if sliced else H.clone().requires_grad_()
        return base, (base[:, 8:8 + D] if sliced else base), W.clone().requires_grad_()

    base, h, w = leaves()
    want = torch.autograd.grad(call(h, w, ids, mask, T, cu, keep), (base, w))
    base, h, w = leaves()
    rest = [t.clone() for t in (ids, mask, T, cu)]
    with torch.autograd.graph.save_on_cpu():
        loss = call(h, w, *rest, keep)
    with torch.no_grad():
        base.fill_(float("nan")), w.fill_(float("nan"))
        for t in rest:
            t.zero_()
    got = torch.autograd.grad(loss, (base, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_saved_tensors_that_do_not_fit_are_refused():
    """Hooks that give back another type or a host tensor: an error, not a launch."""
    for back, error in ((lambda t: t.cpu(), ValueError),
                        (lambda t: t.double() if t.is_floating_point() else t, TypeError),
                        (lambda t: t[:-1], (ValueError, RuntimeError))):
        H, W, ids = _inputs(2)
        W.requires_grad_()
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, back):
            loss = ck.fused_logp(H, W, ids).sum()
        with pytest.raises(error):
            loss.backward()


def test_checkpointed():
    """Under activation checkpointing the forward runs again in the backward."""
    from torch.utils.checkpoint import checkpoint

    H, W, ids, mask, T, cu = _arguments(3)
    adv = torch.linspace(-1, 1, N, device="cuda")
    out = []
    for wrap in (False, True):
        h, w = H.clone().requires_grad_(), W.clone().requires_grad_()

        def body(x):
            return ck.fused_policy_loss(x * 2, w, ids, adv, mask=mask)

        loss = checkpoint(body, h, use_reentrant=False) if wrap else body(h)
        out.append((loss.detach(), *torch.autograd.grad(loss, (h, w))))
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_without_a_kept_chunk_nothing_is_held():
    """keep_chunk=False: a few numbers per row stay allocated between the passes, not the
    forward's workspace; and inputs that only the forward reads are let go."""
    H, W, ids = _inputs(4)
    W.requires_grad_()
    adv, mb = torch.ones(N, device="cuda"), 1 << 20
    ck.fused_policy_loss(H, W, ids, adv, keep_chunk=False)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    big = torch.zeros(1 << 22, device="cuda")
    weight = big[:N]
    loss = ck.fused_policy_loss(H, W, ids, adv, row_weight=weight, keep_chunk=False)
    del big, weight
    held = torch.cuda.memory_allocated() - before
    assert held < 32 * N + 8192, held
    kept = ck.fused_policy_loss(H, W, ids, adv)
    assert torch.cuda.memory_allocated() - before > mb  # the kept chunk, until its backward
    (loss + kept).backward()
    del loss, kept
    W.grad = None
    assert torch.cuda.memory_allocated() - before < 8192


def test_hooks_free_the_originals():
    """Saved tensors that hooks move to the host are not held on the device as well."""
    n = 4096
    g = torch.Generator().manual_seed(6)
    base = torch.randn(n, D, generator=g).bfloat16().cuda().requires_grad_()
    W = torch.randn(V, D, generator=g).bfloat16().cuda().requires_grad_()
    ids, adv = torch.randint(V, (n,), generator=g).cuda(), torch.ones(n, device="cuda")
    grads = []
    for hooks in (False, True):
        before = torch.cuda.memory_allocated()
        h = base * 2
        if hooks:
            with torch.autograd.graph.save_on_cpu():
                loss = ck.fused_policy_loss(h, W, ids, adv, keep_chunk=False)
        else:
            loss = ck.fused_policy_loss(h, W, ids, adv, keep_chunk=False)
        del h
        held = torch.cuda.memory_allocated() - before
        assert held < 8192 if hooks else held >= base.numel() * 2, held
        grads.append(torch.autograd.grad(loss, (base, W)))
        del loss
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_row_inputs_that_require_grad_are_refused():
    """They are constants of the losses: no gradient would reach them."""
    H, W, ids = _inputs(5)
    W.requires_grad_()
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    one, two = torch.ones(N, device="cuda"), torch.ones(2, device="cuda")
    leaf, leaf2 = one.clone().requires_grad_(), two.clone().requires_grad_()
    calls = [
        lambda x, y: ck.fused_logp(H, W, ids, T=x),
        lambda x, y: ck.fused_policy_loss(H, W, ids, x),
        lambda x, y: ck.fused_policy_loss(H, W, ids, one, old_logp=x),
        lambda x, y: ck.fused_policy_loss(H, W, ids, one, ref_logp=x, kl_coef=0.1),
        lambda x, y: ck.fused_policy_loss(H, W, ids, one, row_weight=x),
        lambda x, y: ck.fused_policy_loss(H, W, ids, one, T=x),
        lambda x, y: ck.fused_preference_loss(H, W, ids, cu, ref_logp=y),
        lambda x, y: ck.fused_preference_loss(H, W, ids, cu, T=x),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(ValueError, match="require"):
            call(leaf, leaf2)
            pytest.fail(f"call {k} was not refused")
        call(leaf.detach(), leaf2.detach()).sum().backward()
        with torch.no_grad():
            call(leaf, leaf2)
