"""clip_grad_norm_ writes through addresses: it refuses parameters, which its name may
invite, and tells autograd which tensors it changed."""
import pytest
import torch

import chunked_kl_loss_tma_b200 as ck

pytestmark = pytest.mark.gpu


def test_parameters_are_refused():
    """As sources in place and as destinations; their norm alone may be asked for."""
    model = torch.nn.Linear(40, 30).cuda()
    grads = [torch.full_like(p, 3.0) for p in model.parameters()]
    before = [p.detach().clone() for p in model.parameters()]
    for call in (lambda: ck.clip_grad_norm_(model.parameters(), 1e-3),
                 lambda: ck.clip_grad_norm_(model.weight, 1e-3),
                 lambda: ck.clip_grad_norm_(grads, 1e-3, out=list(model.parameters())),
                 lambda: ck.clip_grad_norm_(list(model.parameters()), 1e-3, out=grads),
                 lambda: ck.clip_grad_norm_([grads[0], model.bias], 1e-3)):
        for guard in (torch.enable_grad, torch.no_grad):
            with guard(), pytest.raises(ValueError, match="gradient"):
                call()
    assert all(torch.equal(a, b) for a, b in zip(before, model.parameters()))
    assert all((g == 3).all() for g in grads)
    want = torch.cat([b.double().flatten() for b in before]).norm().item()
    assert ck.grad_norm(list(model.parameters())).item() == pytest.approx(want, rel=2.0**-20)


def test_gradients_of_a_step():
    """The gradients of the same parameters, in place: those that have a graph of their
    own (create_graph) too, as torch's own clipping does."""
    for create in (False, True):
        model = torch.nn.Linear(40, 30).cuda()
        loss = model(torch.ones(5, 40, device="cuda")).square().sum()
        grads = torch.autograd.grad(loss, tuple(model.parameters()), create_graph=create)
        assert grads[0].requires_grad == create
        before = [g.detach().clone() for g in grads]
        norm = ck.clip_grad_norm_(grads, 0.5)
        want = torch.cat([b.double().flatten() for b in before]).norm().item()
        for b, g in zip(before, grads):
            assert torch.allclose(g.detach(), b * (0.5 / (want + 1e-6)), rtol=1e-5, atol=0)
        assert norm.item() == pytest.approx(want, rel=1e-6)


def test_autograd_sees_what_changed():
    """A saved tensor that is clipped before its backward is an error there."""
    for into in (False, True):
        x = torch.ones(100, device="cuda", requires_grad=True)
        y = x * 2  # saved by the square below
        loss = y.square().sum()
        if into:
            ck.clip_grad_norm_([torch.ones(100, device="cuda")], 0.1, out=[y.detach()])
        else:
            ck.clip_grad_norm_([y.detach()], 0.1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    src = torch.ones(100, device="cuda")
    at = src._version
    ck.clip_grad_norm_([src], 0.1, out=[torch.empty_like(src)])
    ck.grad_norm([src])
    assert src._version == at  # only read


def test_inference_tensors():
    """They have no version to count, and are clipped as before."""
    with torch.inference_mode():
        a = torch.full((100,), 2.0, device="cuda")
    norm = ck.clip_grad_norm_([a], 1.0)
    assert norm.item() == 20 and a[0].item() == pytest.approx(2 / 20, rel=1e-6)


def test_autograd_sees_an_accumulated_head_gradient():
    """The dW that a loss writes, likewise."""
    g = torch.Generator().manual_seed(0)
    H = torch.randn(20, 64, generator=g).bfloat16().cuda()
    W = torch.randn(100, 64, generator=g).bfloat16().cuda()
    ids, one = torch.arange(20, device="cuda"), torch.ones(20, device="cuda")
    cu = torch.tensor([0, 8, 20], dtype=torch.int32, device="cuda")
    dW = torch.zeros(100, 64, device="cuda")
    lse = ck.logp_fwd(H, W, ids)["lse"]
    for call in (lambda: ck.policy_fwd_bwd(H, W, ids, one, dW=dW, accumulate_dW=True),
                 lambda: ck.preference_fwd_bwd(H, W, ids, cu, dW=dW, accumulate_dW=True),
                 lambda: ck.logp_bwd(H, W, ids, lse, one, dW=dW)):
        at = dW._version
        call()
        assert dW._version > at
