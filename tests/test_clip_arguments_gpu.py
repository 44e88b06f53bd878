"""clip_grad_norm_ writes through addresses: it refuses parameters, which its name may
invite."""
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
