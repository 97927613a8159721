"""What autograd sees of a lookup whose gradient goes to a buffer, as its docstring says. The kernels are replaced by
the formula on the host."""
import pytest
import torch

import adamw_hybrid_optimizer_muon_b200 as ma


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    monkeypatch.setattr(ma, "embedding_lookup", lambda ids, table, scale=1.0, padding=None, out=None, dtype=None,
                        stream=None: table[ids] * scale)
    monkeypatch.setattr(ma, "embedding_grad", lambda ids, dy, buf, scale=1.0, padding=None, accumulate=False, ws=None,
                        stream=None: (buf if accumulate else buf.zero_()).index_add_(0, ids, dy * scale))
    monkeypatch.setattr(ma, "_sum_in_turn", lambda device, add: add())


def lookup(grad):
    table = torch.ones((5, 4), requires_grad=True)
    seen = []
    table.register_hook(lambda g: seen.append(g.clone()))
    return table, seen, ma.embedding(torch.tensor([0, 3, 3]), table, scale=2.0, grad=grad)


def test_a_returned_gradient_is_seen_by_hooks():
    table, seen, out = lookup(None)
    out.sum().backward()
    assert len(seen) == 1 and torch.equal(seen[0], table.grad) and table.grad[3].tolist() == [4.0] * 4


def test_a_gradient_in_a_buffer_is_not():
    buf = torch.zeros((5, 4))
    table, seen, out = lookup(buf)
    assert out.requires_grad
    out.sum().backward()
    assert not seen and table.grad is None and buf[3].tolist() == [4.0] * 4


def test_a_gradient_in_a_buffer_is_no_path_to_the_table():
    table, _, out = lookup(torch.zeros((5, 4)))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(out.sum(), table)


@pytest.mark.parametrize("grad", [None, torch.zeros((5, 4))])
def test_function_transforms_are_refused(grad):
    ids = torch.tensor([0, 3])
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda t: ma.embedding(ids, t, grad=grad).sum())(torch.ones((5, 4)))
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda i: ma.embedding(i, torch.ones((5, 4), requires_grad=True), grad=grad))(ids[None])


def test_not_differentiable_twice():
    table, _, out = lookup(None)
    (g,) = torch.autograd.grad((out * out).sum(), table, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), table)
