"""What the autograd entry points do around the library's calls, with stand-ins
for these. No GPU needed."""
import pytest
import torch

from gated_delta_rule_chunk_amd import autograd


def _like(*ts):
    return tuple(None if t is None else torch.ones_like(t) for t in ts)


def _mla(mp):
    q, kv, r = torch.ones(1, 3, 2, 6), torch.ones(1, 3, 2, 8), torch.ones(1, 3, 2)
    mp.setattr(autograd, "mla_fwd", lambda q, kv, r, **_: (q[..., :4] * 2, q.sum(-1)))
    mp.setattr(autograd, "mla_bwd", lambda q, kv, r, *a, **_: _like(q, kv, r))
    return lambda *x: autograd.mla(*x), (q, kv, r)


def _chunk(mp):
    x = [torch.ones(1, 3, 2, 4) for _ in range(4)] + [torch.ones(1, 3, 2), torch.ones(1, 2, 4, 4)]
    mp.setattr(autograd, "chunk_fwd", lambda q, *a, initial_state, **_: (q * 2, initial_state * 2))
    mp.setattr(autograd, "chunk_bwd", lambda *a, initial_state, **_: _like(*a[:5], initial_state))
    return lambda *x: autograd.chunk_kda(*x[:5], initial_state=x[5])[0], x


def _prologue(mp):
    x = [torch.ones(1, 3, 2, 4) for _ in range(4)] + [torch.ones(1, 3, 2), torch.ones(2), torch.ones(8)]
    mp.setattr(autograd, "chunk_fwd_prologue", lambda q, *a, **_: (q * 2, q[:, 0]))
    mp.setattr(autograd, "chunk_bwd_prologue", lambda *a, **_: _like(*a[:7], None))
    return lambda *x: autograd.chunk_kda_prologue(*x)[0], x


def _conv(mp):
    names = ("xq", "xk", "xv", "wq", "wk", "wv", "g_logit", "beta_logit", "A_log", "dt_bias")
    x = [torch.ones(1, 3, 8) for _ in names]
    mp.setattr(autograd, "chunk_fwd_conv", lambda q, *a, **_: (q * 2, q[:, 0], (q[:, 1], q[:, 1], q[:, 2])))
    mp.setattr(autograd, "chunk_bwd_conv", lambda *a, **_: dict(zip(names, _like(*a[:10])), initial_state=None))
    return lambda *x: autograd.chunk_kda_conv(*x)[0], x


@pytest.mark.parametrize("entry", [_mla, _chunk, _prologue, _conv])
def test_gradients_of_gradients_are_refused(entry, monkeypatch):
    """There is no second-order backward. A term of a loss that needs one raises and is not lost, whether or
    not the incoming gradient needs a gradient itself."""
    f, x = entry(monkeypatch)
    leaves = [t.requires_grad_() for t in x]
    other = torch.ones(1, requires_grad=True)
    first = torch.autograd.grad(f(*leaves).sum(), leaves)
    assert all(torch.equal(g, torch.ones_like(g)) and not g.requires_grad for g in first)
    for weight in (1.0, torch.ones(1, requires_grad=True)):
        grads = torch.autograd.grad((f(*leaves) * weight).sum(), leaves, create_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(first, grads))
        for g in grads:
            with pytest.raises(RuntimeError, match="second"):
                (g.pow(2).sum() + other.sum()).backward(retain_graph=True)


@pytest.mark.parametrize("entry", [_mla, _chunk, _prologue, _conv])
def test_a_graph_of_first_gradients_alone_is_no_error(entry, monkeypatch):
    f, x = entry(monkeypatch)
    leaves = [t.requires_grad_() for t in x]
    grads = torch.autograd.grad(f(*leaves).sum(), leaves, create_graph=True)
    assert all(torch.equal(g, torch.ones_like(g)) for g in grads)
    frozen = [t.detach() for t in x[1:]]
    g, = torch.autograd.grad(f(leaves[0], *frozen).sum(), leaves[:1])
    assert torch.equal(g, torch.ones_like(g))


def test_an_incoming_gradient_off_its_alignment_is_copied(monkeypatch):
    """kda_mla_bwd takes 16-byte aligned rows; a slice that autograd hands on (here of a concatenation's
    gradient) need not be."""
    seen = []
    f, x = _mla(monkeypatch)
    monkeypatch.setattr(autograd, "mla_bwd", lambda q, kv, r, o, lse, d_o, **_: seen.append(d_o) or _like(q, kv, r))
    leaves = [t.requires_grad_() for t in x]
    o = f(*leaves)
    w = torch.arange(3.0 + o.numel())
    (torch.cat((torch.ones(3), o.flatten())) * w).sum().backward()
    assert seen[0].is_contiguous() and seen[0].data_ptr() % 16 == 0
    assert torch.equal(seen[0].flatten(), w[3:])
