"""What rope does about gradients in place, and what it refuses, without a GPU: the library call is replaced by one that reports success and writes
nothing."""
import pytest
import torch
from torch.autograd import forward_ad

from mamba_ssm_scan_amd import attention

T, H, D = 3, 2, 16


@pytest.fixture
def calls(monkeypatch):
    got = []

    class Library:
        def m3_rope(self, *args):
            got.append(args)
            return 0

    monkeypatch.setattr(attention, "_device_of", lambda t, name: t.device)
    monkeypatch.setattr(attention, "_handle", lambda device: 0)
    monkeypatch.setattr(attention, "_lib", Library)
    return got


def inputs():
    return torch.ones(T, H, D), torch.arange(T, dtype=torch.int32), torch.ones(D // 2)


def test_in_place_is_a_step_of_autograd(calls):
    """out = x kept x's history, of rows that were not turned. (The replaced call turns nothing, forward or backward.)"""
    x, pos, f = inputs()
    leaf = x.clone().requires_grad_()
    for t in (leaf * 2, (leaf * 2).view(T, H, D), (leaf.view(T, 2 * D) * 2).view(T, H, D)):
        before = t._version
        assert attention.rope(t, pos, f, out=t) is t
        assert t._version > before
        n = len(calls)
        torch.autograd.grad(t.sum(), leaf)
        assert len(calls) == n + 1                           # (the gradient passed through the transposed map)
    square = leaf * 2
    kept = square.square().sum()
    attention.rope(square, pos, f, out=square)
    with pytest.raises(RuntimeError, match="inplace"):
        kept.backward()


def test_out_that_autograd_would_misread(calls):
    x, pos, f = inputs()
    leaf = x.clone().requires_grad_()
    both = torch.cat([leaf, leaf]) * 2
    for t in (leaf, leaf[:], leaf.view(T, H, D), both.split(T)[0], both.unflatten(0, (2, T)).unbind(0)[1], both.chunk(2)[1][:]):
        with pytest.raises(RuntimeError, match="leaf"):
            attention.rope(t, pos, f, out=t)
    for out in (leaf, leaf * 2):
        with pytest.raises(RuntimeError, match="out"):
            attention.rope(x, pos, f, out=out)
    assert not calls
    with torch.no_grad():
        attention.rope(leaf, pos, f, out=leaf)
    attention.rope(x, pos, f, out=x)
    assert not attention.rope(leaf, pos, f, out=torch.empty(T, H, D)).requires_grad
    assert len(calls) == 3


def test_rows_that_autograd_kept_and_that_out_overwrites(calls):
    x, pos, f = inputs()
    s = torch.ones(D, requires_grad=True)
    y = (x * s).sum()
    attention.rope(x, pos, f, out=x)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()


@pytest.mark.parametrize("asked", [False, True])
def test_forward_mode_is_refused(calls, asked):
    x, pos, f = inputs()
    x.requires_grad_(asked)
    with forward_ad.dual_level():
        with pytest.raises(NotImplementedError, match="forward"):
            attention.rope(forward_ad.make_dual(x, torch.ones_like(x)), pos, f)
        with pytest.raises(NotImplementedError, match="forward"):
            attention.rope(x, pos, forward_ad.make_dual(f, torch.ones_like(f)))
    assert not calls
