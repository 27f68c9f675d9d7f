"""What the joint's Python entry refuses or says about gradients, without a GPU: the library call is replaced by one that
reports success and writes nothing."""
import warnings

import pytest
import torch

from mamba_ssm_scan_amd import norm


@pytest.fixture
def calls(monkeypatch):
    """residual_norm on CPU tensors; the calls that reached the library."""
    got = []

    class Library:
        def m3_residual_norm(self, *args):
            got.append(args)
            return 0

    monkeypatch.setattr(norm, "_device_of", lambda t, name: t.device)
    monkeypatch.setattr(norm, "_handle", lambda device: 0)
    monkeypatch.setattr(norm, "_lib", Library)
    return got


T, W = 3, 64
GIVEN = ("x", "o", "gate", "scale", "post_weight", "weight")


def tensors(*leaves):
    """All inputs; those named require grad."""
    t = {k: torch.ones(T, W) if k in ("x", "o", "gate") else torch.ones(W) for k in GIVEN}
    for k in leaves:
        t[k].requires_grad_()
    return t


@pytest.mark.parametrize("leaf", GIVEN[1:])
def test_in_place_of_the_stream_with_a_gradient_asked_for(calls, leaf):
    """h in place of x would be x with x's history: whatever input asks for a gradient would not get it."""
    t = tensors(leaf)
    before = t["x"]._version
    with pytest.raises(RuntimeError, match="out"):
        norm.residual_norm(**t, out=t["x"])
    with pytest.raises(RuntimeError, match="out"):
        norm.residual_norm(**t, out=t["x"].detach())
    assert not calls and t["x"]._version == before


@pytest.mark.parametrize("form", ["leaf", "step", "view"])
def test_an_out_that_is_part_of_a_graph(calls, form):
    """A leaf that requires grad, a step's result, a view of either: in place of x or not, whether or not other inputs do."""
    s = torch.ones(2, T, W, requires_grad=True)
    own = {"leaf": torch.ones(T, W, requires_grad=True), "step": (2 * s)[0], "view": s[1]}[form]
    t = tensors()
    with pytest.raises(RuntimeError, match="out"):
        norm.residual_norm(own, t["o"], weight=t["weight"], out=own)
    with pytest.raises(RuntimeError, match="out"):
        norm.residual_norm(t["x"], t["o"], weight=t["weight"], out=own)
    with pytest.raises(RuntimeError, match="out"):
        norm.residual_norm(own, t["o"], out=own.detach())
    assert not calls


@pytest.mark.parametrize("leaf", GIVEN)
def test_an_out_of_its_own_says_that_gradients_end(calls, leaf):
    t = tensors(leaf)
    out = torch.empty(T, W)
    with pytest.warns(UserWarning, match="out") as seen:
        h, y = norm.residual_norm(**t, out=out)
    assert seen[0].filename == __file__                      # (the caller's line)
    assert h is out and not h.requires_grad and not y.requires_grad and len(calls) == 1


def test_nothing_is_said_where_no_gradient_is_asked_for(calls):
    t = tensors(*GIVEN)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.no_grad():
            norm.residual_norm(**t, out=t["x"])
            norm.residual_norm(**t, out=torch.empty(T, W))
        with torch.inference_mode():
            norm.residual_norm(**t, out=t["x"])
        t = tensors()
        norm.residual_norm(**t, out=t["x"])
        norm.residual_norm(**t, out=torch.empty(T, W))
    assert len(calls) == 5


@pytest.mark.parametrize("dual", GIVEN)
@pytest.mark.parametrize("also", ["", "asked", "no_grad", "out"])
def test_forward_mode_is_refused(calls, dual, also):
    """An input with a tangent, which the results would not carry on; also where a gradient is asked for as well."""
    from torch.autograd import forward_ad
    t = tensors(*(GIVEN if also == "asked" else ()))
    with forward_ad.dual_level():
        t[dual] = forward_ad.make_dual(t[dual], torch.ones_like(t[dual]))
        with pytest.raises(NotImplementedError, match="forward"), torch.set_grad_enabled(also != "no_grad"):
            norm.residual_norm(**t, out=torch.empty(T, W) if also == "out" else None)
        assert not calls
        norm.residual_norm(**tensors())                      # no tangent: as ever
    assert len(calls) == 1


@pytest.mark.parametrize("dual", ["dh", "dy", "h", "o", "weight"])
def test_forward_mode_is_refused_by_the_gradients_too(calls, dual):
    from torch.autograd import forward_ad
    t = dict(dh=torch.ones(T, W), dy=torch.ones(T, W), h=torch.ones(T, W), o=torch.ones(T, W), weight=torch.ones(W))
    with forward_ad.dual_level():
        t[dual] = forward_ad.make_dual(t[dual], torch.ones_like(t[dual]))
        with pytest.raises(NotImplementedError, match="forward"):
            norm.residual_norm_backward(**t)


def test_transforms_of_functions_are_refused(calls):
    t = tensors()
    with pytest.raises(NotImplementedError, match="forward"):
        torch.func.jvp(lambda x: norm.residual_norm(x, t["o"]), (t["x"],), (t["x"],))
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda x: norm.residual_norm(x, t["o"]).sum())(t["x"])
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda x: norm.residual_norm(x[None], t["o"][:1]))(t["x"])
    assert not calls
