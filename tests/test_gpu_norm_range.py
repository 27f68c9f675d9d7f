"""The joint over the range of values that m3_norm.h states: rows of entries at its ends."""
import pytest
import torch

from mamba_ssm_scan_amd import norm
from tests.test_gpu_norm import DEV, NAMES, call, check_backward, check_forward, dev, problem

pytestmark = pytest.mark.gpu

TOP, LEAST_RMS = 2.0 ** 60, 2.0 ** -48


@pytest.mark.parametrize("types", ["bf16", "mixed", "f32"])
@pytest.mark.parametrize("W", [64, 1001, 4096, 8185, 8192])
def test_full_rows_at_the_top(W, types):
    """Every entry of h and of o at +-2^60, where a row's sum of squares is 2^120 times the width."""
    p = problem(6, W, types, seed=50, gate="", scale=None)
    sign = lambda t: torch.where(t < 0, -1.0, 1.0).to(t.dtype)  # noqa: E731
    p["o"] = sign(p["o"]) * TOP
    p["x"] = sign(p["x"]) * TOP
    got = call(p)                                     # h: the rows of x, and an o of about 1 that is lost beside them
    check_forward(p, got)
    assert (got["y"].abs() > 0.1).all()
    g = norm.residual_norm_backward(p["dh"].to(DEV), p["dy"].to(DEV), got["h"], p["o"].to(DEV), **dev(p, *NAMES))
    check_backward(p, g, got["h"].cpu())
    p["x"] = torch.zeros_like(p["x"])
    p["post_weight"] = None                           # h: o itself
    got = call(p)
    check_forward(p, got)
    assert torch.equal(got["h"].cpu().float(), p["o"].float())


@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("W", [64, 1001, 8192])
def test_small_rows_beside_a_small_eps(W, eps):
    """Rows of root mean square 2^-48 and a little more, from entries of all sizes below their own."""
    p = problem(6, W, "f32", seed=51, gate="", scale=None)
    for k in ("x", "o"):
        v = p[k] * torch.exp2(-12 * torch.rand(p[k].shape, generator=torch.Generator().manual_seed(W)))
        p[k] = v * (LEAST_RMS * (1 + torch.arange(6.0)[:, None]) / v.square().mean(-1, keepdim=True).sqrt())
    for post in (p["post_weight"], None):
        p["post_weight"] = post
        got = call(p, eps=eps)
        check_forward(p, got, eps=eps)
