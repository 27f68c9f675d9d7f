"""More rows than one pass of the joint's grids: every workgroup's later rows (loads ahead, the row sums' two buffers in
turn, sums kept over several rows, outputs in place of inputs) against the definition in 64 bits."""
import pytest
import torch

from mamba_ssm_scan_amd import norm
from tests import norm_ref as ref
from tests.test_gpu_norm import DEV, NAMES, TYPES, call, dev, problem, within

pytestmark = pytest.mark.gpu

# rows of a pass, forward and backward: 256 and 256 above width 4096, 512 and 256 above 2048, 1024 and 512 above 1024,
# 2048 and 1024 above 512, 4096 and 2048 above 128 (and below, where rows are not 16-byte aligned), 16384 and 8192
SIZES = [(530, 8192, "bf16"), (530, 8192, "f32"), (530, 8184, "mixed"), (600, 5001, "bf16"), (530, 5001, "f32"),
         (1100, 4096, "bf16"), (1100, 4096, "mixed"), (1100, 3001, "f32"), (2100, 2048, "bf16"), (2100, 1283, "f32"),
         (2100, 1283, "mixed"), (4200, 1024, "f32"), (4200, 999, "bf16"), (8300, 512, "bf16"), (8300, 130, "f32"),
         (33000, 64, "mixed"), (17000, 96, "f32"), (9001, 33, "bf16")]


def check(p, got, grads, h):
    """As the checks of test_gpu_norm.py, the 64-bit definition evaluated on the device (there are millions of entries)."""
    d = lambda k: p[k].to(DEV) if isinstance(p[k], torch.Tensor) else p[k]  # noqa: E731
    parts = d("o"), d("gate"), p["fn"], d("scale"), d("post_weight"), d("weight"), 1e-6
    for have, (want, bound), d_ in ((got, ref.forward(d("x"), *parts), ""), (grads, ref.backward(d("dh"), d("dy"), h, *parts), "d")):
        assert {k for k, v in have.items() if v is not None} == set(want)
        for k in want:
            within(have[k], want[k].cpu(), bound[k].cpu(), d_ + k)


def rows_of(t):
    return norm.M3Lines(t.data_ptr(), t.stride(0))


def handle():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T,W,types", SIZES)
def test_rows_of_later_passes(T, W, types):
    p = problem(T, W, types, seed=40)
    got = call(p)
    x = p["x"].to(DEV)
    h, y = norm.residual_norm(x, p["o"].to(DEV), gate_fn=p["fn"], out=x, **dev(p, *NAMES))
    assert h is x and torch.equal(h, got["h"]) and torch.equal(y, got["y"])
    args = (p["dh"].to(DEV), p["dy"].to(DEV), got["h"], p["o"].to(DEV))
    kw = dict(gate_fn=p["fn"], **dev(p, *NAMES))
    check(p, got, norm.residual_norm_backward(*args, **kw), got["h"])


@pytest.mark.parametrize("T,W,types", SIZES[::3])
def test_outputs_in_place(T, W, types):
    """y in place of o, dx in place of dh (the C entries' own forms): the bits of the calls with outputs apart."""
    p = problem(T, W, types, seed=41)
    got = call(p)
    d = dev(p, "x", "o", "dh", "dy", *NAMES)
    xt, ot = TYPES[types]
    j = norm._joint(xt, ot, d["x"], d["x"].device, p["fn"], d["scale"], d["post_weight"], d["weight"], 1e-6)
    lib, h, o = norm._lib(), torch.empty_like(d["x"]), d["o"].clone()
    assert lib.m3_residual_norm(j, rows_of(d["x"]), rows_of(o), rows_of(d["gate"]), rows_of(h), rows_of(o), handle()) == 0
    assert torch.equal(h, got["h"]) and torch.equal(o, got["y"])
    want = norm.residual_norm_backward(d["dh"], d["dy"], h, d["o"], gate_fn=p["fn"], **dev(p, *NAMES))
    dx, do, dg = d["dh"].clone(), torch.empty_like(o), torch.empty_like(o)
    sums = torch.empty(3, W, device=DEV)
    n = lib.m3_residual_norm_backward_workspace_size(j, 1)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert lib.m3_residual_norm_backward(j, rows_of(dx), rows_of(d["dy"]), rows_of(h), rows_of(d["o"]), rows_of(d["gate"]),
                                         rows_of(dx), rows_of(do), rows_of(dg), sums[0].data_ptr(), sums[1].data_ptr(),
                                         sums[2].data_ptr(), ws.data_ptr(), n, handle()) == 0
    for k, t in (("x", dx), ("o", do), ("gate", dg), ("weight", sums[0]), ("post_weight", sums[1]), ("scale", sums[2])):
        assert torch.equal(t, want[k]), k


@pytest.mark.parametrize("T,W", [(530, 8192), (1100, 4096), (2100, 1283), (4200, 512), (17000, 64)])
@pytest.mark.parametrize("form", ["norm", "add", "add_norm"])
def test_one_sum_a_row_or_none(T, W, form):
    """y = N(x) alone, x + o alone, and both: the forms with other numbers of sums a row."""
    p = problem(T, W, "bf16", seed=42, gate="", scale=None, post=False, pre=form != "add")
    if form == "norm":
        p["o"] = None
    got = call(p)
    h = p["x"].to(DEV) if form == "norm" else got["h"]
    g = norm.residual_norm_backward(p["dh"].to(DEV), p["dy"].to(DEV) if p["dy"] is not None else None,
                                    h if p["dy"] is not None else None, p["o"].to(DEV) if p["o"] is not None else None,
                                    **dev(p, "weight"))
    check(p, got, g, h)
