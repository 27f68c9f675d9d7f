"""Checks of the joint's C entry points that need no GPU: what include/m3_norm.h declares is exported, the workspace, and
every refusal before any HIP call. Pointers are fake, aligned addresses, never dereferenced."""
import os
import re

import pytest

from mamba_ssm_scan_amd import binding as bd
from mamba_ssm_scan_amd import norm as nm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, G = 1 << 44, 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from mamba_ssm_scan_amd import build
        build.build()
    return nm._lib()


def place(j):
    return FAKE + 64 * j * G


def joint(**kw):
    d = dict(tokens=5, width=128, stream_dtype=0, io_dtype=1, gate_fn=1, eps=1e-6, factor=1.0, scale=place(20),
             post_weight=place(21), weight=place(22))
    d.update(kw)
    return nm.M3Joint(*[d[n] for n, _ in nm.M3Joint._fields_])


def lines(j, **kw):
    d = dict(p=place(j), stride=128)
    d.update(kw)
    return nm.M3Lines(d["p"], d["stride"])


def refused(lib, status, text, code):
    assert status == code, (status, lib.m3_last_error())
    assert text in lib.m3_last_error().decode(), lib.m3_last_error()


def test_exports_every_declared_symbol(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "m3_norm.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(m3_[a-z_]+)\s*\(", src)))
    assert names == sorted(nm.EXPORTS)
    for n in names:
        assert hasattr(lib, n)


ABSENT = object()


def forward(lib, j=None, x=None, o=None, gate=None, h=None, y=None):
    pick = lambda v, d: None if v is ABSENT else d if v is None else v  # noqa: E731
    return lib.m3_residual_norm(pick(j, joint()), pick(x, lines(0)), pick(o, lines(1)), pick(gate, lines(2)),
                                pick(h, lines(3)), pick(y, lines(4)), None)


def test_forward_refusals(lib):
    refused(lib, forward(lib, j=ABSENT), "joint is NULL", 1)
    for kw, text, code in ((dict(stream_dtype=2), "dtype", 3), (dict(io_dtype=-1), "dtype", 3),
                           (dict(stream_dtype=1, io_dtype=0), "bf16 stream", 5), (dict(tokens=-1), "tokens", 1),
                           (dict(tokens=(1 << 30) + 1), "tokens", 1), (dict(width=0), "width", 1),
                           (dict(width=8193), "width", 5), (dict(gate_fn=3), "gate function", 1),
                           (dict(eps=-1e-9), "eps", 1), (dict(eps=float("nan")), "eps", 1), (dict(eps=float("inf")), "eps", 1),
                           (dict(factor=float("inf")), "factor", 1), (dict(weight=place(22) + 2), "weight", 4)):
        refused(lib, forward(lib, j=joint(**kw)), text, code)
    refused(lib, forward(lib, x=ABSENT), "x is NULL", 1)
    refused(lib, forward(lib, o=ABSENT), "without o", 1)
    refused(lib, forward(lib, o=ABSENT, gate=ABSENT), "without o", 1)
    refused(lib, forward(lib, h=ABSENT), "h is NULL", 1)
    refused(lib, forward(lib, y=ABSENT), "together", 1)
    refused(lib, forward(lib, j=joint(weight=None)), "together", 1)
    refused(lib, forward(lib, j=joint(weight=None), o=ABSENT, gate=ABSENT, h=ABSENT, y=ABSENT), "neither", 1)
    refused(lib, forward(lib, gate=lines(2, p=None)), "gate is NULL", 1)
    refused(lib, forward(lib, x=lines(0, p=place(0) + 2)), "x is not aligned", 4)
    refused(lib, forward(lib, o=lines(1, p=place(1) + 1)), "o is not aligned", 4)
    refused(lib, forward(lib, o=lines(1, stride=-1)), "stride", 1)
    refused(lib, forward(lib, o=lines(1, stride=(1 << 31) + 1)), "stride", 1)
    refused(lib, forward(lib, y=lines(4, stride=127)), "rows overlap", 1)
    refused(lib, forward(lib, h=lines(0, p=place(0) + 512)), "h overlaps x", 1)
    refused(lib, forward(lib, h=lines(0, stride=256)), "h overlaps x", 1)
    refused(lib, forward(lib, h=lines(1)), "h overlaps o", 1)
    refused(lib, forward(lib, y=lines(2)), "y overlaps gate", 1)
    refused(lib, forward(lib, y=lines(0)), "y overlaps x", 1)
    refused(lib, forward(lib, h=lines(4)), "h overlaps y", 1)
    refused(lib, forward(lib, y=lines(22)), "y overlaps weight", 1)
    assert forward(lib, j=joint(tokens=0), h=lines(0, p=None), x=lines(0, p=None), o=lines(1, p=None), gate=lines(2, p=None),
                   y=lines(4, p=None)) == 0


def backward(lib, **kw):
    d = dict(joint=joint(), dh=lines(0), dy=lines(1), h=lines(2), o=lines(3), gate=lines(4), dx=lines(5), d_o=lines(6),
             d_gate=lines(7), d_weight=place(8), d_post_weight=place(9), d_scale=place(10), ws=place(11), n=1 << 20)
    d.update(kw)
    return lib.m3_residual_norm_backward(*d.values(), None)


def test_backward_refusals(lib):
    refused(lib, backward(lib, joint=None), "joint is NULL", 1)
    refused(lib, backward(lib, joint=joint(width=9000)), "width", 5)
    refused(lib, backward(lib, dy=None), "together", 1)
    refused(lib, backward(lib, joint=joint(weight=None)), "together", 1)
    refused(lib, backward(lib, joint=joint(weight=None), dy=None, dh=None, d_weight=None), "neither", 1)
    refused(lib, backward(lib, h=None), "h is NULL", 1)
    refused(lib, backward(lib, o=None), "without o", 1)
    refused(lib, backward(lib, gate=None), "without gate", 1)
    refused(lib, backward(lib, joint=joint(weight=None), dy=None), "without weight", 1)
    refused(lib, backward(lib, joint=joint(post_weight=None)), "without post_weight", 1)
    refused(lib, backward(lib, joint=joint(scale=None)), "without scale", 1)
    nothing = dict(dx=None, d_o=None, d_gate=None, d_weight=None, d_post_weight=None, d_scale=None)
    refused(lib, backward(lib, **nothing), "no gradient", 1)
    refused(lib, backward(lib, d_o=lines(6, stride=100)), "rows overlap", 1)
    refused(lib, backward(lib, dx=lines(2)), "dx overlaps h", 1)
    refused(lib, backward(lib, d_o=lines(1)), "d_o overlaps dy", 1)
    refused(lib, backward(lib, d_gate=lines(6)), "d_o overlaps d_gate", 1)
    refused(lib, backward(lib, d_weight=place(2)), "d_weight overlaps h", 1)
    refused(lib, backward(lib, d_weight=place(22)), "d_weight overlaps weight", 1)
    refused(lib, backward(lib, d_scale=place(9) + 4), "d_post_weight overlaps d_scale", 1)
    refused(lib, backward(lib, d_scale=place(10) + 2), "not 4-byte", 4)
    need = lib.m3_residual_norm_backward_workspace_size(joint(), 1)
    assert need == 3 * 1 * 128 * 4          # 5 rows are one workgroup's
    refused(lib, backward(lib, n=need - 1), "workspace", 7)
    refused(lib, backward(lib, ws=None, n=0), "workspace", 7)
    refused(lib, backward(lib, ws=place(11) + 8), "workspace is not", 4)
    refused(lib, backward(lib, ws=place(5)), "workspace overlaps dx", 1)
    assert backward(lib, joint=joint(tokens=0), d_weight=None, d_post_weight=None, d_scale=None, ws=None, n=0) == 0


def test_workspace_size(lib):
    size = lib.m3_residual_norm_backward_workspace_size
    assert size(joint(), 0) == 0 and size(joint(width=0), 1) == 0 and size(joint(tokens=0), 1) == 0
    for T, W in ((1, 1), (8192, 2048), (1 << 20, 64), (100, 8192)):
        assert 0 < size(joint(tokens=T, width=W), 1) <= 3 * 256 * W * 4


def test_python_refuses_cpu_tensors():
    import torch
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        nm.residual_norm(x, weight=torch.ones(64))
    with pytest.raises(ValueError):
        nm.residual_norm_backward(x, None, None, x)
