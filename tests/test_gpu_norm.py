"""The joint between two blocks (mamba_ssm_scan_amd.norm) against its definition in 64 bits: outputs, gradients, layouts."""
import pytest
import torch

from mamba_ssm_scan_amd import norm
from tests import norm_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
TYPES = {"bf16": (BF, BF), "mixed": (F32, BF), "f32": (F32, F32)}
NAMES = ("gate", "scale", "post_weight", "weight")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, bound, what):
    """bound: of fp32 arithmetic; the output's own rounding, half a step of its value, comes on top."""
    got, want = got.detach().cpu(), want.detach()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    room = bound * (1 + ref.HALF[got.dtype]) + want.abs() * ref.HALF[got.dtype] + 1e-37
    err = (got.double() - want).abs()
    worst = (err / room).nan_to_num(0.0).max().item() if got.numel() else 0.0
    print(f"  {what}: largest error / bound {worst:.3f}", flush=True)
    assert not ((err > room) | (got.isnan() != want.isnan())).any(), (what, worst)


def problem(T, W, types, seed=0, gate="silu", scale=True, post=True, pre=True):
    g = gen(1000 * seed + T + W)
    xt, ot = TYPES[types]
    n = lambda t, *s: torch.randn(s, generator=g).to(t)  # noqa: E731
    p = dict(x=3 * n(xt, T, W), o=n(ot, T, W), gate=n(ot, T, W) * 2 if gate else None, fn=gate or "silu",
             scale=0.5 + 0.1 * n(F32, W) if scale is True else scale, post_weight=1 + 0.2 * n(F32, W) if post else None,
             weight=1 + 0.2 * n(F32, W) if pre else None, dh=n(xt, T, W), dy=n(ot, T, W) if pre else None)
    return p


def dev(p, *names):
    return {k: p[k].to(DEV) if isinstance(p[k], torch.Tensor) else p[k] for k in names if p[k] is not None}


def call(p, eps=1e-6, **over):
    a = dict(dev(p, *NAMES), **over)
    x, o = a.pop("x", None), a.pop("o", None)
    x = p["x"].to(DEV) if x is None else x
    o = (p["o"].to(DEV) if p["o"] is not None else None) if o is None else o
    got = norm.residual_norm(x, o, gate_fn=p["fn"], eps=eps, **a)
    return dict(zip(("h", "y"), got)) if isinstance(got, tuple) else {"h" if p["weight"] is None else "y": got}


def expect(p, eps=1e-6):
    return ref.forward(p["x"], p["o"], p["gate"], p["fn"], p["scale"], p["post_weight"], p["weight"], eps)


def check_forward(p, got, eps=1e-6, what=""):
    want, bound = expect(p, eps)
    assert sorted(want) == sorted(got)
    for k in want:
        within(got[k], want[k], bound[k], f"{what}{k}")


def check_backward(p, got, h, eps=1e-6, keys=None, what=""):
    want, bound = ref.backward(p["dh"], p["dy"], h, p["o"], p["gate"], p["fn"], p["scale"], p["post_weight"], p["weight"], eps)
    for k in want if keys is None else keys:
        within(got[k], want[k], bound[k], f"{what}d{k}")
    for k in set(got) - set(want if keys is None else keys):
        assert got[k] is None, k


SIZES = [(1, 1), (3, 7), (5, 64), (33, 128), (2, 130), (700, 96), (9, 512), (4, 1000), (131, 1024), (7, 1283), (128, 2048),
         (3, 2050), (11, 4096), (5, 4104), (2, 5001), (3, 8192), (1, 8191), (0, 64), (300, 2056)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,W", SIZES)
def test_sizes(T, W, types):
    p = problem(T, W, types)
    got = call(p)
    check_forward(p, got)
    g = norm.residual_norm_backward(p["dh"].to(DEV), p["dy"].to(DEV), got["h"], p["o"].to(DEV), gate_fn=p["fn"], **dev(p, *NAMES))
    check_backward(p, g, got["h"].cpu())


@pytest.mark.parametrize("types", ["bf16", "f32"])
@pytest.mark.parametrize("pre", [True, False], ids=["pre", "no_pre"])
@pytest.mark.parametrize("post", [True, False], ids=["post", "no_post"])
@pytest.mark.parametrize("scale", [True, 0.25, None], ids=["scale", "factor", "no_scale"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid", "identity", ""])
def test_parts(gate, scale, post, pre, types):
    p = problem(19, 320, types, seed=1, gate=gate, scale=scale, post=post, pre=pre)
    got = call(p)
    check_forward(p, got)
    g = norm.residual_norm_backward(p["dh"].to(DEV), p["dy"].to(DEV) if pre else None, got["h"] if pre else None,
                                    p["o"].to(DEV), gate_fn=p["fn"], **dev(p, *NAMES))
    check_backward(p, g, got["h"].cpu())


@pytest.mark.parametrize("T,W", [(1, 64), (17, 2048), (6, 999), (3, 8192)])
@pytest.mark.parametrize("types", ["bf16", "f32"])
def test_without_branch(T, W, types):
    """y = N(x) alone; its gradient with and without a gradient of the stream itself."""
    p = problem(T, W, types, seed=2)
    p.update(o=None, gate=None, scale=None, post_weight=None)
    got = call(p)
    assert list(got) == ["y"]
    check_forward(p, got)
    for dh in (p["dh"], None):
        q = dict(p, dh=dh)
        g = norm.residual_norm_backward(None if dh is None else dh.to(DEV), p["dy"].to(DEV), p["x"].to(DEV),
                                        weight=p["weight"].to(DEV))
        check_backward(q, g, p["x"])


def test_norm_alone_into_bf16():
    """The first block's input from an fp32 stream, for blocks in bf16; its gradient by autograd."""
    p = problem(9, 300, "f32", seed=2)
    p.update(o=None, gate=None, scale=None, post_weight=None, dy=p["dy"].to(BF))
    x = p["x"].to(DEV).requires_grad_()
    y = norm.residual_norm(x, weight=p["weight"].to(DEV), dtype=BF)
    assert y.dtype == BF
    check_forward(p, {"y": y})
    (dx,) = torch.autograd.grad(y, x, p["dy"].to(DEV))
    check_backward(dict(p, dh=None), {"x": dx}, p["x"], keys=["x"])


def test_only_what_is_asked():
    p = problem(40, 768, "mixed", seed=3)
    h = call(p)["h"]
    args = (p["dh"].to(DEV), p["dy"].to(DEV), h, p["o"].to(DEV))
    kw = dict(gate_fn=p["fn"], **dev(p, *NAMES))
    whole = norm.residual_norm_backward(*args, **kw)
    for want in (["x"], ["o"], ["gate"], ["scale"], ["post_weight"], ["weight"], ["x", "weight"], ["o", "scale"], []):
        g = norm.residual_norm_backward(*args, want=want, **kw)
        for k in whole:
            assert (g[k] is None) if k not in want else torch.equal(g[k], whole[k]), (want, k)
    none = norm.residual_norm_backward(None, p["dy"].to(DEV), h, p["o"].to(DEV), **kw)
    check_backward(dict(p, dh=None), none, h.cpu())
    with pytest.raises(ValueError):
        norm.residual_norm_backward(*args, want=["bias"], **kw)


def test_no_rows_give_zero_sums():
    p = problem(0, 72, "f32")
    z = torch.empty(0, 72, device=DEV)
    g = norm.residual_norm_backward(z, z, z, z, gate=z, **{k: v for k, v in dev(p, *NAMES).items() if k != "gate"})
    for k in ("scale", "post_weight", "weight"):
        assert torch.equal(g[k], torch.zeros(72, device=DEV))
    assert g["x"].shape == g["o"].shape == g["gate"].shape == (0, 72)


@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("types", TYPES)
def test_rows_of_a_projection(types, shift):
    """o and the gate as neighbours in one buffer, aligned or not, the stream in rows of its own stride; the buffer and
    the places between the rows keep their bits; then the stream in place, in every layout of the leading axes."""
    W, T = 136, 21
    p = problem(T, W, types, seed=4)
    xt, ot = TYPES[types]
    both = torch.randn(T, 2 * W + 24, generator=gen(7)).to(ot).to(DEV)
    o, gate = both[:, shift:shift + W], both[:, shift + W + 8:shift + 2 * W + 8]
    o.copy_(p["o"])
    gate.copy_(p["gate"])
    room = torch.randn(T, W + 24, generator=gen(8)).to(xt).to(DEV)
    x = room[:, shift:shift + W]
    x.copy_(p["x"])
    before, held = both.clone(), room.clone()
    got = call(p, x=x, o=o, gate=gate)
    check_forward(p, got)
    assert torch.equal(both, before) and torch.equal(room, held)
    h, y = norm.residual_norm(x, o, gate=gate, gate_fn=p["fn"], out=x, **{k: v for k, v in dev(p, *NAMES).items() if k != "gate"})
    assert h is x and torch.equal(x, got["h"]) and torch.equal(y, got["y"])
    mask = torch.ones_like(room, dtype=torch.bool)
    mask[:, shift:shift + W] = False
    assert torch.equal(room[mask], held[mask]) and torch.equal(both, before)
    x3 = p["x"].to(DEV).view(3, 7, W)
    a = norm.residual_norm(x3, o.unflatten(0, (3, 7)), weight=p["weight"].to(DEV))
    b = norm.residual_norm(p["x"].to(DEV), o, weight=p["weight"].to(DEV))
    assert a[0].shape == a[1].shape == (3, 7, W) and torch.equal(a[0].view(T, W), b[0]) and torch.equal(a[1].view(T, W), b[1])
    g1 = norm.residual_norm_backward(room[:, shift:shift + W], p["dy"].to(DEV), got["h"], o, gate=gate, gate_fn=p["fn"],
                                     **{k: v for k, v in dev(p, *NAMES).items() if k != "gate"})
    g2 = norm.residual_norm_backward(room[:, shift:shift + W].contiguous(), p["dy"].to(DEV), got["h"], o.contiguous(),
                                     gate=gate.contiguous(), gate_fn=p["fn"],
                                     **{k: v for k, v in dev(p, *NAMES).items() if k != "gate"})
    q = dict(p, dh=room[:, shift:shift + W].cpu())
    check_backward(q, g1, got["h"].cpu())
    check_backward(q, g2, got["h"].cpu())


def test_one_row_in_one_place():
    """One token, width 1, a stride of nothing, a single row read by every row."""
    x = torch.tensor([[2.0]], device=DEV)
    y = norm.residual_norm(x, weight=torch.tensor([3.0], device=DEV), eps=0.0)
    assert y.item() == 3.0
    p = problem(6, 256, "f32", seed=5)
    row = p["o"][:1].to(DEV)
    got = call(p, o=row.expand(6, 256), gate=p["gate"][:1].to(DEV).expand(6, 256))
    check_forward(dict(p, o=p["o"][:1].expand(6, 256), gate=p["gate"][:1].expand(6, 256)), got)


def test_far_rows():
    """Offsets beyond 2^32 bytes and entries."""
    T, W, stride = 1100, 64, 1 << 22
    buf = torch.empty(T * stride, dtype=BF, device=DEV)
    x = buf.view(T, stride)[:, :W]
    p = problem(T, W, "bf16", seed=6)
    x.copy_(p["x"])
    got = call(p, x=x)
    check_forward(p, got)
    o = buf.view(T, stride)[:, W:2 * W]
    o.copy_(p["o"])
    dx = norm.residual_norm_backward(x, p["dy"].to(DEV), got["h"], o, gate_fn=p["fn"], **dev(p, *NAMES))
    check_backward(dict(p, dh=p["x"]), dx, got["h"].cpu())


def test_zeros_infinities_and_nan_stay_in_their_row():
    p = problem(8, 512, "f32", seed=7)
    p["x"][1], p["o"][1] = 0.0, 0.0
    p["o"][2] = 0.0
    clean = call(p)
    check_forward(p, clean)
    assert clean["y"][1].abs().max() == 0
    p["o"][3, 5], p["gate"][4, 0], p["x"][5, 9], p["o"][6, 7] = float("nan"), float("nan"), float("inf"), float("inf")
    got = call(p)
    for k in got:
        assert torch.equal(got[k][[0, 1, 2, 7]], clean[k][[0, 1, 2, 7]])
    assert got["y"][3].isnan().all() and got["y"][4].isnan().all() and got["h"][4].isnan().sum() == 1
    assert got["h"][5, 9] == float("inf")
    g = norm.residual_norm_backward(p["dh"].to(DEV), p["dy"].to(DEV), got["h"], p["o"].to(DEV), gate_fn=p["fn"], **dev(p, *NAMES))
    rest = [0, 1, 2, 7]
    want, bound = ref.backward(p["dh"][rest], p["dy"][rest], got["h"].cpu()[rest], p["o"][rest], p["gate"][rest], p["fn"],
                               p["scale"], p["post_weight"], p["weight"], 1e-6)
    for k in ("x", "o", "gate"):
        within(g[k][rest], want[k], bound[k], k)


@pytest.mark.parametrize("W", [256, 1001])
def test_saturated_gates(W):
    """Gates far out on both sides: no overflow on the way, slopes that end at 0 and 1."""
    p = problem(4, W, "f32", seed=8, post=False, scale=None)
    p["gate"] = torch.linspace(-100, 100, 4 * W).view(4, W)
    for fn in ("silu", "sigmoid"):
        p["fn"] = fn
        got = call(p)
        check_forward(p, got)
        g = norm.residual_norm_backward(p["dh"].to(DEV), p["dy"].to(DEV), got["h"], p["o"].to(DEV), gate_fn=fn, **dev(p, *NAMES))
        check_backward(p, g, got["h"].cpu())


# ---------------------------------------------------------------------------------------------------------- autograd

@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("T,W", [(1, 64), (45, 520), (10, 2048)])
def test_autograd(T, W, types):
    p = problem(T, W, types, seed=9)
    leaf = {k: v.requires_grad_() for k, v in dev(p, "x", "o", *NAMES).items()}
    h, y = norm.residual_norm(**leaf, gate_fn=p["fn"])
    assert h.requires_grad and y.requires_grad
    check_forward(p, {"h": h, "y": y})
    grads = torch.autograd.grad([h, y], list(leaf.values()), [p["dh"].to(DEV), p["dy"].to(DEV)], retain_graph=True)
    check_backward(p, dict(zip(leaf, grads)), h.detach().cpu())
    for k, g in zip(leaf, grads):
        assert g.dtype == leaf[k].dtype
    (only,) = torch.autograd.grad(y, leaf["x"], p["dy"].to(DEV), retain_graph=True)
    check_backward(dict(p, dh=None), {"x": only}, h.detach().cpu(), keys=["x"])
    only = torch.autograd.grad(h, [leaf["x"], leaf["o"], leaf["scale"]], p["dh"].to(DEV))
    check_backward(dict(p, dy=None, weight=None), dict(zip(("x", "o", "scale"), only)), h.detach().cpu(), keys=["x", "o", "scale"])


def test_autograd_against_differences():
    """Central differences of a loss along random directions, for every input (64 bits: the definition's own)."""
    p = problem(6, 48, "f32", seed=10)
    leaf = {k: v.requires_grad_() for k, v in dev(p, "x", "o", *NAMES).items()}
    h, y = norm.residual_norm(**leaf, gate_fn=p["fn"])
    loss = (h * p["dh"].to(DEV)).sum() + (y * p["dy"].to(DEV)).sum()
    grads = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))

    def value(q):
        got, _ = ref.forward(q["x"], q["o"], q["gate"], q["fn"], q["scale"], q["post_weight"], q["weight"], 1e-6)
        return (got["h"] * p["dh"].double()).sum() + (got["y"] * p["dy"].double()).sum()

    q = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    for k in leaf:
        d = torch.randn(q[k].shape, generator=gen(11), dtype=torch.float64)
        e = 1e-5                         # truncation e^2 times a third derivative, some hundreds here; rounding 1e-16 / e
        diff = (value(dict(q, **{k: q[k] + e * d})) - value(dict(q, **{k: q[k] - e * d}))) / (2 * e)
        got = (grads[k].cpu().double() * d).sum()
        size = (grads[k].cpu().double() * d).abs().sum()
        assert abs(float(diff - got)) <= 1e-6 * max(1.0, float(size)), (k, float(diff), float(got))


def test_gradients_through_a_stack():
    """Pre-norm, a product, the joint, another product, the last sum; gradients of weights shared by both joints, of a
    broadcast gate and of a sum (whose gradient has no strides); on a stream of its own too."""
    g = gen(12)
    T, W = 24, 64
    rnd = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    x, m1, m2 = rnd(T, W), rnd(W, W) / 8, rnd(W, W) / 8
    leaf = [t.requires_grad_() for t in (x, m1, m2, 1 + 0.1 * rnd(W), 1 + 0.1 * rnd(W), rnd(1, W))]

    def stack(f, x, m1, m2, w, s, gate):
        y = f(x, weight=w)
        x, y = f(x, y @ m1, gate=gate.expand(T, W), scale=s, post_weight=w, weight=w)
        return f(x, y @ m2, scale=s).sum()

    def plain(x, o=None, gate=None, scale=None, post_weight=None, weight=None):
        if o is not None:
            o = o if post_weight is None else ref.norm(o, post_weight, 1e-6)[0]
            o = o if gate is None else o * gate * torch.sigmoid(gate)
            x = x + (o if scale is None else o * scale)
        if weight is None:
            return x
        y = ref.norm(x, weight, 1e-6)[0]
        return y if o is None else (x, y)

    copies = [t.detach().cpu().double().requires_grad_() for t in leaf]
    want = torch.autograd.grad(stack(plain, *copies), copies)
    for stream in (None, torch.cuda.Stream()):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            got = torch.autograd.grad(stack(lambda *a, **k: norm.residual_norm(*a, stream=stream, **k), *leaf), leaf)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            # three joints and three products of 64 terms in fp32: some hundreds of roundings of the largest entries
            assert (a.cpu().double() - b).abs().max() <= 1000 * ref.U * b.abs().max()


def test_gradients_of_broadcast_results():
    """Sums over tokens or batches of three-axis rows: gradients whose rows lie at no one stride."""
    g = gen(16)
    x, o, w = (torch.randn(s, generator=g).to(DEV).requires_grad_() for s in ((3, 5, 64), (3, 5, 64), (64,)))
    v = torch.randn(3, 64, generator=g).to(DEV)
    h, y = norm.residual_norm(x, o, weight=w)
    got = torch.autograd.grad((y.sum(1) * v).sum() + (h.mean((0, 2)) ** 2).sum(), [x, o, w])
    a, b, c = (t.detach().cpu().double().requires_grad_() for t in (x, o, w))
    hh = a + b
    yy = ref.norm(hh, c, 1e-6)[0]
    want = torch.autograd.grad((yy.sum(1) * v.cpu().double()).sum() + (hh.mean((0, 2)) ** 2).sum(), [a, b, c])
    for s, t in zip(got, want):   # rows of 64 terms and sums of 15 rows in fp32: some hundreds of roundings
        assert (s.cpu().double() - t).abs().max() <= 500 * ref.U * t.abs().max()


def test_outside_autograd_and_not_twice():
    p = problem(5, 128, "f32", seed=13)
    leaf = {k: v.requires_grad_() for k, v in dev(p, "x", "o", *NAMES).items()}
    with torch.no_grad():
        a = norm.residual_norm(**leaf)
    b = norm.residual_norm(**leaf, out=torch.empty(5, 128, device=DEV))
    c = norm.residual_norm(**leaf)
    for i in range(2):
        assert not a[i].requires_grad and not b[i].requires_grad and torch.equal(a[i], b[i]) and torch.equal(a[i], c[i])
    (d,) = torch.autograd.grad(c[1].sum(), leaf["x"], create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(d.sum(), leaf["x"])


# ---------------------------------------------------------------------------------------------------------- calls

def test_captured_step_replays():
    """A training step of the joint captured with leaves of its own, replayed with new inputs and eager work between."""
    sizes = (37, 640)
    p = problem(*sizes, "mixed", seed=14)
    live = dev(p, "x", "o", "dh", "dy", *NAMES)

    def step():
        leaf = {k: live[k].detach().requires_grad_() for k in ("x", "o", *NAMES)}
        h, y = norm.residual_norm(**leaf)
        return [h.detach(), y.detach(), *torch.autograd.grad([h, y], list(leaf.values()), [live["dh"], live["dy"]])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        q = problem(*sizes, "mixed", seed=20 + k)
        for n in live:
            live[n].copy_(q[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_same_bits_every_time_and_two_calls_at_once():
    p = problem(900, 2048, "bf16", seed=15)
    a = dev(p, "dh", "dy", "x", "o")
    kw = dict(gate_fn=p["fn"], **dev(p, *NAMES))
    first = norm.residual_norm_backward(a["dh"], a["dy"], a["x"], a["o"], **kw)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    many = [norm.residual_norm_backward(a["dh"], a["dy"], a["x"], a["o"], stream=s, **kw) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for g in many:
        for k in first:
            assert torch.equal(g[k], first[k])


def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    b = x.to(BF)
    for kw in (dict(o=x[:, :32]), dict(o=x.cpu()), dict(o=x, gate=b), dict(weight=w[:32]), dict(o=x, scale=w.double()),
               dict(o=x, weight=w.to(BF)), dict(gate=x), dict(out=x), dict(o=x, gate_fn="relu"), dict(), dict(o=x, out=b),
               dict(o=x.t().contiguous().t()), dict(o=x, post_weight=w.cpu()),
               dict(o=x, weight=w, dtype=BF)):
        with pytest.raises((ValueError, TypeError, norm.binding.M3Error)):
            norm.residual_norm(x, **kw)
    for args in ((x.half(), x), (b, x), (torch.zeros(2, 8200, device=DEV), torch.zeros(2, 8200, device=DEV)),
                 (torch.zeros(4, 64), None), (x.view(2, 2, 64).transpose(0, 1), None)):
        with pytest.raises((ValueError, TypeError, norm.binding.M3Error)):
            norm.residual_norm(*args, weight=torch.ones(args[0].shape[-1], device=DEV))
    with pytest.raises(norm.binding.M3Error):
        norm.residual_norm(x, x + 1, eps=-1.0)
    flat = torch.zeros(5 * 64, device=DEV)
    with pytest.raises(norm.binding.M3Error):                    # h would overlap x a row further on
        norm.residual_norm(flat[:256].view(4, 64), x, out=flat[64:].view(4, 64))
    for args, kw in (((x, None, x), dict(weight=w)), ((x, x, x), {}), ((None, None, x), {}), ((None, x, None), dict(weight=w)),
                     ((x, x, x[:2]), dict(weight=w)), ((x, b.half(), x), dict(weight=w))):
        with pytest.raises((ValueError, TypeError, norm.binding.M3Error)):
            norm.residual_norm_backward(*args, **kw)


def test_out_that_autograd_still_needs():
    """A tensor that autograd kept for a backward pass and that `out` then overwrites is found out."""
    x = torch.randn(4, 64, generator=gen(31)).to(DEV)
    s = torch.ones(64, device=DEV, requires_grad=True)
    y = (x * s).sum()
    with torch.no_grad():
        norm.residual_norm(x, torch.ones_like(x), out=x)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
