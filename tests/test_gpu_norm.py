"""Global norm and clipping of many tensors on the GPU against 64-bit sums.

Bounds: the norm is summed in 64 bits (relative error below N 2^-53, far under
the 2^-24 of its rounding to 32 bits); a clipped element is one product by a
factor rounded to 32 bits (64 for float64), then rounded to its type.
"""
import math

import numpy as np
import pytest
import torch

import differentiable_sparse_linear_csr_b200 as sla
from differentiable_sparse_linear_csr_b200 import _lib as L

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DTYPES = [torch.float64, torch.float32, torch.bfloat16, torch.float16]
SETS = {
    "one": [1], "odd": [7, 1, 4097, 0, 33], "chunk_edges": [8191, 8192, 8193, 16384, 16385, 4096, 2048, 65536],
    "many": [1 + 37 * k % 911 for k in range(300)], "large": [3_000_001, 12, 5_000_000],
    "empty": [0, 0],
}


def make(sizes, dtypes, seed=0, spread=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(n, generator=gen, device=DEV) * spread).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def exact_norm(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


def check(ts, outs, norm, limit, kind=2.0):
    ref = exact_norm(ts) if kind == 2.0 else max([float(t.double().abs().max()) for t in ts if t.numel()] or [0.0])
    u = 2.0 ** -53 if norm.dtype == torch.float64 else 2.0 ** -24
    slack = sum(t.numel() for t in ts) * 2.0 ** -53 if kind == 2.0 else 0.0
    assert abs(float(norm) - ref) <= (u + slack) * ref * 1.01
    f = min(1.0, limit / (ref + 1e-6))
    for t, o in zip(ts, outs):
        assert o.dtype == t.dtype and o.shape == t.shape
        uo = torch.finfo(t.dtype).eps / 2
        uf = 2.0 ** -53 if t.dtype == torch.float64 else 2.0 ** -24
        tiny = torch.finfo(t.dtype).smallest_normal * uo * 2
        want = t.double() * f
        bound = want.abs() * (uo + 2 * uf + slack + 2.0 ** -52) * 1.01 + tiny
        assert ((o.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("name", sorted(SETS))
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_norm_and_clip(name, dtype, kind):
    ts = make(SETS[name], [dtype])
    before = [t.clone() for t in ts]
    for limit in (0.37, 1e30, 0.0):
        outs, norm = sla.clip_by_global_norm(ts, limit, norm_type=kind)
        check(ts, outs, norm, limit, kind)
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
    assert torch.equal(sla.global_norm(ts, kind), norm)


def test_mixed_types_in_place_and_repeatable():
    ts = make(SETS["many"] + SETS["chunk_edges"], DTYPES)
    before = [t.clone() for t in ts]
    outs, norm = sla.clip_by_global_norm(ts, 3.0)
    assert norm.dtype == torch.float64
    same, norm2 = sla.clip_by_global_norm(ts, 3.0, out=ts)
    assert all(a is b for a, b in zip(same, ts)) and torch.equal(norm, norm2)
    assert all(torch.equal(a, b) for a, b in zip(ts, outs))
    check(before, ts, norm, 3.0)


def test_squares_beyond_32_bits():
    for spread in (1e25, 1e-25):
        ts = make([1000, 33], [torch.float32, torch.bfloat16], spread=spread)
        assert abs(float(sla.global_norm(ts)) / exact_norm(ts) - 1) < 1e-6


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_not_finite(bad, kind):
    ts = make([5, 70000], [torch.float32])
    ts[1][69999] = bad
    outs, norm = sla.clip_by_global_norm(ts, 1.0, norm_type=kind)
    if math.isnan(bad):
        assert math.isnan(float(norm)) and all(torch.isnan(o).all() for o in outs)
    else:
        assert float(norm) == math.inf
        assert torch.isnan(outs[1][69999]) and not outs[0].any() and not outs[1][:69999].any()


def test_layouts():
    """Transposed, sliced and offset tensors; an output laid out otherwise."""
    base = make([1200, 601, 900], [torch.float32])
    ts = [base[0].view(30, 40).t(), base[1][1:], base[2].view(30, 30)[:, ::2]]
    outs, norm = sla.clip_by_global_norm(ts, 0.5)
    check(ts, outs, norm, 0.5)
    other = [torch.empty(40, 30, device=DEV), torch.empty(1200, device=DEV)[::2], torch.empty(30, 15, device=DEV)]
    got, _ = sla.clip_by_global_norm(ts, 0.5, out=other)
    assert all(torch.equal(a, b) for a, b in zip(got, outs))
    sla.clip_by_global_norm(ts, 0.5, out=ts)
    assert all(torch.equal(a, b) for a, b in zip(ts, outs))
    assert torch.equal(base[1][:1], make([1200, 601, 900], [torch.float32])[1][:1])     # what lies before a view
    assert torch.equal(base[2].view(30, 30)[:, 1::2], make([1200, 601, 900], [torch.float32])[2].view(30, 30)[:, 1::2])


def test_clip_grad_norm_of_parameters():
    ps = [torch.nn.Parameter(t) for t in make([100, 7, 50], [torch.float32])]
    for p in ps[:2]:
        p.grad = torch.randn_like(p)
    g = [p.grad.clone() for p in ps[:2]]
    norm = sla.clip_grad_norm_(ps, 0.1)
    check(g, [p.grad for p in ps[:2]], norm, 0.1)
    assert ps[2].grad is None
    assert float(sla.clip_grad_norm_([ps[2]], 1.0)) == 0.0
    one = torch.nn.Parameter(torch.zeros(3, device=DEV))
    one.grad = torch.tensor([3.0, 0.0, 4.0], device=DEV)
    assert float(sla.clip_grad_norm_(one, 1.0)) == 5.0


def test_zero_gradients_and_norm_under_the_bound_are_untouched():
    z = [torch.zeros(1000, device=DEV)]
    assert float(sla.clip_grad_norm_([torch.nn.Parameter(z[0])], 1.0)) == 0.0
    assert float(sla.global_norm(z)) == 0.0
    ts = make([1000], [torch.bfloat16])
    outs, _ = sla.clip_by_global_norm(ts, 1e6)
    assert torch.equal(outs[0], ts[0])


def test_captured_and_replayed():
    ts = make([100, 70000, 3], [torch.float32, torch.bfloat16])
    outs = [torch.empty_like(t) for t in ts]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sla.clip_by_global_norm(ts, 1.0, out=outs)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, norm = sla.clip_by_global_norm(ts, 1.0, out=outs)
        alone = sla.global_norm(ts)
    for t, x in zip(ts, make([100, 70000, 3], [torch.float32, torch.bfloat16], seed=5)):
        t.copy_(x)
    graph.replay()
    want, n2 = sla.clip_by_global_norm(ts, 1.0)
    assert torch.equal(norm, n2) and torch.equal(alone, n2)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    ts = make([10, 10], [torch.float32])
    for kw in ({"norm_type": 3.0}, {"out": ts[:1]}, {"out": [ts[0], ts[1].double()]}):
        with pytest.raises(ValueError):
            sla.clip_by_global_norm(ts, 1.0, **kw)
    for limit in (-1.0, math.nan, math.inf):
        with pytest.raises(ValueError):
            sla.clip_by_global_norm(ts, limit)
    with pytest.raises(ValueError):
        sla.global_norm([ts[0], ts[1].cpu()])
    with pytest.raises(TypeError):
        sla.global_norm([ts[0].int()])
    with pytest.raises(L.SlaError, match="shares memory"):           # one tensor twice, in place
        sla.clip_by_global_norm([ts[0], ts[0]], 1.0, out=[ts[0], ts[0]])
    big = torch.randn(100, device=DEV)
    with pytest.raises(L.SlaError, match="shares memory"):           # an output over another's input
        sla.clip_by_global_norm([big[:50], big[50:]], 1.0, out=[big[10:60], torch.empty(50, device=DEV)])
    # the same input twice is two gradients, with an output each
    outs, norm = sla.clip_by_global_norm([ts[0], ts[0]], 1.0)
    check([ts[0], ts[0]], outs, norm, 1.0)


def test_writing_counts_as_a_change():
    """A tensor that autograd saved and clipping overwrote is refused by the backward pass."""
    x = torch.ones(5, device=DEV)
    w = torch.ones(5, device=DEV, requires_grad=True)
    y = (x * w).sum()
    sla.clip_by_global_norm([x], 1.0)                  # new outputs: x is as it was
    torch.autograd.grad(y, w, retain_graph=True)
    sla.clip_by_global_norm([x], 1.0, out=[x])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, w)


def test_outputs_written_by_way_of_a_copy_are_checked_first():
    """A gradient that two parameters share, or that is expanded, is refused before any
    other gradient is scaled, also where it is not dense."""
    wide = torch.ones(4, 6, device=DEV)
    for grads in ([wide[:, :3]] * 2, [torch.ones(1, device=DEV).expand(5)], [wide[::2, :3]], [wide[:0, :3]] * 2):
        params = [torch.zeros(7, device=DEV, requires_grad=True)] + \
            [torch.zeros(g.shape, device=DEV, requires_grad=True) for g in grads]
        params[0].grad = torch.full((7,), 5.0, device=DEV)
        for p, g in zip(params[1:], grads):
            p.grad = g
        bad = len(grads) > 1 and grads[0].numel() > 0 or 0 in grads[0].stride()
        if bad:
            with pytest.raises(ValueError, match="twice|expanded"):
                sla.clip_grad_norm_(params, 1.0)
            assert torch.equal(params[0].grad, torch.full((7,), 5.0, device=DEV)) and torch.equal(wide, torch.ones_like(wide))
        else:
            want = torch.sqrt(sum((p.grad.double() ** 2).sum() for p in params))
            norm = sla.clip_grad_norm_(params, 1.0)
            assert abs(float(norm) - float(want)) <= 1e-6 * float(want)
            assert torch.allclose(params[0].grad, torch.full((7,), 5.0 / float(want), device=DEV), rtol=1e-6)
            wide.fill_(1.0)
