"""Attention over a CSR pattern on the GPU against the 64-bit definition
(tests/attention_oracle.py), with its derived error bounds: every type, head
layout and kind of row (empty, one entry, longer than one work item), strides,
masks, broadcast values, streams, captured calls and the autograd chain to the
other operators of the package.
"""
import numpy as np
import pytest
import torch

import differentiable_sparse_linear_csr_b200 as sla
from differentiable_sparse_linear_csr_b200 import _lib as L
from differentiable_sparse_linear_csr_b200 import workloads as W
from tests.attention_oracle import attention, within

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f64": torch.float64, "f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def T(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def H(t):
    torch.cuda.synchronize()
    return t.detach().double().cpu().numpy()


def from_rows(rows, m):
    rp = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
    ci = np.concatenate([np.sort(np.asarray(r, dtype=np.int32)) for r in rows] + [np.zeros(0, np.int32)])
    return rp, ci.astype(np.int32), m


def pattern(name):
    """(rowptr, colind, n_cols)"""
    rng = np.random.default_rng(7)
    pick = lambda m, c: rng.choice(m, size=c, replace=False)  # noqa: E731
    if name == "one":
        return from_rows([[0]], 1)
    if name == "one_row_long":                       # split over many work items
        return from_rows([np.arange(700)], 700)
    if name == "one_column":                         # a long row of A^T
        return from_rows([[0]] * 333, 1)
    if name == "full":
        return from_rows([np.arange(70)] * 37, 70)
    if name == "empty_rows":
        return from_rows([pick(50, c) for c in (0, 3, 0, 0, 50, 1, 17, 0, 16, 15, 2, 0, 33, 0, 0, 4, 0, 0, 9, 0)], 50)
    if name == "no_entries":
        return from_rows([[], [], []], 5)
    if name == "hub":                                # one long row among short ones, one long column
        rows = [np.unique(np.concatenate([[3], pick(900, int(c))])) for c in rng.integers(0, 6, 61)]
        rows[40] = pick(900, 400)
        return from_rows(rows, 900)
    if name == "grid":
        rp, ci, _ = W.poisson2d(17)
        return rp.astype(np.int32), ci.astype(np.int32), 289
    raise KeyError(name)


def inputs(name, batch, heads, kv, dim, code, values, seed=0, spread=1.0):
    """Tensors of the type, and the same numbers in 64 bits."""
    rp, ci, m = pattern(name)
    n = rp.shape[0] - 1
    gen = torch.Generator().manual_seed(seed)
    new = lambda *s: (torch.randn(*s, generator=gen, dtype=torch.float64) * spread).to(DT[code])  # noqa: E731
    q, k, v, do = new(batch, n, heads, dim), new(batch, m, kv, dim), new(batch, m, kv, dim), new(batch, n, heads, dim)
    vals = None
    vt = torch.float64 if code == "f64" else torch.float32
    if values:
        vals = torch.randn(batch, ci.shape[0], generator=gen, dtype=torch.float64).to(vt)
    A = sla.CSR(T(rp), T(ci), n_cols=m, batch=batch, dtype=vt)
    return A, rp, ci, q, k, v, vals, do


def run(A, q, k, v, vals, do, scale=None):
    ts = [t.to(DEV).requires_grad_() for t in (q, k, v) + ((vals,) if vals is not None else ())]
    o = A.attention(*ts, scale=scale)
    grads = torch.autograd.grad(o, ts, do.to(DEV))
    return [H(o)] + [H(g) for g in grads]


def compare(A, rp, ci, q, k, v, vals, do, code, scale=None):
    got = run(A, q, k, v, vals, do, scale)
    sc = q.shape[3] ** -0.5 if scale is None else scale
    worst = {}
    for b in range(q.shape[0]):
        res, err = attention(rp, ci, *(x[b].double().numpy() for x in (q, k, v)),
                             None if vals is None else vals[b].double().numpy(), sc, do[b].double().numpy(), code)
        for x, g in zip(("o", "dq", "dk", "dv", "dvals"), got):
            worst[x] = max(worst.get(x, 0.0), within(g[b], res[x], err[x]))
    assert all(w <= 1.0 for w in worst.values()), worst
    return got


LENGTHS = {
    "long_among_middle": [60, 17, 64, 65, 5000, 0, 63, 1, 129, 16],    # one row in hundreds of parts, others whole
    "many_of_few_parts": [100] * 140,
    "many_of_many_parts": [700] * 140,
}


@pytest.mark.parametrize("name", LENGTHS)
@pytest.mark.parametrize("code", ["f64", "f32", "bf16", "f16"])
def test_split_rows(name, code):
    """Rows of every number of parts: joined by one warp, or by several."""
    rng = np.random.default_rng(11)
    m = max(LENGTHS[name]) + 13
    rp, ci, m = from_rows([rng.choice(m, size=c, replace=False) for c in LENGTHS[name]], m)
    for heads, kv, dim in ((8, 8, 16), (4, 1, 32)):
        gen = torch.Generator().manual_seed(3)
        new = lambda *s: torch.randn(1, *s, generator=gen, dtype=torch.float64).to(DT[code])  # noqa: E731
        n = rp.shape[0] - 1
        q, do, k, v = new(n, heads, dim), new(n, heads, dim), new(m, kv, dim), new(m, kv, dim)
        vt = torch.float64 if code == "f64" else torch.float32
        vals = torch.randn(1, ci.shape[0], generator=gen, dtype=torch.float64).to(vt)
        vals[0, ::7] = -np.inf
        A = sla.CSR(T(rp), T(ci), n_cols=m, batch=1, dtype=vt)
        compare(A, rp, ci, q, k, v, vals, do, code)


@pytest.mark.parametrize("name", ["one", "one_row_long", "one_column", "full", "empty_rows", "no_entries", "hub", "grid"])
@pytest.mark.parametrize("code", ["f64", "f32", "bf16", "f16"])
def test_patterns(name, code):
    compare(*inputs(name, 1, 2, 2, 32, code, True), code)


@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 16), (4, 4, 64), (8, 2, 32), (6, 3, 48), (3, 1, 80), (2, 2, 96), (2, 1, 112),
                                          (2, 1, 128), (2, 2, 20), (1, 1, 1), (5, 5, 33), (2, 1, 100), (1, 1, 256),
                                          (1, 1, 255), (16, 1, 8), (33, 11, 4), (16, 1, 64), (24, 2, 32), (32, 1, 16),
                                          (8, 1, 128), (10, 5, 64), (8, 8, 16), (4, 4, 32)])
@pytest.mark.parametrize("code", ["f64", "f32", "bf16", "f16"])
def test_head_layouts(heads, kv, dim, code):
    compare(*inputs("hub", 1, heads, kv, dim, code, True, seed=dim), code)


@pytest.mark.parametrize("code", ["f64", "f32", "bf16", "f16"])
def test_batch_without_values(code):
    compare(*inputs("empty_rows", 3, 4, 2, 64, code, False), code)


@pytest.mark.parametrize("code", ["f32", "bf16", "f16"])
def test_given_scale_and_large_scores(code):
    """Scores of several hundred: the running maximum keeps exp in range."""
    compare(*inputs("hub", 1, 2, 2, 64, code, True, spread=6.0), code, scale=0.7)


@pytest.mark.parametrize("code", ["f64", "f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 20])
def test_masked_entries_hold_anything(code, dim):
    """Values of -inf leave entries out: k and v there are NaN and infinite,
    whole rows are masked, and nothing of it reaches an output or gradient."""
    A, rp, ci, q, k, v, vals, do = inputs("hub", 2, 4, 2, dim, code, True)
    m = k.shape[1]
    dead = torch.zeros(m, dtype=torch.bool)
    dead[::5] = True
    dead[3] = True                                  # the long column
    vals[:, dead[torch.from_numpy(ci.astype(np.int64))]] = -np.inf
    rows = np.repeat(np.arange(rp.shape[0] - 1), np.diff(rp))
    vals[0, torch.from_numpy(rows % 7 == 2)] = -np.inf
    kk, vv = k.clone(), v.clone()
    kk[:, dead], vv[:, dead] = float("nan"), float("inf")
    k[:, dead], v[:, dead] = 0.0, 0.0
    clean = run(A, q, k, v, vals, do)
    got = run(A, q, kk, vv, vals, do)
    for x, y in zip(got, clean):
        assert np.isfinite(x).all() and np.array_equal(x, y)
    compare(A, rp, ci, q, k, v, vals, do, code)


@pytest.mark.parametrize("code", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_column_stays_in_its_rows(code, bad):
    """A v that is not finite shows in the rows that attend to it and in no
    other row of the same work item."""
    A, rp, ci, q, k, v, vals, do = inputs("grid", 1, 2, 2, 64, code, False)
    clean = run(A, q, k, v, None, do)
    v2 = v.clone()
    v2[0, 100] = bad
    got = run(A, q, k, v2, None, do)
    rows = np.repeat(np.arange(rp.shape[0] - 1), np.diff(rp))
    hit = np.zeros(rp.shape[0] - 1, bool)
    hit[rows[ci == 100]] = True
    assert not np.isfinite(got[0][0, hit]).any()
    # rows that share work with a bad one are summed entry by entry, in another order
    # than otherwise: the bounds hold for any order, equal bits do not
    res, err = attention(rp, ci, *(x[0].double().numpy() for x in (q, k, v)), None, 64 ** -0.5, do[0].double().numpy(),
                         code)
    for x, y in (("o", 0), ("dq", 1)):
        assert within(got[y][0, ~hit], res[x][~hit], err[x][~hit]) <= 1.0
    far = ~hit & (np.abs(np.arange(rp.shape[0] - 1) - 100) > 40)       # work items that hold no bad row
    assert np.array_equal(got[0][0, far], clean[0][0, far]) and np.array_equal(got[1][0, far], clean[1][0, far])


def test_lowest_finite_values_are_no_mask():
    """A row whose values are all the lowest finite number weighs its entries
    alike (the products are lost against it), in 32 bits and from 64-bit values."""
    rp, ci, m = pattern("full")
    for vt in (torch.float32, torch.float64):
        A = sla.CSR(T(rp), T(ci), n_cols=m, dtype=vt)
        q, k, v = (torch.randn(s, 2, 64, device=DEV).bfloat16() for s in (37, m, m))
        vals = torch.full((A.nnz,), torch.finfo(vt).min, dtype=vt, device=DEV)
        for t in (torch.bfloat16, torch.float32):
            o = A.attention(q.to(t), k.to(t), v.to(t), vals)
            mean = v.double().mean(0).expand(37, 2, 64)
            # m equal weights: the mean, to the type's rounding and m + 16 roundings of 32 bits
            bound = (2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -24) * mean.abs() + \
                (2.0 ** -11 + (m + 16) * 2.0 ** -24) * v.double().abs().mean(0)
            assert ((o.double() - mean).abs() <= bound).all()


def test_values_of_a_64_bit_handle_with_16_bit_heads():
    rp, ci, m = pattern("hub")
    A = sla.CSR(T(rp), T(ci), n_cols=m, dtype=torch.float64)
    _, _, _, q, k, v, vals, do = inputs("hub", 1, 2, 2, 32, "bf16", True)
    got = compare(A, rp, ci, q, k, v, vals.double(), do, "bf16")
    assert got[4].dtype == np.float64


@pytest.mark.parametrize("code", ["f32", "bf16"])
def test_strides_and_alignment(code):
    """Views of a fused projection, head-major tensors, a last dimension that is
    not contiguous and an odd offset give the bits of contiguous tensors."""
    A, rp, ci, q, k, v, vals, do = inputs("hub", 2, 4, 4, 32, code, True)
    want = run(A, q, k, v, vals, do)
    fused = torch.stack([k, v], 2)                                  # [B, m, 2, K, D]
    got = run(A, q, fused[:, :, 0], fused[:, :, 1], vals, do)
    major = lambda t: t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)  # noqa: E731
    last = lambda t: t.transpose(2, 3).contiguous().transpose(2, 3)           # noqa: E731

    def odd(t):
        flat = torch.zeros(t.numel() + 1, dtype=t.dtype)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    def on_gpu(f, t):                                               # keeps the layout on the way
        return f(t.to(DEV))

    assert all(np.array_equal(x, y) for x, y in zip(got, want))
    for f in (major, last):
        ts = [on_gpu(f, t).requires_grad_() for t in (q, k, v)]
        o = A.attention(*ts, vals.to(DEV))
        g = torch.autograd.grad(o, ts, on_gpu(f, do))
        assert all(np.array_equal(H(x), y) for x, y in zip((o, *g), want))
    ts = []
    for t in (q, k, v):
        flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1).to(DEV)
        ts.append(flat[1:].view(t.shape).requires_grad_())
    o = A.attention(*ts, vals.to(DEV))
    g = torch.autograd.grad(o, ts, do.to(DEV))
    for b in range(2):                                              # another kernel: within the bounds
        res, err = attention(rp, ci, *(x[b].double().numpy() for x in (q, k, v)), vals[b].double().numpy(), 32 ** -0.5,
                             do[b].double().numpy(), code)
        for x, y in zip(("o", "dq", "dk", "dv"), (o, *g)):
            assert within(H(y)[b], res[x], err[x]) <= 1.0, x


def test_broadcast_inputs_sum_their_gradients():
    """Values shared by the systems, one key head for all and an output gradient
    of stride zero (o.sum()): autograd sums what was expanded."""
    A, rp, ci, q, k, v, vals, do = inputs("empty_rows", 3, 2, 2, 16, "f64", True)
    shared = vals[:1].to(DEV).requires_grad_()
    kk = k[:1].to(DEV).requires_grad_()
    o = A.attention(q.to(DEV), kk.expand(3, -1, -1, -1), v.to(DEV), shared.expand(3, -1))
    o.sum().backward()
    total, dk = 0.0, 0.0
    for b in range(3):
        res, _ = attention(rp, ci, *(x.double().numpy() for x in (q[b], k[0], v[b])), vals[0].numpy(), 0.25,
                           np.ones(q.shape[1:]), "f64")
        total, dk = total + res["dvals"], dk + res["dk"]
    # three systems' sums in 64 bits: far inside 1e-12 of the largest term
    assert np.max(np.abs(H(shared.grad)[0] - total)) < 1e-12 and np.max(np.abs(H(kk.grad)[0] - dk)) < 1e-12


def test_gradient_against_differences():
    """Central differences in 64 bits: step 1e-6, so cut-off near 1e-12 times the
    third derivative and cancellation near 1e-10 times the loss."""
    A, rp, ci, q, k, v, vals, do = inputs("empty_rows", 1, 2, 1, 8, "f64", True)
    got = run(A, q, k, v, vals, do)
    ts = [t.to(DEV) for t in (q, k, v, vals)]
    rng = np.random.default_rng(3)
    for x, t in enumerate(ts):
        d = torch.from_numpy(rng.standard_normal(t.shape)).to(DEV)
        side = []
        for sign in (1, -1):
            moved = [u + sign * 1e-6 * d if y == x else u for y, u in enumerate(ts)]
            side.append(float((A.attention(*moved) * do.to(DEV)).sum()))
        fd, an = (side[0] - side[1]) / 2e-6, float((torch.from_numpy(got[1 + x]).to(DEV) * d).sum())
        assert abs(fd - an) < 1e-7 * max(1.0, abs(an)), (x, fd, an)


@pytest.mark.parametrize("code", ["f32", "bf16"])
@pytest.mark.parametrize("n,m", [(0, 5), (3, 0), (0, 0)])
def test_no_rows_or_no_columns(n, m, code):
    rp = np.zeros(n + 1, np.int32)
    A = sla.CSR(T(rp), torch.zeros(0, dtype=torch.int32, device=DEV), n_cols=m, dtype=torch.float32)
    q = torch.randn(n, 2, 32, device=DEV).to(DT[code]).requires_grad_()
    k, v = (torch.randn(m, 2, 32, device=DEV).to(DT[code]).requires_grad_() for _ in range(2))
    vals = torch.zeros(0, device=DEV, requires_grad=True)
    o = A.attention(q, k, v, vals)
    assert o.shape == q.shape and not o.any()
    for g, t in zip(torch.autograd.grad(o, [q, k, v, vals], torch.ones_like(o)), (q, k, v, vals)):
        assert g.shape == t.shape and not g.any()


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in k and v: the last columns are read where they are."""
    m, H_, D = 1 << 21, 8, 136                       # 2^31 + 2^27 elements
    cols = [[0, m - 1], [m - 3], [m - 2, m - 1]]
    rp, ci, _ = from_rows(cols, m)
    A = sla.CSR(T(rp), T(ci), n_cols=m, dtype=torch.float32)
    for width, code in ((D, "bf16"), (128, "bf16")):         # a row kernel, and a tile kernel through the strides
        store = torch.zeros(m, H_, D, dtype=DT[code], device=DEV)
        k = store[:, :, :width]
        near = torch.tensor([0, m - 3, m - 2, m - 1], device=DEV)
        k[near] = torch.randn(4, H_, width, device=DEV).to(DT[code])
        q = torch.randn(3, H_, width, device=DEV).to(DT[code])
        got = H(A.attention(q, k, k))
        where = {0: 0, m - 3: 1, m - 2: 2, m - 1: 3}
        rp2, ci2, _ = from_rows([[where[c] for c in r] for r in cols], 4)
        small = H(k[near])
        res, err = attention(rp2, ci2, H(q), small, small, None, width ** -0.5, None, code)
        assert within(got, res["o"], err["o"]) <= 1.0
        del store, k


def test_only_the_asked_gradients():
    A, rp, ci, q, k, v, vals, do = inputs("hub", 1, 2, 1, 64, "bf16", True)
    want = run(A, q, k, v, vals, do)
    for x in range(4):
        ts = [t.to(DEV) for t in (q, k, v, vals)]
        ts[x].requires_grad_()
        (g,) = torch.autograd.grad(A.attention(*ts), [ts[x]], do.to(DEV))
        assert np.array_equal(H(g), want[1 + x])


def test_list_of_patterns_and_three_dimensions():
    """A list handle (items of their own patterns, block-diagonal) attends item by item."""
    items = [W.poisson2d(5)[:2], W.poisson2d(9)[:2], (np.array([0, 1]), np.array([0]))]
    A = sla.CSRList.from_items(items, dtype=torch.float32)
    n = 25 + 81 + 1
    q, k, v = (torch.randn(n, 2, 32, device=DEV) for _ in range(3))
    o = A.attention(q, k, v)
    assert o.shape == (n, 2, 32)
    for part, (rp, ci), (a, b) in zip(A.split(o), items, ((0, 25), (25, 106), (106, 107))):
        one = sla.CSR(T(np.asarray(rp, np.int32)), T(np.asarray(ci, np.int32)), dtype=torch.float32)
        assert torch.equal(one.attention(q[a:b], k[a:b], v[a:b]).reshape(-1), o[a:b].reshape(-1))


@pytest.mark.parametrize("code", ["f32", "bf16"])
def test_bits_repeat_and_other_stream(code):
    A, rp, ci, q, k, v, vals, do = inputs("hub", 2, 4, 2, 64, code, True)
    want = run(A, q, k, v, vals, do)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(A, q, k, v, vals, do)
    assert all(np.array_equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("code", ["f32", "bf16"])
def test_captured_and_replayed(code):
    """Forward and backward in one graph, replayed on new inputs; a first call
    inside a capture is refused, and two captured calls do not share workspace."""
    A, rp, ci, q, k, v, vals, do = inputs("hub", 1, 4, 2, 64, code, True)
    ts = [t.to(DEV).requires_grad_() for t in (q, k, v, vals)]
    g_out = do.to(DEV)
    A.prepare_attention(backward=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.autograd.grad(A.attention(*ts), ts, g_out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o1 = A.attention(*ts)
        o2 = A.attention(ts[0], ts[1], ts[2])
        grads = torch.autograd.grad(o1, ts, g_out)
    new = inputs("hub", 1, 4, 2, 64, code, True, seed=9)[3:]
    with torch.no_grad():
        for t, x in zip(ts, new[:4]):
            t.copy_(x)
        g_out.copy_(new[4])
    graph.replay()
    want = run(A, *new)
    assert all(np.array_equal(H(x), y) for x, y in zip((o1, *grads), want))
    assert np.array_equal(H(o2), H(A.attention(*(t.to(DEV) for t in new[:3]))))


def test_first_call_in_a_capture_is_refused():
    rp, ci, m = pattern("grid")
    A = sla.CSR(T(rp), T(ci), dtype=torch.float32)
    q = torch.randn(289, 2, 32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(L.SlaError, match="sla_attention_prepare"):
        with torch.cuda.graph(graph):
            A.attention(q, q, q)
    assert torch.isfinite(A.attention(q, q, q)).all()          # and the handle still works


def test_refusals():
    rp, ci, m = pattern("hub")
    A = sla.CSR(T(rp), T(ci), n_cols=m, batch=2, dtype=torch.float32)
    n = A.n_rows
    q, k = torch.randn(2, n, 4, 32, device=DEV), torch.randn(2, m, 2, 32, device=DEV)
    ok = A.attention(q, k, k)
    assert ok.shape == q.shape
    for args, kind in (((q[0], k, k), ValueError), ((q, k[:, :-1], k), ValueError), ((q, k, k[..., :16]), ValueError),
                       ((q[:, :, :3], k, k), ValueError), ((q.double(), k, k), TypeError),
                       ((q.cpu(), k, k), TypeError), ((q.int(), k.int(), k.int()), TypeError),
                       ((q, k[:, :, :0], k[:, :, :0]), ValueError)):
        with pytest.raises(kind):
            A.attention(*args)
    with pytest.raises(ValueError):
        A.attention(torch.randn(2, n, 1, 257, device=DEV), torch.randn(2, m, 1, 257, device=DEV), torch.randn(2, m, 1, 257, device=DEV))
    with pytest.raises(ValueError):
        A.attention(q, k, k, scale=float("inf"))
    with pytest.raises(TypeError):
        A.attention(q, k, k, torch.zeros(2, A.nnz, dtype=torch.float64, device=DEV))
    with pytest.raises(RuntimeError):
        A.attention(q, k, k, torch.zeros(2, A.nnz - 1, device=DEV))
    opts = L.make_attn_opts(torch.float32, 4, 2, 32, 1.0, q.stride()[:3], k.stride()[:3], k.stride()[:3])
    out, lse = torch.empty_like(q), torch.empty(2, n, 4, device=DEV)
    need = L.sla_attention_workspace_bytes(A.handle, opts, 0)
    assert need > 0                                        # a split row
    ws = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
    for bad in (ws[:need - 1], ws[1:need + 1]):
        with pytest.raises(L.SlaError, match="workspace"):
            L.sla_attention(A.handle, q, k, k, None, out, None, lse, opts, bad)


def test_a_training_step_with_the_other_operators():
    """Attention over a mesh learns edge weights of a Laplacian whose solve gives
    the loss; the gradients are clipped together.  Against the same chain in
    64-bit dense torch operations."""
    ei, ej = W.grid_edges((8, 8))
    n, E = 64, ei.shape[0]
    rp, ci, _ = W.weighted_laplacian(n, ei, ej, np.ones(E), 0.0)
    A = sla.CSR(T(rp), T(ci), dtype=torch.float64, symmetric=True)
    lap = sla.EdgeLaplacian(A, T(ei), T(ej))
    gen = torch.Generator(device=DEV).manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=torch.float64)  # noqa: E731
    feat, b = new(n, 16), new(n)
    weights = [(new(16, 16) / 4).requires_grad_() for _ in range(3)]
    bias = (0.3 * new(A.nnz)).requires_grad_()
    li, lj = (torch.from_numpy(x.astype(np.int64)).to(DEV) for x in (ei, ej))
    row = torch.from_numpy(np.repeat(np.arange(n), np.diff(rp))).to(DEV)
    col = T(ci).long()

    def loss(dense):
        q, k, v = ((feat @ w).reshape(n, 2, 8) for w in weights)
        if dense:
            s = torch.full((n, n), -torch.inf, device=DEV, dtype=torch.float64).index_put((row, col), bias)
            s = s + torch.einsum("ihd,jhd->hij", q, k) * 8 ** -0.5
            o = torch.einsum("hij,jhd->ihd", torch.softmax(s, 2), v)
        else:
            o = A.attention(q, k, v, bias)
        o = o.reshape(n, 16)
        w = torch.nn.functional.softplus((o[li] * o[lj]).sum(1))
        if dense:
            M = torch.diag(torch.full((n,), 0.1, device=DEV, dtype=torch.float64))
            M = M.index_put((li, lj), -w, accumulate=True).index_put((lj, li), -w, accumulate=True)
            M = M.index_put((li, li), w, accumulate=True).index_put((lj, lj), w, accumulate=True)
            x = torch.linalg.solve(M, b)
        else:
            x = lap.solve(w, b, 0.1, rtol=1e-13)
        return 0.5 * (x * x).sum()

    params = [*weights, bias]
    want = torch.autograd.grad(loss(True), params)
    loss(False).backward()
    for p, g in zip(params, want):
        # the solver's stated gradient accuracy (1e-6 at rtol 1e-10) holds with room at rtol 1e-13
        assert float((p.grad - g).norm() / g.norm()) < 1e-8
    total = float(torch.sqrt(sum((g * g).sum() for g in want)))
    norm = sla.clip_grad_norm_(params, 0.25 * total)
    assert abs(float(norm) - total) < 1e-7 * total
    after = float(torch.sqrt(sum((p.grad * p.grad).sum() for p in params)))
    assert abs(after - 0.25 * total) < 1e-5 * total


def test_counts_beyond_32_bits_are_refused():
    """16 heads on a key head repeat A^T's columns 16 times: 2^28 entries would wrap."""
    n, m = 1 << 12, 1 << 16
    rp = torch.arange(n + 1, dtype=torch.int32, device=DEV) * m
    A = sla.CSR(rp, torch.arange(m, dtype=torch.int32, device=DEV).repeat(n), n_cols=m, dtype=torch.float32)
    with pytest.raises((RuntimeError, ValueError), match="sharing a key head"):
        A.prepare_attention(backward=True, heads_per_key=16)
