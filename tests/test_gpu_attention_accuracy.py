"""Attention over a CSR pattern where 32-bit sums, weights and statistics can go
wrong: long rows, values far from the scores, and what the C calls give beside the
rounded output.  Against the definition in 64 bits.
"""
import numpy as np
import pytest
import torch

import differentiable_sparse_linear_csr_b200 as sla
from tests import attention_oracle
from tests.attention_oracle import attention, within

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f64": torch.float64, "f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def full_pattern(n, m, **kw):
    rp = torch.arange(n + 1, dtype=torch.int32, device=DEV) * m
    return sla.CSR(rp, torch.arange(m, dtype=torch.int32, device=DEV).repeat(n), n_cols=m, **kw)


def forward_parts(A, q, k, v, vals=None, scale=None):
    """(o, o before its rounding, lse) of the C call; q [n, H, D], k and v [m, K, D]."""
    from differentiable_sparse_linear_csr_b200 import _lib as L
    scale = q.shape[2] ** -0.5 if scale is None else scale
    opts = L.make_attn_opts(q.dtype, q.shape[1], k.shape[1], q.shape[2], scale,
                            *((0, *x.stride()[:2]) for x in (q, k, v)))
    wide = torch.float64 if q.dtype == torch.float64 else torch.float32
    o, o_wide = torch.empty_like(q), torch.empty(q.shape, dtype=wide, device=DEV)
    lse = torch.empty(q.shape[:2], dtype=wide, device=DEV)
    L.sla_attention_prepare(A.handle, opts)
    ws = torch.empty(max(1, L.sla_attention_workspace_bytes(A.handle, opts)), dtype=torch.uint8, device=DEV)
    L.sla_attention(A.handle, q, k, v, vals, o, o_wide, lse, opts, ws)
    return o, (o_wide if q.element_size() == 2 else o), lse


@pytest.mark.parametrize("code", ["bf16", "f16"])
def test_sums_of_long_rows_do_not_drift(code):
    """2003 entries a row, whole (64 heads): the mean error of sums of positive terms.
    A weight may lose up to 2^-20 of itself (what two 11-bit parts cannot hold) and a
    chunk's four products 2^-23 of their sum each, both always downwards; chunks are
    added with rounding to nearest, whose mean over all outputs is far below 2^-21.
    126 chunks that were added up in the truncating sums of the tensor core would drift
    by about 1e-5."""
    n, m, H, D = 300, 2003, 64, 16
    A = full_pattern(n, m, dtype=torch.float32)
    gen = torch.Generator(device=DEV).manual_seed(4)
    q, k = (torch.randn(s, H, D, generator=gen, device=DEV).to(DT[code]) for s in (n, m))
    v = (1 + torch.rand(m, H, D, generator=gen, device=DEV)).to(DT[code])
    _, o, _ = forward_parts(A, q, k, v)
    want = torch.empty(n, H, D, dtype=torch.float64, device=DEV)
    for h in range(H):
        want[:, h] = torch.softmax(q[:, h].double() @ k[:, h].double().T * D ** -0.5, 1) @ v[:, h].double()
    drift = float((o.double() / want - 1).mean())
    assert abs(drift) <= 2.0 ** -20 + 4 * 2.0 ** -23 + 2.0 ** -21, drift


def test_sums_of_long_columns_do_not_drift():
    """The same of dv, over columns of 2003 entries: 2^-20 more for the weights, which
    the backward pass forms anew, and the rounding of the float16 outputs, uniform
    within 2^-12 of 300 x 64 x 16 values."""
    n, m, H, D = 2003, 300, 64, 16
    A = full_pattern(n, m, dtype=torch.float32)
    gen = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn(s, H, D, generator=gen, device=DEV).half() for s in (n, m, m))
    do = (1 + torch.rand(n, H, D, generator=gen, device=DEV)).half()
    v.requires_grad_()
    (dv,) = torch.autograd.grad(A.attention(q, k, v), [v], do)
    want = torch.empty(m, H, D, dtype=torch.float64, device=DEV)
    for h in range(H):
        want[:, h] = torch.softmax(q[:, h].double() @ k[:, h].double().T * D ** -0.5, 1).T @ do[:, h].double()
    drift = float((dv.double() / want - 1).mean())
    assert abs(drift) <= 2 * 2.0 ** -20 + 4 * 2.0 ** -23 + 2.0 ** -21 + 4 * 2.0 ** -12 / np.sqrt(3 * want.numel()), drift


def left_padded(code, vt, low, level, heads=(2, 2), dim=64, m=70):
    """A full pattern whose first 10 to 64 columns hold the value `low` (rows differ),
    and what is left values around `level`: (A, q, k, v, vals, out) with out the
    same values and -inf in place of `low`."""
    n = 37
    A = full_pattern(n, m, dtype=vt)
    gen = torch.Generator(device=DEV).manual_seed(6)
    q, k, v = (torch.randn(s, h, dim, generator=gen, device=DEV).to(DT[code])
               for s, h in ((n, heads[0]), (m, heads[1]), (m, heads[1])))
    vals = level + torch.randn(n, m, generator=gen, device=DEV, dtype=vt)
    pad = torch.arange(m, device=DEV) < (10 + torch.arange(n, device=DEV) * 3 % 55)[:, None]
    return (A, q, k, v, torch.where(pad, torch.full_like(vals, low), vals).reshape(1, -1),
            torch.where(pad, torch.full_like(vals, -float("inf")), vals).reshape(1, -1))


LOWS = [-1e9, -1e10, -1e30, float(torch.finfo(torch.bfloat16).min), float(torch.finfo(torch.float32).min)]


def oracle_of(A, q, k, v, vals, do, code):
    num = lambda t: None if t is None else t.detach().double().cpu().numpy()  # noqa: E731
    return attention(A.rowptr.cpu().numpy(), A.colind.cpu().numpy(), num(q), num(k), num(v), num(vals)[0],
                     q.shape[2] ** -0.5, num(do), code)


@pytest.mark.parametrize("level", [-300.0, -100.0, 0.0, 86.0, 120.0])
@pytest.mark.parametrize("low", LOWS)
@pytest.mark.parametrize("code,heads", [("f32", (2, 2)), ("bf16", (2, 2)), ("f16", (8, 2))])
def test_low_finite_values_before_scores_of_any_size(code, heads, low, level):
    """Entries of a very low finite value have weight 0 beside others (exp of -1e9 is 0
    in 64 bits too), so the result is that of leaving them out, to its own bounds."""
    A, q, k, v, vals, out = left_padded(code, torch.float32, low, level, heads)
    o, wide, lse = forward_parts(A, q, k, v, vals)
    res, err = oracle_of(A, q, k, v, out, None, code)
    got = {"o": o, "lse": lse}
    assert all(within(t.double().cpu().numpy(), res[x], err[x]) <= 1.0 for x, t in got.items())


def test_low_finite_values_of_64_bits():
    """The same with a float64 handle, whose lowest number is beyond 32 bits."""
    low = float(torch.finfo(torch.float64).min)
    for code in ("f64", "bf16"):
        A, q, k, v, vals, out = left_padded(code, torch.float64, low, -100.0)
        o, _, lse = forward_parts(A, q, k, v, vals)
        res, err = oracle_of(A, q, k, v, out, None, code)
        assert within(o.double().cpu().numpy(), res["o"], err["o"]) <= 1.0
        assert within(lse.double().cpu().numpy(), res["lse"], err["lse"]) <= 1.0


def training(A, q, k, v, vals, do):
    ts = [t.clone().requires_grad_() for t in (q, k, v, vals)]
    o = A.attention(*ts)
    return [t.double().cpu().numpy() for t in (o.detach(), *torch.autograd.grad(o, ts, do))]


@pytest.mark.parametrize("level", [-10000.0, -1e9, -1e30, "lowest"])
@pytest.mark.parametrize("code,heads,dim", [("f64", (2, 2), 32), ("f32", (2, 2), 64), ("f32", (4, 1), 20), ("bf16", (2, 2), 64),
                                            ("bf16", (8, 2), 32), ("f16", (4, 4), 32), ("f16", (1, 1), 100)])
def test_gradients_of_rows_of_equal_low_values(code, heads, dim, level):
    """Rows whose entries all hold one very low finite value are the rows without it:
    softmax does not see what all scores share.  q = 0, so that no score is lost beside
    the value: every weight is 1 / n, and the gradients have closed forms,
        o = mean v,  ds_t = (do . v_t - do . mean v) / n,  dv = sum do / n,
        dq = scale sum_t ds_t k_t,  dk = 0,  dvals = sum over heads of ds.
    Every row also has a part beyond 64 entries that is split from it."""
    vt = torch.float64 if code == "f64" else torch.float32
    n, m = 37, 700
    A = full_pattern(n, m, dtype=vt)
    low = float(torch.finfo(vt).min) if level == "lowest" else level
    gen = torch.Generator(device=DEV).manual_seed(8)
    k, v, do = (torch.randn(s, h, dim, generator=gen, device=DEV, dtype=torch.float64).to(DT[code])
                for s, h in ((m, heads[1]), (m, heads[1]), (n, heads[0])))
    q = torch.zeros(n, heads[0], dim, device=DEV, dtype=DT[code])
    got = training(A, q, k, v, torch.full((1, m * n), low, dtype=vt, device=DEV), do)
    res, err = oracle_of(A, q, k, v, torch.zeros(1, m * n, device=DEV), do, code)
    assert np.array_equal(res["dk"], np.zeros_like(res["dk"]))
    worst = {x: within(g, res[x], err[x]) for x, g in zip(("o", "dq", "dk", "dv", "dvals"),
                                                          (got[0], got[1], got[2], got[3], got[4][0]))}
    assert all(w <= 1.0 for w in worst.values()), worst


@pytest.mark.parametrize("low", LOWS)
@pytest.mark.parametrize("code,heads", [("f32", (2, 2)), ("bf16", (2, 2)), ("f16", (8, 2))])
def test_gradients_with_low_finite_values_before_others(code, heads, low):
    """As in the forward pass: the gradients of leaving those entries out."""
    A, q, k, v, vals, out = left_padded(code, torch.float32, low, -100.0, heads)
    do = torch.randn(q.shape, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV).to(DT[code])
    got = training(A, q, k, v, vals, do)
    res, err = oracle_of(A, q, k, v, out, do, code)
    worst = {x: within(g, res[x], err[x]) for x, g in zip(("o", "dq", "dk", "dv", "dvals"), (*got[:4], got[4][0]))}
    assert all(w <= 1.0 for w in worst.values()), worst


def test_pairs_of_maximum_and_sum():
    """The C call's pairs (m, l) give lse, on whole and split rows, rows without an
    entry left and in every kind of kernel; gradients without pairs are refused."""
    from differentiable_sparse_linear_csr_b200 import _lib as L
    for code, heads, dim, m in (("f64", (2, 1), 16, 70), ("f32", (2, 2), 32, 700), ("bf16", (2, 2), 64, 70),
                                ("bf16", (2, 2), 64, 3000), ("f16", (8, 1), 16, 700)):
        vt = torch.float64 if code == "f64" else torch.float32
        for values in (True, False):
            A = full_pattern(5, m, dtype=vt)
            gen = torch.Generator(device=DEV).manual_seed(10)
            q, k = (torch.randn(s, h, dim, generator=gen, device=DEV).to(DT[code]) for s, h in zip((5, m), heads))
            vals = None
            if values:
                vals = 50 * torch.randn(5, m, generator=gen, device=DEV, dtype=vt)
                vals[3] = -float("inf")
                vals = vals.reshape(1, -1)
            opts = L.make_attn_opts(q.dtype, *heads, dim, 0.3, *((0, *x.stride()[:2]) for x in (q, k, k)), lse_pairs=True)
            o, ml = torch.empty_like(q), torch.empty(5, heads[0], 2, dtype=vt, device=DEV)
            L.sla_attention_prepare(A.handle, opts, 1)
            ws = torch.empty(max(1, L.sla_attention_workspace_bytes(A.handle, opts)), dtype=torch.uint8, device=DEV)
            L.sla_attention(A.handle, q, k, k, vals, o, None, ml, opts, ws)
            res, err = attention(A.rowptr.cpu().numpy(), A.colind.cpu().numpy(), *(x.double().cpu().numpy() for x in (q, k, k)),
                                 None if vals is None else vals[0].double().cpu().numpy(), 0.3, None, code)
            ml = ml.double().cpu().numpy()
            dead = ~np.isfinite(res["lse"])
            assert dead.any() == values and np.array_equal(ml[dead], np.tile([-np.inf, 0.0], (int(dead.sum()), 1)))
            got = ml[..., 0][~dead] + np.log(ml[..., 1][~dead])
            assert within(got, res["lse"][~dead], err["lse"][~dead]) <= 1.0
            opts.lse_pairs = 0
            room = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
            with pytest.raises(L.SlaError, match="lse_pairs"):
                L.sla_attention_grad(A.handle, q, k, k, vals, o, torch.empty(10, dtype=vt, device=DEV), q, q, None, None, None,
                                     opts, room)


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("at", range(4))
def test_forward_mode_is_refused(at, grad):
    """A tangent of any input is refused, not dropped, as matvec does; other inputs
    within a forward-mode level, and calls after it, are computed as before."""
    A = full_pattern(3, 5, dtype=torch.float32)
    ts = [torch.randn(s, 2, 16, device=DEV) for s in (3, 5, 5)] + [torch.randn(1, 15, device=DEV)]
    want = A.attention(*ts)
    with torch.set_grad_enabled(grad), torch.autograd.forward_ad.dual_level():
        dual = list(ts)
        dual[at] = torch.autograd.forward_ad.make_dual(ts[at], torch.ones_like(ts[at]))
        with pytest.raises((NotImplementedError, RuntimeError), match="jvp|forward"):
            A.attention(*dual)
        with pytest.raises((NotImplementedError, RuntimeError), match="jvp|forward"):
            A.attention(*(t[None] if t.dim() == 3 else t for t in dual))
        assert torch.equal(A.attention(*ts), want)
    assert torch.equal(A.attention(*ts), want)


def test_function_transforms_are_refused():
    A = full_pattern(3, 5, dtype=torch.float32)
    q, k = torch.randn(3, 2, 16, device=DEV), torch.randn(5, 2, 16, device=DEV)
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: A.attention(x, k, k), (q,), (q,))
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda x: A.attention(x, k, k))(q.expand(4, -1, -1, -1))
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda x: A.attention(x, k, k).sum())(q)


TIGHT = (2.0 ** -24, 2.0 ** -20)           # sums in 32 bits, weights to 2^-20 of themselves: both 16-bit types


def random_rows(lengths, heads, dim, code, seed=0, offset=0.0):
    """A pattern of rows of the given lengths, with values (every 7th -inf); keys share
    `offset` in every element."""
    rng = np.random.default_rng(11)
    m = max(lengths) + 13
    ci = np.concatenate([np.sort(rng.choice(m, size=c, replace=False)) for c in lengths]).astype(np.int32)
    rp = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    n = len(lengths)
    q, k, v, do = new(n, heads[0], dim), new(m, heads[1], dim) + offset, new(m, heads[1], dim), new(n, heads[0], dim)
    vt = torch.float64 if code == "f64" else torch.float32
    vals = new(1, ci.shape[0]).to(vt)
    vals[0, ::7] = -float("inf")
    A = sla.CSR(torch.from_numpy(rp).to(DEV), torch.from_numpy(ci).to(DEV), n_cols=m, dtype=vt)
    return A, *(x.to(DT[code]) for x in (q, k, v)), vals, do.to(DT[code])


ROWS = {"split": [60, 17, 64, 65, 5000, 0, 63, 1, 129, 16], "whole": [5, 0, 33, 64, 1, 16, 17, 40, 3]}


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("heads,dim", [((2, 2), 64), ((4, 4), 32), ((8, 1), 16), ((6, 2), 128), ((1, 1), 20)])
@pytest.mark.parametrize("code", ["f64", "f32", "bf16", "f16"])
def test_outputs_before_their_rounding(code, heads, dim, rows, monkeypatch):
    """o in 32 bits, lse, and the gradients to the bounds of weights in two parts, on
    whole and on joined rows."""
    A, q, k, v, vals, do = random_rows(ROWS[rows], heads, dim, code)
    if code in ("bf16", "f16"):
        ut = attention_oracle.CODES[code][1]
        monkeypatch.setitem(attention_oracle.CODES, code, (TIGHT[0], 0.0, TIGHT[1]))
    o, wide, lse = forward_parts(A, q, k, v, vals)
    res, err = oracle_of(A, q, k, v, vals, None, code)
    worst = {"wide": within(wide.double().cpu().numpy(), res["o"], err["o"]),
             "lse": within(np.where(np.isfinite(res["lse"]), lse.double().cpu().numpy(), 0.0),
                           np.where(np.isfinite(res["lse"]), res["lse"], 0.0), err["lse"])}
    assert np.array_equal(np.isneginf(lse.double().cpu().numpy()), np.isneginf(res["lse"]))
    assert torch.equal(o, wide.to(o.dtype))
    if code in ("bf16", "f16"):
        monkeypatch.setitem(attention_oracle.CODES, code, (TIGHT[0], ut, TIGHT[1]))
    got = training(A, q, k, v, vals, do)
    res, err = oracle_of(A, q, k, v, vals, do, code)
    worst |= {x: within(g, res[x], err[x]) for x, g in zip(("o", "dq", "dk", "dv", "dvals"), (*got[:4], got[4][0]))}
    assert all(w <= 1.0 for w in worst.values()), worst


@pytest.mark.parametrize("code", ["f32", "bf16", "f16"])
def test_what_keys_share_leaves_no_trace_in_dq(code):
    """256 keys of a row share an offset of 512: ds sums to zero over a row, so the
    offset cancels from dq = scale sum ds k if the weights ds keep their bits.  q = 0 and
    small integers elsewhere: p = 2^-8, dp, D (multiples of 2^-8) and ds (20 bits) are
    exact, so what is left is the rounding of the sums: 16 chunks to nearest, u each, and
    4 products of a chunk truncated, 2 u each (32-bit heads: 64 steps of 4 entries, their
    partial sums near zero like the total): 32 u sum |ds| |k| covers both; then the
    output's own.  Weights of 11 bits would be off by 2^-12 of each term."""
    n, m, H, D = 6, 256, 2, 64
    A = full_pattern(n, m, dtype=torch.float32)
    gen = torch.Generator(device=DEV).manual_seed(12)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=gen, device=DEV).double()  # noqa: E731
    K = 512 * torch.sign(ints(0, 1, D) - 0.5) + 4 * ints(-2, 2, m, H, D)
    V, G = ints(-8, 8, m, H, D), ints(-8, 8, n, H, D)
    q = torch.zeros(n, H, D, device=DEV, dtype=DT[code], requires_grad=True)
    k, v, do = (x.to(DT[code]) for x in (K, V, G))
    assert torch.equal(k.double(), K)
    (dq,) = torch.autograd.grad(A.attention(q, k, v), [q], do)
    dp = torch.einsum("ihd,jhd->ihj", G, V)
    ds = (dp - dp.mean(2, keepdim=True)) / m
    want = torch.einsum("ihj,jhd->ihd", ds, K) * D ** -0.5
    ut = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[code]
    bound = 32 * 2.0 ** -24 * torch.einsum("ihj,jhd->ihd", ds.abs(), K.abs()) * D ** -0.5 + ut * want.abs()
    assert bool(((dq.double() - want).abs() <= bound).all()), float(((dq.double() - want).abs() / bound).max())


@pytest.mark.parametrize("heads", [(64, 64), (64, 1), (66, 11)])
@pytest.mark.parametrize("code", ["f32", "bf16"])
def test_split_rows_with_many_heads(code, heads):
    """Plans for 64 and more systems and heads, with rows and columns that are split."""
    A, q, k, v, vals, do = random_rows(ROWS["split"], heads, 16, code, seed=3)
    got = training(A, q, k, v, vals, do)
    res, err = oracle_of(A, q, k, v, vals, do, code)
    worst = {x: within(g, res[x], err[x]) for x, g in zip(("o", "dq", "dk", "dv", "dvals"), (*got[:4], got[4][0]))}
    assert all(w <= 1.0 for w in worst.values()), worst


@pytest.mark.parametrize("vt", [torch.float32, torch.float64])
@pytest.mark.parametrize("code,heads,dim", [("f32", (2, 1), 32), ("f64", (2, 2), 16), ("bf16", (4, 2), 64), ("bf16", (2, 2), 128),
                                            ("f16", (4, 4), 16), ("bf16", (2, 2), 24)])
def test_workspaces_of_what_a_call_needs(code, heads, dim, vt):
    """Every set of gradients, with and without values, in a workspace of exactly the
    bytes asked for: the bits of the whole call, and nothing written behind it."""
    from differentiable_sparse_linear_csr_b200 import _lib as L
    A, q, k, v, vals, do = random_rows(ROWS["split"], heads, dim, code)
    A = sla.CSR(A.rowptr, A.colind, n_cols=A.n_cols, dtype=vt)
    vals = vals.to(vt)
    wide = torch.float64 if code == "f64" else torch.float32
    opts = L.make_attn_opts(q.dtype, *heads, dim, 0.25, *((0, *x.stride()[:2]) for x in (q, k, v, do)), lse_pairs=True)
    L.sla_attention_prepare(A.handle, opts, 1)

    def room(what):
        need = L.sla_attention_workspace_bytes(A.handle, opts, what)
        return need, torch.full((need + 4096,), 171, dtype=torch.uint8, device=DEV)

    for has_values in (True, False):
        x = vals if has_values else None
        no = 0 if has_values else L.SLA_ATTN_NO_VALS
        o, o_wide = torch.empty_like(q), torch.empty(q.shape, dtype=wide, device=DEV)
        ml = torch.empty(*q.shape[:2], 2, dtype=wide, device=DEV)
        need, ws = room(no)
        L.sla_attention(A.handle, q, k, v, x, o, o_wide, ml, opts, ws[:need])
        assert bool((ws[need:] == 171).all())
        whole = None
        for wanted in range(15 if has_values else 7, 0, -1):
            dq, dk, dv = (torch.empty_like(t) if wanted >> i & 1 else None for i, t in enumerate((q, k, v)))
            dvals = torch.empty_like(vals) if wanted & 8 else None
            need, ws = room(1 | no | (0 if dvals is not None else L.SLA_ATTN_NO_DVALS) | (0 if dq is not None else L.SLA_ATTN_NO_DQ) |
                            (0 if dk is not None or dv is not None else L.SLA_ATTN_NO_DK_DV))
            assert need <= L.sla_attention_workspace_bytes(A.handle, opts, 1)
            L.sla_attention_grad(A.handle, q, k, v, x, o_wide if q.element_size() == 2 else o, ml, do, dq, dk, dv, dvals, opts,
                                 ws[:need])
            assert bool((ws[need:] == 171).all())
            whole = whole or (dq, dk, dv, dvals)
            assert all(t is None or torch.equal(t, u) for t, u in zip((dq, dk, dv, dvals), whole)), wanted
            if need > 0:
                with pytest.raises(L.SlaError, match="workspace"):
                    L.sla_attention_grad(A.handle, q, k, v, x, o_wide if q.element_size() == 2 else o, ml, do, dq, dk, dv, dvals,
                                         opts, ws[:need - 1])


def test_training_asks_for_no_memory_that_it_leaves_alone():
    """A million entries and 16 heads: 67 MB for 32-bit ds of every entry and head, which
    only the values' gradient reads, and 134 MB for pairs (p, ds), which dq does not."""
    A = full_pattern(512, 2048, dtype=torch.float32)
    for code, only_q in (("bf16", False), ("f32", True)):
        q, k, v = (torch.randn(s, 16, 16, device=DEV).to(DT[code]) for s in (512, 2048, 2048))
        ts = [q.requires_grad_()] if only_q else [t.requires_grad_() for t in (q, k, v)]
        do = torch.randn_like(q)
        torch.autograd.grad(A.attention(q, k, v), ts, do)
        o = A.attention(q, k, v)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        torch.autograd.grad(o, ts, do)
        torch.cuda.synchronize()
        assert torch.cuda.max_memory_allocated() - before < 32 << 20
