"""Attention over a CSR pattern where 32-bit sums, weights and statistics can go
wrong: long rows, values far from the scores, and what the C calls give beside the
rounded output.  Against the definition in 64 bits.
"""
import numpy as np
import pytest
import torch

import differentiable_sparse_linear_csr_b200 as sla
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
