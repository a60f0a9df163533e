"""Attention and clipping: refusals that need no GPU, and the 64-bit definition
the GPU tests compare with against autograd and dense products."""
import ctypes

import numpy as np
import pytest
import torch

from differentiable_sparse_linear_csr_b200 import _lib as L
from tests.attention_oracle import attention


def test_attention_argument_errors_need_no_gpu():
    lib = L.lib()
    opts = L.make_attn_opts(torch.float32, 2, 1, 32, 1.0, (0, 0, 0), (0, 0, 0), (0, 0, 0))
    null = [None] * 8
    assert lib.sla_attention(*null, ctypes.byref(opts), None, 0, None) == L.SLA_ERR_INVALID
    assert "NULL handle" in L.sla_last_error_string()
    assert lib.sla_attention_grad(*([None] * 12), ctypes.byref(opts), None, 0, None) == L.SLA_ERR_INVALID
    assert lib.sla_attention_prepare(None, None, 1, None) == L.SLA_ERR_INVALID
    assert lib.sla_attention_workspace_bytes(None, ctypes.byref(opts), 0) == 0


def _list(*rows):
    words = [w for r in rows for w in r]
    return (ctypes.c_int64 * max(len(words), 1))(*words), len(rows)


@pytest.mark.parametrize("rows,message", [
    (((4096, 4096, 10, 7),), "dtype"),
    (((4096, 4096, -1, 1),), "count"),
    (((0, 4096, 10, 1),), "NULL"),
    (((4096, 0, 10, 1),), "NULL"),
    (((4098, 4096, 10, 1),), "aligned"),
    (((4096, 4097, 10, 2),), "aligned"),
    (((4096, 8192, 10, 1), (6000, 8192, 10, 1)), "shares memory"),           # one output twice
    (((4096, 8192, 10, 1), (6000, 8228, 10, 1)), "shares memory"),           # the last element of one
    (((4096, 4100, 10, 1),), "shares memory"),                               # over its own input, shifted
    (((4096, 8192, 10, 1), (8228, 12288, 10, 1)), "shares memory"),          # over another's input
    (((4096, 4096, 10, 0), (4096, 4096, 10, 0)), "shares memory"),           # in place, twice
])
def test_clip_refuses_bad_lists(rows, message):
    words, n = _list(*rows)
    st = L.lib().sla_clip_norm(n, words, 0, 1.0, 256, 1, 256, 1 << 20, None)
    assert st == L.SLA_ERR_INVALID and message in L.sla_last_error_string()


def test_clip_argument_errors_need_no_gpu():
    lib = L.lib()
    words, n = _list((4096, 4096, 10, 1))
    for bad in (-1.0, float("nan"), float("inf")):
        assert lib.sla_clip_norm(n, words, 0, bad, 256, 1, 256, 1 << 20, None) == L.SLA_ERR_INVALID
    assert lib.sla_clip_norm(n, words, 2, 1.0, 256, 1, 256, 1 << 20, None) == L.SLA_ERR_INVALID
    assert lib.sla_clip_norm(n, words, 0, 1.0, None, 1, 256, 1 << 20, None) == L.SLA_ERR_INVALID
    assert lib.sla_clip_norm(n, words, 0, 1.0, 256, 2, 256, 1 << 20, None) == L.SLA_ERR_INVALID
    assert lib.sla_clip_norm(n, words, 0, 1.0, 256, 1, 256, 64, None) == L.SLA_ERR_INVALID
    assert "workspace" in L.sla_last_error_string()
    assert lib.sla_clip_norm(n, words, 0, 1.0, 256, 1, 264, 1 << 20, None) == L.SLA_ERR_INVALID
    assert lib.sla_global_norm(-1, None, 0, 256, 1, 256, 1 << 20, None) == L.SLA_ERR_INVALID
    assert lib.sla_global_norm(2, None, 0, 256, 1, 256, 1 << 20, None) == L.SLA_ERR_INVALID
    assert lib.sla_norm_workspace_bytes(-1) == 0
    assert 0 < lib.sla_norm_workspace_bytes(0) <= lib.sla_norm_workspace_bytes(1000)


def test_definition_against_dense_autograd():
    rng = np.random.default_rng(0)
    rows = [np.sort(rng.choice(9, c, replace=False)) for c in (3, 9, 1, 5)]
    rp = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
    ci = np.concatenate(rows).astype(int)
    q, k, v, do = (rng.standard_normal(s) for s in ((4, 4, 8), (9, 2, 8), (9, 2, 8), (4, 4, 8)))
    vals = rng.standard_normal(len(ci))
    vals[1] = -np.inf
    res, err = attention(rp, ci, q, k, v, vals, 0.3, do, "f64")
    Q, K, V, B = (torch.tensor(x, requires_grad=True) for x in (q, k, v, vals))
    at = (torch.tensor(np.repeat(np.arange(4), np.diff(rp))), torch.tensor(ci))
    s = torch.full((4, 9), -torch.inf, dtype=torch.float64).index_put(at, B)
    s = s + torch.einsum("ihd,jhd->hij", Q, K.repeat_interleave(2, 1)) * 0.3
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s, 2), V.repeat_interleave(2, 1))
    got = torch.autograd.grad(o, [Q, K, V, B], torch.tensor(do))
    for x, t in zip(("o", "dq", "dk", "dv", "dvals"), (o, *got)):
        assert (np.abs(res[x] - t.detach().numpy()) <= err[x] + 1e-15).all(), x
