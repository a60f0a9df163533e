"""Attention under the bounds-checking build (run as a script).

Loads libsla_debug_bounds.so (SLA_LIBRARY_VARIANT=debug_bounds), in which every
column and entry the attention kernels take from a pattern is checked before
use.  Runs the row and tile kernels, forward and backward, on rows that are empty,
short, split and shared by few columns, compares them with the 64-bit definition
and requires a clean record; then plants one out-of-range column in a pattern
created without validation and requires the record to name it.  Prints
"debug bounds: ok" when every check holds.
"""
import os
import sys

os.environ["SLA_LIBRARY_VARIANT"] = "debug_bounds"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch         # noqa: E402

import differentiable_sparse_linear_csr_b200 as sla          # noqa: E402
from differentiable_sparse_linear_csr_b200 import _lib as L   # noqa: E402
from tests import test_gpu_attention as G                     # noqa: E402


def clean(label):
    torch.cuda.synchronize()
    v, code, idx = L.sla_debug_bounds_report()
    assert v == 0, f"{label}: {v} out-of-range indices, first code {code} index {idx}"
    print(f"{label}: ok")


def main():
    assert "bounds-checking" in L.sla_version(), L.sla_version()
    L.sla_debug_bounds_report(reset=True)
    for name in ("one", "one_row_long", "one_column", "full", "empty_rows", "no_entries", "hub", "grid"):
        for code, heads, kv, dim in (("f64", 2, 1, 16), ("f32", 4, 2, 32), ("f32", 1, 1, 33), ("bf16", 4, 4, 32),
                                     ("bf16", 2, 2, 64), ("f16", 4, 1, 128), ("f16", 3, 3, 48), ("bf16", 1, 1, 20)):
            G.compare(*G.inputs(name, 2, heads, kv, dim, code, True), code)
        clean(f"attention on {name}")
    # a v that is not finite: rows are redone entry by entry
    A, rp, ci, q, k, v, vals, do = G.inputs("grid", 1, 4, 2, 64, "bf16", True)
    v[0, 100] = float("nan")
    G.run(A, q, k, v, vals, do)
    clean("rows redone entry by entry")

    rp, ci, m = G.pattern("grid")
    bad = ci.copy()
    bad[-1] = m + 5                                    # the last row's last entry: rows stay sorted
    A = sla.CSR(G.T(rp), G.T(bad), n_cols=m, dtype=torch.float32, validate=False)
    for t in (torch.float32, torch.bfloat16):
        x = torch.randn(m, 2, 64, device=G.DEV).to(t)
        want = sla.CSR(G.T(rp), G.T(ci), dtype=torch.float32).attention(x, x, x)
        got = A.attention(x, x, x)
        torch.cuda.synchronize()
        n_bad, code, idx = L.sla_debug_bounds_report(reset=True)
        assert n_bad >= 1 and code == 1 and idx == m + 5, (n_bad, code, idx)
        assert torch.equal(got[:m - 1], want[:m - 1])
    clean("after reset")
    print("debug bounds: ok")


if __name__ == "__main__":
    main()
