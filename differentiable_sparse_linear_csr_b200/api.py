"""PyTorch surface of the library: a shared-pattern CSR matrix with
autograd-aware `solve` and `matvec`.

Mirrors the API of "torch-sla: Differentiable Sparse Linear Algebra with Adjoint
Solvers and Sparse Tensor Parallelism for PyTorch" (technical summary,
"Methodology" 1: `.solve`, `.matvec`, a SparseTensor holding one matrix or a
batch sharing one pattern; "Methodology" 2: the backward of a linear solve is
one adjoint solve A^T lambda = dL/dx, then dL/db = lambda and
dL/dA_ij = -lambda_i x_j on the pattern, so autograd stores O(1) nodes and
O(n + nnz) memory whatever the iteration count).

PyTorch provides device memory, streams and autograd bookkeeping; every step of
the computation runs in libsla.so's kernels (see _lib.py).
"""
from __future__ import annotations

import contextlib
import math
import operator
from dataclasses import dataclass

import torch
from torch.autograd import forward_ad

from . import _lib as L


@dataclass
class SolveInfo:
    """Per-system outcome of a solve, kept on the device (no host sync)."""
    iters: torch.Tensor      # int32 [B]
    relres: torch.Tensor     # float64 [B]
    status: torch.Tensor     # int32 [B], see _lib.STATUS_NAMES


def _workspace(nbytes: int, device) -> torch.Tensor:
    # the caching allocator hands out blocks aligned to 512 bytes
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _new_info(B: int, device) -> SolveInfo:
    return SolveInfo(torch.empty(B, dtype=torch.int32, device=device),
                     torch.empty(B, dtype=torch.float64, device=device),
                     torch.empty(B, dtype=torch.int32, device=device))


class CSR:
    """A CSR pattern on the GPU shared by ``batch`` value sets of one dtype.

    rowptr: int32 [n_rows + 1], colind: int32 [nnz] (device tensors, kept alive
    by this object).  Values and vectors are passed per call, batch-major:
    values [B, nnz] (or [nnz] when B == 1), vectors [B, n] (or [n]).
    ``symmetric=True`` asserts A^T == A for every value set, so the adjoint
    solve reuses the forward pattern and values unchanged.
    """

    def __init__(self, rowptr: torch.Tensor, colind: torch.Tensor, n_cols: int | None = None,
                 batch: int = 1, dtype: torch.dtype = torch.float64, symmetric: bool = False,
                 validate: bool = True, build_transpose: bool = False):
        if rowptr.device.type != "cuda" or colind.device.type != "cuda":
            raise ValueError("CSR needs CUDA tensors")
        self.rowptr = rowptr.to(torch.int32).contiguous()
        self.colind = colind.to(torch.int32).contiguous()
        self.n_rows = self.rowptr.numel() - 1
        self.n_cols = self.n_rows if n_cols is None else int(n_cols)
        self.nnz = self.colind.numel()
        self.batch = int(batch)
        self.dtype = dtype
        self.device = self.rowptr.device
        self.symmetric = bool(symmetric)
        flags = (L.SLA_FLAG_VALIDATE if validate else 0) | (L.SLA_FLAG_SYMMETRIC if symmetric else 0) \
            | (L.SLA_FLAG_BUILD_TRANSPOSE if build_transpose else 0)
        with torch.cuda.device(self.device):
            self.handle = L.sla_csr_create(self.n_rows, self.n_cols, self.nnz, self.rowptr, self.colind,
                                           self.batch, L.dtype_code(dtype), flags)
        self.n_info = self.batch                 # entries of a solve's SolveInfo
        self._attn_calls = {}
        self.last_info: SolveInfo | None = None
        self.last_adjoint_info: SolveInfo | None = None

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            try:
                torch.cuda.synchronize(self.device)
                L.sla_csr_destroy(h)
            except Exception:
                pass
            self.handle = None

    @property
    def props(self) -> L.sla_csr_props:
        return L.sla_csr_get_props(self.handle)

    # ------------------------------------------------------------ shapes
    def _values(self, values: torch.Tensor) -> torch.Tensor:
        v = values.reshape(self.batch, self.nnz)
        if v.dtype != self.dtype or v.device != self.device:
            raise TypeError(f"values must be {self.dtype} on {self.device}")
        return v.contiguous()

    def _vec(self, x: torch.Tensor, n: int) -> torch.Tensor:
        v = x.reshape(self.batch, n)
        if v.dtype != self.dtype or v.device != self.device:
            raise TypeError(f"vectors must be {self.dtype} on {self.device}")
        return v.contiguous()

    # -------------------------------------------------------- primitives
    def spmv(self, values, x, transpose: bool = False) -> torch.Tensor:
        """y = op(A) x without autograd (op = A or A^T)."""
        v = self._values(values)
        xin = self._vec(x, self.n_rows if transpose else self.n_cols)
        y = torch.empty(self.batch, self.n_cols if transpose else self.n_rows,
                        dtype=self.dtype, device=self.device)
        L.sla_spmv(self.handle, v, xin, y, int(transpose), 1.0, 0.0)
        return y

    def cg(self, values, b, *, adjoint=False, rtol=1e-10, atol=0.0, max_iter=0, fixed_iters=0,
           precond=True, x0=None, strategy=L.SLA_STRATEGY_AUTO, wait_timeout_ns=0):
        """Solve A x = b (or A^T x = b) without autograd; returns (x, SolveInfo)."""
        v = self._values(values)
        rhs = self._vec(b, self.n_rows)
        x = self._vec(x0, self.n_rows).clone() if x0 is not None else \
            torch.empty(self.batch, self.n_rows, dtype=self.dtype, device=self.device)
        info = _new_info(self.n_info, self.device)
        opts = L.make_opts(rtol, atol, max_iter, fixed_iters, precond, x0 is not None,
                           wait_timeout_ns, strategy)
        op = L.SLA_OP_ADJOINT if adjoint else L.SLA_OP_CG
        ws = _workspace(L.sla_workspace_bytes(self.handle, op), self.device)
        fn = L.sla_cg_adjoint if adjoint else L.sla_cg_solve
        fn(self.handle, v, rhs, x, opts, L.make_info(info.iters, info.relres, info.status), ws)
        return x, info

    def grad_values(self, lam, x, out=None, accumulate=False) -> torch.Tensor:
        """dL/dvalues[t] = -lam[row t] * x[col t] on the pattern."""
        lm = self._vec(lam, self.n_rows)
        xv = self._vec(x, self.n_cols)
        g = out if out is not None else torch.empty(self.batch, self.nnz, dtype=self.dtype,
                                                    device=self.device)
        L.sla_grad_values(self.handle, lm, xv, g, int(accumulate))
        return g

    def matvec_grad_values(self, gy, x, out=None, accumulate=False) -> torch.Tensor:
        """dL/dvalues[t] = gy[row t] * x[col t] on the pattern (for y = A x)."""
        gv = self._vec(gy, self.n_rows)
        xv = self._vec(x, self.n_cols)
        g = out if out is not None else torch.empty(self.batch, self.nnz, dtype=self.dtype,
                                                    device=self.device)
        L.sla_matvec_grad_values(self.handle, gv, xv, g, int(accumulate))
        return g

    # ---------------------------------------------------- autograd calls
    def matvec(self, values, x) -> torch.Tensor:
        """y = A x, differentiable in values and x."""
        return _MatVec.apply(self, values, x)

    def solve(self, values, b, *, rtol=1e-10, atol=0.0, max_iter=0, fixed_iters=0, precond=True,
              strategy=L.SLA_STRATEGY_AUTO) -> torch.Tensor:
        """x = A^-1 b by Jacobi-PCG, differentiable in values and b through one
        adjoint solve with the same options."""
        opts = dict(rtol=rtol, atol=atol, max_iter=max_iter, fixed_iters=fixed_iters,
                    precond=precond, strategy=strategy)
        return _Solve.apply(self, values, b, opts)


    # --------------------------------------------------------- attention
    def prepare_attention(self, backward: bool = False, heads_per_key: int = 1) -> None:
        """Build the work plan of ``attention`` (and, with ``backward``, A^T's
        pattern and plan) now instead of at the first call: needed before the
        calls are captured into a CUDA graph.  heads_per_key: H // K of the calls.
        Synchronises the host.  A captured backward pass also needs that no graph of
        the same leaves made outside the capture is still alive (drop the warm-up's
        outputs): autograd would tie the capture to that graph's stream."""
        if heads_per_key < 1:
            raise ValueError("heads_per_key must be positive")
        with _on_device(self.device):
            L.sla_attention_prepare(self.handle, None, backward)
            if heads_per_key > 1:
                opts = L.make_attn_opts(torch.bfloat16, heads_per_key, 1, 16, 1.0, (0, 0, 0), (0, 0, 0), (0, 0, 0))
                L.sla_attention_prepare(self.handle, opts, backward)

    def attention(self, q, k, v, values=None, *, scale: float | None = None) -> torch.Tensor:
        """Attention over the pattern: row i of A is a query that attends to the
        columns stored in that row,

            s_t = scale * q_i . k_j + values_t,  o_i = sum_t softmax(s)_t v_j,

        differentiable in q, k, v and values.  q: [B, n_rows, H, D], k and v:
        [B, n_cols, K, D] (without the leading dimension when B == 1), of one type
        among float64, float32, bfloat16 and float16 (which need not be A's), D at
        most 256, H a multiple of K (query head h reads key head h // (H // K)).
        values [B, nnz] (A's dtype, shared by the heads) are added to the scores;
        an entry whose value is -inf is left out, whatever its k and v hold.  A
        row with no entry left gives zeros.  scale defaults to D ** -0.5.  A tensor's
        last dimension is copied if it is not contiguous, and in 16 bits a tensor
        whose rows do not start on 16 bytes; other strides are used as they are.
        Returns o shaped like q.  Sums have a fixed order: equal calls give equal
        bits.  Forward-mode derivatives are refused.
        """
        scale = None if scale is None else float(scale)
        # what depends on shapes, strides and types alone is checked and laid out once
        key = (q.shape, k.shape, v.shape, q.stride(), k.stride(), v.stride(), q.dtype, k.dtype, v.dtype,
               q.device, k.device, v.device, scale, values is None)
        call = self._attn_calls.get(key)
        if call is None:
            call = _AttentionCall(self, q, k, v, values, scale)
            if len(self._attn_calls) >= 64:
                self._attn_calls.clear()
            self._attn_calls[key] = call
        # inside a forward-mode level the function refuses inputs that carry a tangent
        if (torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or
                                         (values is not None and values.requires_grad))) or _forward_mode():
            if q.dim() == 3:
                return _Attention.apply(self, call, q.unsqueeze(0), k.unsqueeze(0), v.unsqueeze(0), values).squeeze(0)
            return _Attention.apply(self, call, q, k, v, values)
        return call.forward(self, q, k, v, values, False)[0]


class CSRList(CSR):
    """Independent square systems with their own patterns (torch-sla's
    SparseTensorList, technical summary, "Methodology" 1), held as one
    block-diagonal CSR: item s owns rows and columns [item_rows[s],
    item_rows[s+1]).  Values [nnz] and vectors [n_rows] are the items'
    concatenations; ``solve`` / ``cg`` solve every item on its own (SolveInfo
    per item), ``matvec`` and the gradients act item by item as they must for a
    block-diagonal matrix.  Build one with ``CSRList.from_items``.
    """

    def __init__(self, item_rows: torch.Tensor, rowptr: torch.Tensor, colind: torch.Tensor,
                 dtype: torch.dtype = torch.float64, symmetric: bool = False, validate: bool = True):
        if rowptr.device.type != "cuda" or colind.device.type != "cuda":
            raise ValueError("CSRList needs CUDA tensors")
        self.rowptr = rowptr.to(torch.int32).contiguous()
        self.colind = colind.to(torch.int32).contiguous()
        self.item_rows = item_rows.to(device=self.rowptr.device, dtype=torch.int32).contiguous()
        self.n_rows = self.n_cols = self.rowptr.numel() - 1
        self.nnz = self.colind.numel()
        self.batch = 1
        self.n_items = self.item_rows.numel() - 1
        self.dtype = dtype
        self.device = self.rowptr.device
        self.symmetric = bool(symmetric)
        flags = (L.SLA_FLAG_VALIDATE if validate else 0) | (L.SLA_FLAG_SYMMETRIC if symmetric else 0)
        with torch.cuda.device(self.device):
            self.handle = L.sla_csr_list_create(self.n_items, self.item_rows, self.n_rows, self.nnz,
                                                self.rowptr, self.colind, L.dtype_code(dtype), flags)
        self.n_info = self.n_items
        self._attn_calls = {}
        self.last_info = None
        self.last_adjoint_info = None

    @classmethod
    def from_items(cls, items, dtype=torch.float64, symmetric=False, validate=True, device=None):
        """items: sequence of (rowptr, colind) per item (local indices)."""
        rps, cis, rows, ents = [], [], [0], [0]
        for rp, ci in items:
            rp = torch.as_tensor(rp, dtype=torch.int64, device=device)
            ci = torch.as_tensor(ci, dtype=torch.int64, device=device)
            rps.append(rp[:-1] + ents[-1])
            cis.append(ci + rows[-1])
            rows.append(rows[-1] + rp.numel() - 1)
            ents.append(ents[-1] + ci.numel())
        rowptr = torch.cat(rps + [torch.tensor([ents[-1]], dtype=torch.int64, device=rps[0].device)])
        colind = torch.cat(cis)
        item_rows = torch.tensor(rows, dtype=torch.int64)
        dev = device or torch.device("cuda")
        return cls(item_rows.to(dev), rowptr.to(dev), colind.to(dev), dtype=dtype, symmetric=symmetric,
                   validate=validate)

    def split(self, t: torch.Tensor, per: str = "rows"):
        """Per-item views of a concatenated vector (per='rows') or of values
        (per='entries')."""
        bounds = self.item_rows.tolist() if per == "rows" else \
            self.rowptr[self.item_rows.long()].tolist()
        t = t.reshape(-1)
        return [t[a:b] for a, b in zip(bounds[:-1], bounds[1:])]


class _MatVec(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A: CSR, values, x):
        y = A.spmv(values, x)
        ctx.A = A
        ctx.save_for_backward(values, x)
        return y.reshape(x.shape[:-1] + (A.n_rows,))

    @staticmethod
    def backward(ctx, gy):
        A = ctx.A
        values, x = ctx.saved_tensors
        gv = gx = None
        gy = A._vec(gy, A.n_rows)
        if ctx.needs_input_grad[2]:
            gx = A.spmv(values, gy, transpose=True).reshape(x.shape)
        if ctx.needs_input_grad[1]:
            gv = A.matvec_grad_values(gy, x).reshape(values.shape)   # dy_i/dA_ij = x_j
        return None, gv, gx


class _Solve(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A: CSR, values, b, opts):
        x, info = A.cg(values, b, **opts)
        A.last_info = info
        ctx.A, ctx.opts = A, opts
        ctx.save_for_backward(values, x)
        return x.reshape(b.shape)

    @staticmethod
    def backward(ctx, gx):
        A, opts = ctx.A, ctx.opts
        values, x = ctx.saved_tensors
        lam, info = A.cg(values, gx.contiguous(), adjoint=True, **opts)
        A.last_adjoint_info = info
        gv = A.grad_values(lam, x).reshape(values.shape) if ctx.needs_input_grad[1] else None
        gb = lam.reshape(gx.shape) if ctx.needs_input_grad[2] else None
        return None, gv, gb, None


def _forward_mode() -> bool:
    return getattr(forward_ad, "_current_level", 0) >= 0


def _on_device(device):
    """The device as the current one; nothing to enter where it is already."""
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


_HERE = contextlib.nullcontext()


def _aligned(x: torch.Tensor) -> bool:
    """Rows of 16-bit heads start on 16 bytes."""
    st = x.stride()
    return not ((st[-2] | st[-3] | (st[0] if x.dim() == 4 else 0)) & 7 or x.data_ptr() & 15)


def _head_layout(x: torch.Tensor, whole: bool) -> torch.Tensor:
    """x as the kernels read it: the last dimension contiguous and, with `whole`,
    rows on 16 bytes; a copy if it is not."""
    if x.stride(-1) != 1 or (whole and not _aligned(x)):
        x = x.clone(memory_format=torch.contiguous_format)
    return x


class _AttentionCall:
    """What calls of one set of shapes, strides and types share."""

    def __init__(self, A: CSR, q, k, v, values, scale):
        for x, n, name in ((q, A.n_rows, "q"), (k, A.n_cols, "k"), (v, A.n_cols, "v")):
            if tuple(x.shape[:-2]) != (A.batch, n) and not (A.batch == 1 and tuple(x.shape[:-2]) == (n,)):
                raise ValueError(f"{name} must be [{A.batch}, {n}, heads, dim] (got {tuple(x.shape)})")
            if x.dim() != q.dim():
                raise ValueError("q, k and v must have the same number of dimensions")
            if x.device != A.device:
                raise TypeError(f"{name} must be on {A.device}")
        if not (q.dtype == k.dtype == v.dtype) or q.dtype not in L.TENSOR_DTYPES:
            raise TypeError("q, k and v must share one type: float64, float32, bfloat16 or float16")
        (H, D), K = q.shape[-2:], k.shape[-2]
        if k.shape != v.shape or k.shape[-1] != D:
            raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must have one shape, with q's last "
                             f"dimension ({D})")
        if K == 0 or H == 0 or H % K:
            raise ValueError(f"q's {H} heads are not a multiple of k's {K}")
        if not 1 <= D <= 256:
            raise ValueError(f"heads of {D} elements (1 to 256)")
        self.scale = D ** -0.5 if scale is None else float(scale)
        if not math.isfinite(self.scale):
            raise ValueError("scale must be finite")
        self.size = (q.dtype, H, K, D)
        self.whole = q.element_size() == 2 and D % 8 == 0
        self.wide = torch.float64 if q.dtype == torch.float64 else torch.float32
        self.lse = A.batch * A.n_rows * H * (8 if q.dtype == torch.float64 else 4)
        self.ready = [False, False]
        self.rooms = {}
        self.opts = [self.options(q, k, v, pairs=train) for train in (False, True)]
        self.back = {}                           # options of the gradients, by the strides they depend on

    def options(self, q, k, v, do=None, pairs=True):
        def strides(x):
            st = x.stride()
            return st[:3] if len(st) == 4 else (0, *st[:2])

        return L.make_attn_opts(*self.size, self.scale, strides(q), strides(k), strides(v),
                                (0, 0, 0) if do is None else strides(do), pairs)

    def prepare(self, A, opts, backward):
        if not self.ready[backward]:
            L.sla_attention_prepare(A.handle, opts, backward)
            self.ready[0] = self.ready[backward] = True

    def room(self, A, opts, what):
        """Workspace bytes of a prepared call (what: see sla_attention_workspace_bytes)."""
        n = self.rooms.get(what)
        if n is None:
            n = self.rooms[what] = L.sla_attention_workspace_bytes(A.handle, opts, what)
        return n

    def forward(self, A, q, k, v, values, train):
        """(o, its 32-bit form or None, the rows' (m, l) or None, q, k, v as the kernels read them)"""
        vals = None if values is None else A._values(values)
        opts, given = self.opts[train], (q, k, v)
        q, k, v = _head_layout(q, self.whole), _head_layout(k, self.whole), _head_layout(v, self.whole)
        if q is not given[0] or k is not given[1] or v is not given[2]:
            opts = self.options(q, k, v, pairs=train)
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        with _on_device(A.device):
            self.prepare(A, opts, train)
            room = self.room(A, opts, 0 if vals is not None else L.SLA_ATTN_NO_VALS)
            if train:
                lse = torch.empty(A.batch, A.n_rows, q.shape[-2], 2, dtype=self.wide, device=A.device)
                wide = torch.empty(out.shape, dtype=self.wide, device=A.device) if q.element_size() == 2 else None
                L.sla_attention(A.handle, q, k, v, vals, out, wide, lse, opts,
                                _workspace(room, A.device) if room else None)
                return out, wide, lse, q, k, v
            ws = _workspace(room + self.lse, A.device)      # lse behind the workspace proper
            L.sla_attention(A.handle, q, k, v, vals, out, None, None, opts, ws, lse_ptr=ws.data_ptr() + room)
        return out, None, None, q, k, v


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A: CSR, call: _AttentionCall, q, k, v, values):
        out, wide, lse, q, k, v = call.forward(A, q, k, v, values, True)
        ctx.A, ctx.call = A, call
        ctx.save_for_backward(q, k, v, values, out if wide is None else wide, lse)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, go):
        A, call = ctx.A, ctx.call
        q, k, v, values, out, lse = ctx.saved_tensors
        go = _head_layout(go, call.whole)
        vals = None if values is None else A._values(values)
        new = lambda need, t: torch.empty_like(t, memory_format=torch.contiguous_format) if need else None  # noqa: E731
        dq, dk, dv, dvals = (new(need, t) for need, t in zip(ctx.needs_input_grad[2:6], (q, k, v, values)))
        with _on_device(A.device):
            key = (q.stride(), k.stride(), v.stride(), go.stride())
            opts = call.back.get(key)
            if opts is None:
                opts = call.back[key] = call.options(q, k, v, go)
            what = 1 | (0 if vals is not None else L.SLA_ATTN_NO_VALS) | \
                (0 if dvals is not None else L.SLA_ATTN_NO_DVALS) | (0 if dq is not None else L.SLA_ATTN_NO_DQ) | \
                (0 if dk is not None or dv is not None else L.SLA_ATTN_NO_DK_DV)
            ws = _workspace(call.room(A, opts, what), A.device)
            L.sla_attention_grad(A.handle, q, k, v, vals, out, lse, go, dq, dk, dv, dvals, opts, ws)
        return None, None, dq, dk, dv, dvals


class EdgeLaplacian:
    """A = L_w + diag(shift) on the pattern of ``A``: the map from edge
    conductivities to matrix values of inverse coefficient learning ("torch-sla",
    technical summary, "Experimental results", end-to-end application).

    For undirected edges e = (ei[e], ej[e]) (int32 [E] device tensors, each pair
    once, both entries and every diagonal stored in the pattern):
    A_ij = A_ji = -w_e and A_ii = (i's edge weights, ascending neighbour index)
    + shift.  ``assemble`` and ``solve`` are differentiable in w, shift (and b);
    ``solve`` assembles, solves, and in its backward runs one adjoint solve and
    the fused edge-gradient kernel, never forming dL/dvalues.
    """

    def __init__(self, A: CSR, ei: torch.Tensor, ej: torch.Tensor):
        self.A = A
        self.ei = ei.to(device=A.device, dtype=torch.int32).contiguous()
        self.ej = ej.to(device=A.device, dtype=torch.int32).contiguous()
        self.n_edges = self.ei.numel()
        if self.ej.numel() != self.n_edges:
            raise ValueError("ei and ej must have the same length")
        with torch.cuda.device(A.device):
            self.plan = L.sla_edges_create(A.handle, self.n_edges, self.ei, self.ej)

    def __del__(self):
        p = getattr(self, "plan", None)
        if p:
            try:
                torch.cuda.synchronize(self.A.device)
                L.sla_edges_destroy(p)
            except Exception:
                pass
            self.plan = None

    def _w(self, w: torch.Tensor) -> torch.Tensor:
        A = self.A
        v = w.reshape(A.batch, self.n_edges)
        if v.dtype != A.dtype or v.device != A.device:
            raise TypeError(f"weights must be {A.dtype} on {A.device}")
        return v.contiguous()

    def _shift(self, shift):
        A = self.A
        if shift is None:
            return None
        if not torch.is_tensor(shift):
            return torch.full((A.batch,), float(shift), dtype=A.dtype, device=A.device)
        s = shift.reshape(-1)
        if s.numel() == 1 and A.batch > 1:
            s = s.expand(A.batch)
        if s.dtype != A.dtype or s.device != A.device:
            raise TypeError(f"shift must be {A.dtype} on {A.device}")
        return s.contiguous()

    # -------------------------------------------------------- primitives
    def assemble_values(self, w, shift=None) -> torch.Tensor:
        """values [B, nnz] of L_w + shift I, without autograd."""
        A = self.A
        vals = torch.empty(A.batch, A.nnz, dtype=A.dtype, device=A.device)
        L.sla_laplacian_assemble(self.plan, self._w(w), self._shift(shift), vals)
        return vals

    def _grads(self, fn, args, dw, dshift, accumulate, want_shift, shared_shift):
        A = self.A
        dw = dw if dw is not None else torch.empty(A.batch, self.n_edges, dtype=A.dtype, device=A.device)
        if dshift is None and want_shift:
            dshift = torch.empty(1 if shared_shift else A.batch, dtype=A.dtype, device=A.device)
        ws = _workspace(L.sla_edges_workspace_bytes(self.plan), A.device) if dshift is not None else None
        flags = (L.SLA_GRAD_ACCUMULATE if accumulate else 0) | \
            (L.SLA_GRAD_SHIFT_SHARED if shared_shift else 0)
        fn(self.plan, *args, dw, dshift, flags, ws)
        return dw, dshift

    def grad_from_values(self, G, dw=None, dshift=None, accumulate=False, want_shift=True,
                         shared_shift=False):
        """(dL/dw [B, E], dL/dshift [B]) from G = dL/dvalues by the chain rule;
        with shared_shift, dL/dshift [1] of one shift that serves every system."""
        return self._grads(L.sla_laplacian_grad_values, (self.A._values(G),), dw, dshift, accumulate,
                           want_shift, shared_shift)

    def grad(self, lam, x, dw=None, dshift=None, accumulate=False, want_shift=True, shared_shift=False):
        """The same for G = -lam x^T on the pattern, without forming G."""
        A = self.A
        return self._grads(L.sla_laplacian_grad, (A._vec(lam, A.n_rows), A._vec(x, A.n_rows)),
                           dw, dshift, accumulate, want_shift, shared_shift)

    # ---------------------------------------------------- autograd calls
    def assemble(self, w, shift=None) -> torch.Tensor:
        """values = L_w + shift I, differentiable in w and shift."""
        return _Assemble.apply(self, w, shift)

    def solve(self, w, b, shift=None, *, rtol=1e-10, atol=0.0, max_iter=0, fixed_iters=0,
              precond=True, strategy=L.SLA_STRATEGY_AUTO) -> torch.Tensor:
        """x = (L_w + shift I)^-1 b, differentiable in w, shift and b."""
        opts = dict(rtol=rtol, atol=atol, max_iter=max_iter, fixed_iters=fixed_iters,
                    precond=precond, strategy=strategy)
        return _EdgeSolve.apply(self, w, shift, b, opts)


class _Assemble(torch.autograd.Function):
    @staticmethod
    def forward(ctx, E: EdgeLaplacian, w, shift):
        ctx.E = E
        ctx.shift_shape = None if shift is None or not torch.is_tensor(shift) else shift.shape
        return E.assemble_values(w, shift).reshape(w.shape[:-1] + (E.A.nnz,))

    @staticmethod
    def backward(ctx, gv):
        E = ctx.E
        want_s = ctx.needs_input_grad[2]
        shared = want_s and math.prod(ctx.shift_shape) == 1 and E.A.batch > 1
        dw, ds = E.grad_from_values(gv.contiguous(), want_shift=want_s, shared_shift=shared)
        gw = dw.reshape(gv.shape[:-1] + (E.n_edges,)) if ctx.needs_input_grad[1] else None
        gs = ds.reshape(ctx.shift_shape) if want_s else None
        return None, gw, gs


class _EdgeSolve(torch.autograd.Function):
    @staticmethod
    def forward(ctx, E: EdgeLaplacian, w, shift, b, opts):
        A = E.A
        vals = E.assemble_values(w, shift)
        x, info = A.cg(vals, b, **opts)
        A.last_info = info
        ctx.E, ctx.opts = E, opts
        ctx.shift_shape = None if shift is None or not torch.is_tensor(shift) else shift.shape
        ctx.w_shape = w.shape
        ctx.save_for_backward(vals, x)
        return x.reshape(b.shape)

    @staticmethod
    def backward(ctx, gx):
        E, opts = ctx.E, ctx.opts
        A = E.A
        vals, x = ctx.saved_tensors
        lam, info = A.cg(vals, gx.contiguous(), adjoint=True, **opts)
        A.last_adjoint_info = info
        want_s = ctx.needs_input_grad[2]
        gw = gs = None
        if ctx.needs_input_grad[1] or want_s:
            shared = want_s and math.prod(ctx.shift_shape) == 1 and A.batch > 1
            dw, ds = E.grad(lam, x, want_shift=want_s, shared_shift=shared)
            gw = dw.reshape(ctx.w_shape) if ctx.needs_input_grad[1] else None
            if want_s:
                gs = ds.reshape(ctx.shift_shape)
        gb = lam.reshape(gx.shape) if ctx.needs_input_grad[3] else None
        return None, gw, gs, gb, None


@dataclass
class NewtonInfo:
    """Outcome of newton_solve (host values; each Newton step reads ||F||)."""
    steps: int
    residual_norms: list        # per step, the per-system ||F(u_k)||_2
    converged: bool
    linear: list                # per step, (iterations, statuses) of its linear solve


def newton_solve(A: CSR, residual, jacobian, u0, *theta, tol=1e-10, max_steps=50, cg_rtol=1e-12,
                 max_iter=0, precond=True, strategy=L.SLA_STRATEGY_AUTO) -> torch.Tensor:
    """u with F(u, theta) = 0 by Newton's method, differentiable in theta.

    Nonlinear systems of "torch-sla" (technical summary, "Methodology" 2): the
    Jacobian J = dF/du must be SPD with A's pattern (each Newton step is one
    Jacobi-PCG solve J delta = F, u <- u - delta); the backward pass is one
    adjoint solve J(u)^T lambda = dL/du and one vector-Jacobian product,
    dL/dtheta = -lambda^T dF/dtheta, whatever the number of Newton steps.

    theta are tensors; residual(u, *theta) -> F shaped like u (differentiable in
    theta, torch);
    jacobian(u, *theta) -> J's values [B, nnz] on A's pattern.  Stops when
    every system has ||F|| <= tol * max(1, ||F(u0)||).  A.last_newton_info
    holds the NewtonInfo of the last forward.
    """
    opts = dict(tol=tol, max_steps=max_steps, cg=dict(rtol=cg_rtol, max_iter=max_iter,
                                                      precond=precond, strategy=strategy))
    return _Newton.apply(A, residual, jacobian, opts, u0, *theta)


class _Newton(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A: CSR, residual, jacobian, opts, u0, *theta):
        u = A._vec(u0, A.n_rows).clone()
        F = A._vec(residual(u, *theta), A.n_rows)
        # host copies only, so that nothing kept grows with the step count
        norms = [torch.linalg.vector_norm(F, dim=1).tolist()]
        bound = [opts["tol"] * max(1.0, v) for v in norms[0]]
        done = lambda nr: all(v <= t for v, t in zip(nr, bound))  # noqa: E731
        linear = []
        steps = 0
        while steps < opts["max_steps"] and not done(norms[-1]):
            Jv = A._values(jacobian(u, *theta))
            delta, info = A.cg(Jv, F, **opts["cg"])
            linear.append((info.iters.tolist(), info.status.tolist()))
            u.sub_(delta)
            del Jv, delta, info
            F = A._vec(residual(u, *theta), A.n_rows)
            norms.append(torch.linalg.vector_norm(F, dim=1).tolist())
            steps += 1
        A.last_newton_info = NewtonInfo(steps, norms, done(norms[-1]), linear)
        ctx.A, ctx.residual, ctx.jacobian, ctx.opts = A, residual, jacobian, opts
        ctx.u_shape = u0.shape
        ctx.save_for_backward(u, *theta)
        return u.reshape(u0.shape)

    @staticmethod
    def backward(ctx, gu):
        A, opts = ctx.A, ctx.opts
        u, *theta = ctx.saved_tensors
        needs = ctx.needs_input_grad[5:]
        if not any(needs):
            return (None,) * (5 + len(theta))
        with torch.no_grad():
            Jv = A._values(ctx.jacobian(u, *theta))
        lam, info = A.cg(Jv, A._vec(gu.contiguous(), A.n_rows), adjoint=True, **opts["cg"])
        A.last_adjoint_info = info
        with torch.enable_grad():
            th = [t.detach().requires_grad_(need) for t, need in zip(theta, needs)]
            F = ctx.residual(u.detach().reshape(ctx.u_shape), *th)
            wrt = [t for t, need in zip(th, needs) if need]
            got = torch.autograd.grad(F, wrt, grad_outputs=-lam.reshape(F.shape), allow_unused=True)
        it = iter(got)
        grads = [next(it) if need else None for need in needs]
        return (None, None, None, None, None, *grads)


# ------------------------------------------------- norms of many tensors ----
def _norm_kind(norm_type) -> int:
    if norm_type == 2:
        return L.SLA_NORM_L2
    if norm_type == math.inf:
        return L.SLA_NORM_MAX
    raise ValueError(f"norm_type must be 2 or inf (got {norm_type})")


def _codes(tensors):
    """The tensors' types as the library's, all on one CUDA device."""
    devices = {t.device for t in tensors}
    if len(devices) > 1 or devices.pop().type != "cuda":
        raise ValueError("the tensors must be on one CUDA device")
    try:
        return [L.TENSOR_DTYPES[t.dtype] for t in tensors]
    except KeyError as e:
        raise TypeError(f"unsupported dtype {e.args[0]} (float64, float32, bfloat16 or float16)") from None


def _dense(t: torch.Tensor) -> bool:
    """The elements fill one range of memory, in whatever order."""
    return t.is_contiguous() or torch.ops.aten.is_non_overlapping_and_dense(t)


def _dense_list(tensors):
    if all(map(torch.Tensor.is_contiguous, tensors)):
        return tensors
    return [t if _dense(t) else t.detach().contiguous() for t in tensors]


def _check_copied(outs):
    """Outputs that the library does not see: refused before anything is written."""
    if any(n > 1 and st == 0 for o in outs for n, st in zip(o.shape, o.stride())):
        raise ValueError("an output has several elements in one place (an expanded tensor)")
    if len({(o.data_ptr(), o.shape, o.stride()) for o in outs if o.numel()}) < sum(1 for o in outs if o.numel()):
        raise ValueError("one output is given twice")


def _norm_buffers(codes, device):
    return (torch.empty((), dtype=torch.float64 if L.SLA_F64 in codes else torch.float32, device=device),
            _workspace(L.sla_norm_workspace_bytes(len(codes)), device))


def global_norm(tensors, norm_type: float = 2.0) -> torch.Tensor:
    """The norm of all elements of all tensors: sqrt(sum x^2), or max |x| for
    norm_type inf.  A 0-dim tensor, float64 if any tensor is, else float32, outside
    autograd; squares are summed in 64 bits in a fixed order.  No host
    synchronisation.
    """
    tensors = list(tensors)
    kind = _norm_kind(norm_type)
    if not tensors:
        return torch.zeros(())
    codes = _codes(tensors)
    src = _dense_list(tensors)
    with _on_device(tensors[0].device):
        norm, ws = _norm_buffers(codes, tensors[0].device)
        L.sla_global_norm(len(src), L.tensor_list(src, codes), kind, norm, ws)
    return norm


def clip_by_global_norm(tensors, max_norm: float, *, norm_type: float = 2.0, out=None):
    """(clipped, norm): every tensor times min(1, max_norm / (norm + 1e-6)), with
    the norm of all of them together, outside autograd.  ``out``: the tensors to
    write (shapes and types of the inputs; ``out=tensors`` clips in place), new ones
    by default.  The outputs may share memory with their own input only.  A NaN
    makes every output NaN; an infinity makes the factor 0.  No host
    synchronisation.
    """
    tensors = list(tensors)
    kind = _norm_kind(norm_type)
    max_norm = float(max_norm)
    if not (max_norm >= 0.0 and math.isfinite(max_norm)):
        raise ValueError(f"max_norm must be finite and not negative (got {max_norm})")
    outs = None if out is None else list(out)
    if outs is not None and (len(outs) != len(tensors) or any(
            o is not t and (o.shape != t.shape or o.dtype != t.dtype or o.device != t.device)
            for o, t in zip(outs, tensors))):
        raise ValueError("out must match the tensors in number, shapes, types and device")
    if not tensors:
        return [], torch.zeros(())
    codes = _codes(tensors)
    src = _dense_list(tensors)
    if outs is None:
        outs = dst = list(map(torch.empty_like, src))
    elif src is tensors and all(map(operator.is_, outs, src)):
        dst = src
    else:
        # an output laid out otherwise than its input is written by way of a copy
        dst = [o if o is s or (o.stride() == s.stride() and _dense(o)) else torch.empty_like(s)
               for o, s in zip(outs, src)]
        _check_copied([o for o, d in zip(outs, dst) if o is not d])
    with _on_device(tensors[0].device):
        norm, ws = _norm_buffers(codes, tensors[0].device)
        L.sla_clip_norm(len(src), L.tensor_list(src, codes, dst), kind, max_norm, norm, ws)
    if out is not None:                          # for autograd graphs that saved them
        torch.autograd.graph.increment_version(outs)
    if outs is not dst:
        for o, d in zip(outs, dst):
            if o is not d:
                o.detach().copy_(d)
    return outs, norm


def clip_grad_norm_(parameters, max_norm: float, norm_type: float = 2.0) -> torch.Tensor:
    """Clip the parameters' gradients in place to a global norm; returns the norm
    before clipping.  Parameters without a gradient are skipped.  Two parameters
    that share one gradient tensor are an error.  No host synchronisation."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    return clip_by_global_norm(grads, max_norm, norm_type=norm_type, out=grads)[1]
