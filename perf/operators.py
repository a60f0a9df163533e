"""Workloads of the attention over a CSR pattern and of the gradient norm and clipping.

Two operators, each in a plain form (elementary torch operations) and, with
``own`` set, as calls of the package:

attention  row i of a pattern attends to the columns stored in that row,
           s_t = scale * q_i . k_j + values_t,  p = softmax of s over the row,
           o_i = sum_t p_t v_j;  a row without entries (or whose values are all
           -inf) gives zeros.  Training cases return the gradients of q, k, v
           and the values as well.
norm, clip the global norm of many gradients, and the gradients scaled so that
           it does not exceed a bound: g * min(1, max_norm / (norm + 1e-6)).
"""
import math

import torch

own = False

DTYPES = {"f64": torch.float64, "f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f64": 8, "f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases ----
def _attn(name, kind, dtype, heads, kv_heads, dim, *, a, b=1, c=1, batch=1, values=False, train=False):
    """kind "grid": the 5- or 7-point pattern of an a x b (x c) grid; "graph": a rows over b
    columns, irregular rows of about c entries near the diagonal; "full": a rows over b columns,
    every entry stored (with values: each system has its own number of columns, the rest at -inf)."""
    case = {"op": "attention", "kind": kind, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "a": a, "b": b, "c": c, "batch": batch, "values": values, "train": train}
    return dict(case, name=name) if name else case


def _clip(name, op, layout, dtype, count, total):
    """layout "even": `count` tensors of about total / count elements; "mixed": sizes spread over
    their logarithm, every third tensor in 32 bits."""
    case = {"op": op, "layout": layout, "dtype": dtype, "count": count, "total": total}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one row reads many columns: a single query against an encoder's states (latency)
        _attn("one_row_f16", "full", "f16", 8, 2, 64, a=1, b=4096),
        # the 64 x 64 Poisson pattern with learned edge values
        _attn("grid64_f32", "grid", "f32", 4, 4, 32, a=64, b=64, values=True),
        # the 1024 x 1024 Poisson pattern: a network layer over a million unknowns
        _attn("grid1024_bf16", "grid", "bf16", 4, 4, 32, a=1024, b=1024),
        # training over an irregular graph in a bandwidth-reducing order
        _attn("graph_bf16_train", "graph", "bf16", 8, 8, 64, a=100003, b=100003, c=12, values=True, train=True),
        # a batch of 32 x 32 systems that share one pattern, in training
        _attn("batch32_f32_train", "grid", "f32", 4, 4, 32, a=32, b=32, batch=128, values=True, train=True),
        # queries against padded encoder states of other lengths
        _attn("cross_bf16", "full", "bf16", 8, 8, 64, a=300, b=1500, batch=8, values=True),
        # a 3-D diffusion pattern in 64 bits, in training
        _attn("grid3d_f64_train", "grid", "f64", 2, 2, 16, a=32, b=32, c=32, values=True, train=True),
        # few pooled rows over many points, shared key heads, long rows, in training
        _attn("pool_f16_train", "graph", "f16", 8, 2, 128, a=513, b=65536, c=256, train=True),
        # gradients of the 264 conductivities of a 12 x 12 grid and of a shift (latency)
        _clip("clip_edges_f64", "clip", "even", "f64", 2, 265),
        # gradients of a small network: many tensors, odd sizes, two types
        _clip("clip_mixed_bf16", "clip", "mixed", "bf16", 62, 12_000_000),
        # gradients far larger than the caches
        _clip("clip_large_f32", "clip", "even", "f32", 24, 200_000_000),
        # the norm alone, for the edge gradients of a batch of 1024 systems
        _clip("norm_batch_f64", "norm", "even", "f64", 2, 1024 * 1985),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.3:
        dtype = rng.choice(["f64", "f32", "bf16", "f16"])
        return _clip(None, rng.choice(["clip", "clip", "norm"]), rng.choice(["even", "mixed"]), dtype,
                     _log(rng, 1, 62), _log(rng, 1000, 60_000_000))
    dtype = rng.choice(["f64", "f32", "bf16", "f16", "bf16", "f16"])
    kind = rng.choice(["grid", "grid", "graph", "graph", "full"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    dim = rng.choice([16, 20, 32, 32, 48, 64, 64, 80, 128])
    values, train = rng.random() < 0.6, rng.random() < 0.5
    width = heads * dim * (2 if train else 1) * (2 if dtype == "f64" else 1)
    # entries x width: the plain form makes arrays of this many numbers
    entries = max(64, int(_log(rng, 2e5, 2.5e8) / width))
    if kind == "grid":
        batch = rng.choice([1, 1, 2, 7])
        n = max(2, entries // (6 * batch))
        c = rng.choice([1, 1, max(2, round(n ** (1 / 3)))])
        a = max(2, round((n / c) ** 0.5))
        return _attn(None, kind, dtype, heads, kv_heads, dim, a=a, b=max(2, n // (a * c)), c=c, batch=batch,
                     values=values, train=train)
    if kind == "graph":
        c = _log(rng, 4, 300)
        rows = max(1, entries // c)
        cols = max(4 * c, int(rows * rng.choice([1, 1, 0.37, 11])))
        return _attn(None, kind, dtype, heads, kv_heads, dim, a=rows, b=cols, c=c, values=values, train=train)
    batch = rng.choice([1, 1, 3, 6])
    rows = min(_log(rng, 1, 400), max(1, entries // (64 * batch)))
    return _attn(None, kind, dtype, heads, kv_heads, dim, a=rows, b=max(8, entries // (rows * batch)), batch=batch,
                 values=values, train=train)


# --------------------------------------------------------------- patterns ----
def _degrees(rows, mean):
    """Entries of each row of a "graph" pattern: about `mean`, irregular, some rows empty."""
    i = torch.arange(rows)
    deg = mean - mean // 3 + (i * 7919) % (2 * (mean // 3) + 1)
    return torch.where(i % 97 == 96, torch.zeros_like(deg), deg)


def _sizes(case):
    """(rows, columns, entries) of a case's pattern."""
    a, b, c = case["a"], case["b"], case["c"]
    if case["kind"] == "grid":
        n = a * b * c
        return n, n, n + 2 * ((a - 1) * b * c + a * (b - 1) * c + a * b * (c - 1))
    if case["kind"] == "full":
        return a, b, a * b
    return a, b, int(_degrees(a, c).sum())


def _pattern(case, gen, dev):
    """rowptr, colind (int32) of a case's pattern, columns increasing within a row."""
    rows, cols, nnz = _sizes(case)
    if case["kind"] == "full":
        rowptr = torch.arange(rows + 1, device=dev) * cols
        return rowptr.int(), torch.arange(cols, device=dev).int().repeat(rows)
    if case["kind"] == "graph":
        deg = _degrees(rows, case["c"]).to(dev)
        rowptr = torch.zeros(rows + 1, dtype=torch.int64, device=dev)
        rowptr[1:] = deg.cumsum(0)
        row = torch.repeat_interleave(torch.arange(rows, device=dev), deg)
        # increasing columns from gaps of 1 to 4, around the row's place on the columns' axis
        gap = torch.randint(1, 5, (nnz,), generator=gen, device=dev)
        run = gap.cumsum(0)
        first = rowptr[:-1].clamp(max=max(nnz - 1, 0))
        off = run - run[first][row]                                  # 0 at a row's first entry
        last = (rowptr[1:] - 1).clamp(min=0)
        span = torch.where(deg > 0, (run[last] - run[first]), torch.zeros_like(deg))
        start = torch.arange(rows, device=dev) * cols // rows - span // 2
        start = torch.minimum(start, cols - 1 - span).clamp(min=0)
        return rowptr.int(), (start[row] + off).clamp(max=cols - 1).int()
    a, b, c = case["a"], case["b"], case["c"]
    i = torch.arange(rows, device=dev)
    x, y, z = i // (b * c), i // c % b, i % c
    far = [(x > 0, -b * c), (y > 0, -c), (z > 0, -1), (z >= 0, 0), (z < c - 1, 1), (y < b - 1, c), (x < a - 1, b * c)]
    keep = torch.stack([m for m, _ in far], 1)
    col = torch.stack([i + d for _, d in far], 1)
    rowptr = torch.zeros(rows + 1, dtype=torch.int64, device=dev)
    rowptr[1:] = keep.sum(1).cumsum(0)
    return rowptr.int(), col[keep].int()


def _tensor_sizes(case):
    count, total = case["count"], case["total"]
    if case["layout"] == "even":
        small = max(1, total // (8 * count + 1)) | 1                 # one small, odd tensor
        each = max(1, (total - small) // max(1, count - 1))
        return [each] * (count - 1) + [small if count > 1 else total]
    weight = [math.exp(8.0 * ((k * 37) % count) / count) for k in range(count)]
    return [max(1, int(total * w / sum(weight))) for w in weight]


def _tensor_dtypes(case):
    mixed = case["layout"] == "mixed" and case["dtype"] in ("bf16", "f16")
    return ["f32" if mixed and k % 3 == 2 else case["dtype"] for k in range(len(_tensor_sizes(case)))]


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] != "attention":
        tensors = [torch.randn(n, generator=gen, device=dev, dtype=torch.float64 if d == "f64" else torch.float32)
                   .mul_(1e-3).to(DTYPES[d]) for n, d in zip(_tensor_sizes(case), _tensor_dtypes(case))]
        # half of what the norm is expected to be: the gradients are scaled
        return {"case": case, "tensors": tensors, "max_norm": 0.5e-3 * math.sqrt(sum(t.numel() for t in tensors))}
    rowptr, colind = _pattern(case, gen, dev)
    rows, cols, nnz = _sizes(case)
    dt, batch = DTYPES[case["dtype"]], case["batch"]
    vt = torch.float64 if dt == torch.float64 else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=vt).to(dt)

    state = {"case": case, "rowptr": rowptr, "colind": colind,
             "q": normal(batch, rows, case["heads"], case["dim"]),
             "k": normal(batch, cols, case["kv_heads"], case["dim"]),
             "v": normal(batch, cols, case["kv_heads"], case["dim"]),
             "do": normal(batch, rows, case["heads"], case["dim"]) if case["train"] else None, "values": None}
    if case["values"]:
        if case["kind"] == "full":
            length = torch.randint(max(1, cols // 3), cols + 1, (batch, 1), generator=gen, device=dev)
            out = torch.arange(cols, device=dev)[None] >= length
            row = torch.zeros(batch, cols, dtype=vt, device=dev).masked_fill(out, -math.inf)
            state["values"] = row[:, None, :].expand(batch, rows, cols).reshape(batch, nnz).contiguous()
        else:
            state["values"] = torch.randn(batch, nnz, generator=gen, device=dev, dtype=vt) * 0.5
    return state


def prepare(case, seed):
    state = _inputs(case, seed)
    if own and case["op"] == "attention":
        import differentiable_sparse_linear_csr_b200 as sla
        # the pattern's handle, which a program makes once and keeps
        state["A"] = sla.CSR(state["rowptr"], state["colind"], n_cols=_sizes(case)[1], batch=case["batch"],
                             dtype=torch.float64 if case["dtype"] == "f64" else torch.float32)
        state["A"].prepare_attention(backward=case["train"], heads_per_key=case["heads"] // case["kv_heads"])
        if case["train"]:
            state["wrt"] = [state[x].requires_grad_() for x in ("q", "k", "v", "values") if state[x] is not None]
    return state


# -------------------------------------------------------------- plain form ----
def _plain_full(case, q, k, v, values, do, scale):
    """Every column stored: the scores are a matrix product."""
    B, n, H, D = q.shape
    m, G = k.shape[1], H // k.shape[2]
    qh = q.permute(0, 2, 1, 3)
    kh, vh = (t.permute(0, 2, 1, 3).repeat_interleave(G, 1) for t in (k, v))
    s = qh @ kh.transpose(2, 3) * scale
    if values is not None:
        s = s + values.reshape(B, 1, n, m)
    top = s.amax(3, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = e / e.sum(3, keepdim=True).clamp(min=1e-300 if e.dtype == torch.float64 else 1e-38)
    o = p @ vh
    if do is None:
        return [o.permute(0, 2, 1, 3)]
    doh = do.permute(0, 2, 1, 3)
    ds = p * (doh @ vh.transpose(2, 3) - (doh * o).sum(3, keepdim=True))
    dk = (ds.transpose(2, 3) @ qh * scale).reshape(B, H // G, G, m, D).sum(2)
    dv = (p.transpose(2, 3) @ doh).reshape(B, H // G, G, m, D).sum(2)
    out = [o.permute(0, 2, 1, 3), (ds @ kh * scale).permute(0, 2, 1, 3), dk.permute(0, 2, 1, 3), dv.permute(0, 2, 1, 3)]
    return out + ([ds.sum(1).reshape(B, n * m)] if values is not None else [])


def _plain_sparse(rowptr, colind, q, k, v, values, do, scale):
    """Gathers of both sides of every entry, sums over each row's entries."""
    B, n, H, D = q.shape
    m, K = k.shape[1], k.shape[2]
    G, nnz = H // K, colind.numel()
    col = colind.long()
    row = torch.repeat_interleave(torch.arange(n, device=col.device), (rowptr[1:] - rowptr[:-1]).long(), output_size=nnz)
    qg = q.reshape(B, n, K, G, D)[:, row]                              # [B, nnz, K, G, D]
    kg = k[:, col].unsqueeze(3)
    s = (qg * kg).sum(4) * scale                                       # [B, nnz, K, G]
    if values is not None:
        s = s + values.reshape(B, nnz, 1, 1)
    at = row.reshape(1, nnz, 1, 1).expand_as(s)
    top = torch.full((B, n, K, G), -math.inf, dtype=s.dtype, device=s.device).scatter_reduce(1, at, s, "amax")
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(s - top[:, row])
    total = torch.zeros_like(top).index_add(1, row, e).clamp(min=1e-300 if e.dtype == torch.float64 else 1e-38)
    p = e / total[:, row]
    vg = v[:, col].unsqueeze(3)
    o = torch.zeros(B, n, K, G, D, dtype=s.dtype, device=s.device).index_add(1, row, p.unsqueeze(4) * vg)
    if do is None:
        return [o.reshape(B, n, H, D)]
    dor = do.reshape(B, n, K, G, D)
    dog = dor[:, row]
    ds = p * ((dog * vg).sum(4) - (dor * o).sum(4)[:, row])
    dq = torch.zeros_like(o).index_add(1, row, ds.unsqueeze(4) * kg * scale)
    dk = torch.zeros_like(k).index_add(1, col, (ds.unsqueeze(4) * qg).sum(3) * scale)
    dv = torch.zeros_like(v).index_add(1, col, (p.unsqueeze(4) * dog).sum(3))
    out = [o.reshape(B, n, H, D), dq.reshape(B, n, H, D), dk, dv]
    return out + ([ds.sum((2, 3))] if values is not None else [])


def run(state):
    case = state["case"]
    if case["op"] == "attention":
        if own:
            o = state["A"].attention(state["q"], state["k"], state["v"], state["values"])
            if not case["train"]:
                return [o]
            return [o.detach(), *torch.autograd.grad(o, state["wrt"], state["do"])]
        dt = state["q"].dtype
        wide = torch.float64 if dt == torch.float64 else torch.float32
        q, k, v, do = (None if state[x] is None else state[x].to(wide) for x in ("q", "k", "v", "do"))
        scale, values = case["dim"] ** -0.5, state["values"]
        out = (_plain_full(case, q, k, v, values, do, scale) if case["kind"] == "full" else
               _plain_sparse(state["rowptr"], state["colind"], q, k, v, values, do, scale))
        # all but the values' gradient have the inputs' type
        return [t.to(dt) if j < 4 else t for j, t in enumerate(out)]
    tensors, limit = state["tensors"], state["max_norm"]
    if own:
        import differentiable_sparse_linear_csr_b200 as sla
        if case["op"] == "norm":
            return [sla.global_norm(tensors)]
        clipped, norm = sla.clip_by_global_norm(tensors, limit)
        return [norm, *clipped]
    wide = torch.float64 if any(t.dtype == torch.float64 for t in tensors) else torch.float32
    norm = torch.stack([t.double().square().sum() for t in tensors]).sum().sqrt()
    if case["op"] == "norm":
        return [norm.to(wide)]
    scale = (limit / (norm + 1e-6)).clamp(max=1.0).to(wide)
    return [norm.to(wide), *((t.to(wide) * scale).to(t.dtype) for t in tensors)]


# ------------------------------------------------------------ in 64 bits ----
def _exact_attention(case, state):
    """Rows padded to the longest one, softmax and its gradient by autograd, some rows at a time."""
    rows, cols, nnz = _sizes(case)
    H, K, D, B = case["heads"], case["kv_heads"], case["dim"], case["batch"]
    ptr = state["rowptr"].long()
    length = ptr[1:] - ptr[:-1]
    widest = max(1, int(length.max()))
    q, k, v = (state[x].double() for x in ("q", "k", "v"))
    k.requires_grad_(case["train"])
    v.requires_grad_(case["train"])
    vals = None if state["values"] is None else state["values"].double().requires_grad_(case["train"])
    step = max(1, min(rows, int(3e8 / (B * H * D * widest))))
    outs, dqs = [], []
    for r in range(0, rows, step):
        n = min(step, rows - r)
        slot = ptr[r:r + n, None] + torch.arange(widest, device=ptr.device)
        there = torch.arange(widest, device=ptr.device) < length[r:r + n, None]
        slot = torch.where(there, slot, torch.zeros_like(slot)).clamp(max=max(nnz - 1, 0))
        col = state["colind"].long()[slot]
        qr = q[:, r:r + n].detach().requires_grad_(case["train"])
        score = torch.einsum("bnkgd,bnwkd->bnkgw", qr.reshape(B, n, K, H // K, D), k[:, col]) / math.sqrt(D)
        if vals is not None:
            score = score + vals[:, slot][:, :, None, None, :]
        alive = there[None, :, None, None, :].expand_as(score)
        if vals is not None:
            alive = alive & (vals.detach()[:, slot] > -math.inf)[:, :, None, None, :]
        some = alive.any(4, keepdim=True)
        score = torch.where(alive, score, torch.full_like(score, -math.inf))
        prob = torch.where(some, torch.softmax(torch.where(some, score, torch.zeros_like(score)), 4), torch.zeros_like(score))
        o = torch.einsum("bnkgw,bnwkd->bnkgd", prob, v[:, col]).reshape(B, n, H, D)
        outs.append(o.detach())
        if case["train"]:
            o.backward(state["do"][:, r:r + n].double())
            dqs.append(qr.grad)
    if not case["train"]:
        return [torch.cat(outs, 1)]
    got = [torch.cat(outs, 1), torch.cat(dqs, 1), k.grad, v.grad]
    return got + ([vals.grad] if vals is not None else [])


def exact(case, seed):
    state = _inputs(case, seed)
    if case["op"] == "attention":
        with torch.enable_grad():
            return _exact_attention(case, state)
    every = [t.double() for t in state["tensors"]]
    norm = math.sqrt(math.fsum(float((t * t).sum()) for t in every))
    value = torch.tensor(norm, dtype=torch.float64, device="cuda")
    if case["op"] == "norm":
        return [value]
    factor = min(1.0, state["max_norm"] / (norm + 1e-6))
    return [value, *(t * factor for t in every)]


# -------------------------------------------------------------------- work ----
def work(case):
    if case["op"] != "attention":
        sizes = list(zip(_tensor_sizes(case), _tensor_dtypes(case)))
        read = sum(n * SIZE[d] for n, d in sizes)
        count = sum(n for n, _ in sizes)
        return {"bytes": read + 8, "flops": 2 * count} if case["op"] == "norm" else {"bytes": 2 * read + 8, "flops": 3 * count}
    rows, cols, nnz = _sizes(case)
    B, H, K, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    size = SIZE[case["dtype"]]
    query, key = B * rows * H * D * size, B * cols * K * D * size
    value = B * nnz * (8 if case["dtype"] == "f64" else 4) if case["values"] else 0
    pattern = 4 * (rows + 1 + nnz)
    # forward: q, k, v in, o out, two products an entry; backward: do in, three gradients out, four more products
    if case["train"]:
        return {"bytes": 4 * query + 4 * key + 2 * value + pattern, "flops": 12 * B * nnz * H * D}
    return {"bytes": 2 * query + 2 * key + value + pattern, "flops": 4 * B * nnz * H * D}
