"""The operators of a trained and served ball-attention layer, as cases that can be timed and compared.

  attention_backward  gradients of ball attention with respect to Q, K and V
  rms_norm            root-mean-square norm of the features, with the residual's addition
  rms_norm_i8         the same with an output in 8 bits and a scale for each row; without the norm, the
                      quantisation alone (features, or weights by output channel)
  rms_norm_backward   gradients of the norm with respect to its input and its weight
  project_i8          the Q/K/V projection in 8-bit integers with scales for each row and output channel,
                      written in tree (slot) order or in the original order

`own` chooses between the plain form (elementary torch operations in float) and the library's calls.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attn(name, rows, clouds, m, H, d, dt):
    c = {"op": "attention_backward", "rows": rows, "clouds": clouds, "m": m, "H": H, "d": d, "dt": dt}
    return {"name": name, **c} if name else c


def _norm(name, op, rows, C, dt, residual, weight, norm=True):
    c = {"op": op, "rows": rows, "C": C, "dt": dt, "residual": residual, "weight": weight, "norm": norm}
    return {"name": name, **c} if name else c


def _proj(name, rows, clouds, m, C, H, d, dt, tree):
    c = {"op": "project_i8", "rows": rows, "clouds": clouds, "m": m, "C": C, "H": H, "d": d, "dt": dt, "tree": tree}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one small cloud in float (the `tiny` workload): a training step's latency
        _attn("attn_bwd_tiny_f32", 1024, 1, 32, 2, 32, "f32"),
        # the batch of four clouds that the benchmark runs forward
        _attn("attn_bwd_gauss_mix", 65536, 4, 128, 8, 32, "bf16"),
        # one cloud of a million points, four heads: the largest layer
        _attn("attn_bwd_box_cluster", 1048576, 1, 128, 4, 32, "bf16"),
        # uneven clouds padded with dummies, wide heads, an odd number of them, small balls
        _attn("attn_bwd_ragged_d64", 70001, 3, 64, 5, 64, "bf16"),
        # pre-norm of a layer with the residual stream, at the batch's size
        _norm("norm_gauss_mix", "rms_norm", 65536, 256, "bf16", True, True),
        # a handful of rows of an odd width in float
        _norm("norm_few_f32", "rms_norm", 37, 1000, "f32", True, True),
        # pre-norm that feeds the 8-bit projection, a million points
        _norm("norm_i8_box_cluster", "rms_norm_i8", 1048576, 128, "bf16", True, True),
        # a projection's weights (3 H d output channels) quantised by channel
        _norm("quantize_weights", "rms_norm_i8", 768, 256, "f32", False, False, False),
        # the norm's backward pass, the residual stream's gradient added
        _norm("norm_bwd_gauss_mix", "rms_norm_backward", 65536, 256, "bf16", True, True),
        # an odd number of wide rows in float
        _norm("norm_bwd_odd_f32", "rms_norm_backward", 1023, 768, "f32", False, True),
        # projection of the batch's features into tree order
        _proj("project_i8_gauss_mix", 65536, 4, 128, 256, 8, 32, "bf16", True),
        # a few query points against stored weights: serving one small request
        _proj("project_i8_few", 7, 1, 16, 512, 8, 64, "bf16", False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attention_backward", "rms_norm", "rms_norm_i8", "rms_norm_backward", "project_i8"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op == "attention_backward":
        d, H = rng.choice([32, 64]), rng.choice([1, 2, 3, 4, 6, 8, 12])
        m = rng.choice([16, 32, 64, 128, 128, 256, rng.randint(1, 256)])
        # padding at most doubles the slots; float runs on the CUDA cores, so it gets fewer rows
        most = (1 << (33 if dt == "bf16" else 30)) // (max(m, 16) * H * d)
        rows = _log_int(rng, 1, max(1, min(most, 700000)))
        return _attn(None, rows, rng.randint(1, min(8, rows)), m, H, d, dt)
    if op == "project_i8":
        H, d = rng.choice([(2, 32), (4, 32), (8, 32), (3, 64), (8, 64), (5, 24)])
        C = rng.choice([64, 128, 256, 512, 16 * rng.randint(1, 64), rng.randint(1, 300)])
        rows = _log_int(rng, 1, max(1, min(400000, (1 << 36) // (C * 3 * H * d))))
        return _proj(None, rows, rng.randint(1, min(8, rows)), rng.choice([16, 32, 64, 128]), C, H, d, dt,
                     rng.random() < 0.6)
    C = rng.choice([32, 64, 128, 256, 512, 1024, rng.randint(1, 2000), _log_int(rng, 1, 8192)])
    rows = _log_int(rng, 1, max(1, min(1000000, (1 << 27) // C)))
    norm = op != "rms_norm_i8" or rng.random() < 0.7
    return _norm(None, op, rows, C, dt, norm and rng.random() < 0.7, norm and rng.random() < 0.8, norm)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _cloud_sizes(rows, clouds):
    return [rows // clouds + (b < rows % clouds) for b in range(clouds)]


def _padded(n, m):
    return m << max(0, (-(-n // m) - 1).bit_length())


def _tree_perm(case, g):
    """Slot -> row of a tree over the clouds: every cloud's rows in random order over its first slots (a
    leaf's rows ascending, as a build leaves them), dummies (-1) in its last ones."""
    m, parts, r0 = case["m"], [], 0
    for n in _cloud_sizes(case["rows"], case["clouds"]):
        s = torch.full((_padded(n, m),), 1 << 30, dtype=torch.int32, device="cuda")
        s[:n] = (torch.randperm(n, generator=g, device="cuda") + r0).to(torch.int32)
        s = s.view(-1, m).sort(dim=1).values.flatten()
        parts.append(torch.where(s == 1 << 30, -1, s))
        r0 += n
    return torch.cat(parts).to(torch.int32).contiguous()


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": dict(case)}
    op, dt = case["op"], DTYPES[case["dt"]]
    rows = case["rows"]
    if op == "attention_backward":
        shape = (rows, case["H"], case["d"])
        for n in ("Q", "K", "V", "dO"):
            st[n] = _randn(g, *shape).to(dt)
        st["perm"] = _tree_perm(case, g)
        return st
    C = case["C"]
    if op == "project_i8":
        nout = 3 * case["H"] * case["d"]
        # normalised features and a linear layer's weights, quantised by row: the largest value is 127
        x = _randn(g, rows, C)
        w = _randn(g, nout, C) / math.sqrt(C)
        for n, t in (("X", x), ("W", w)):
            s = t.abs().amax(1) / 127
            st[n + "s"] = s
            st[n + "q"] = torch.round(t / s[:, None]).to(torch.int8)
        st["perm"] = st["inv"] = None
        if case["tree"]:
            st["perm"] = _tree_perm(case, g)
            st["inv"] = torch.empty(rows, dtype=torch.int32, device="cuda")
            slots = torch.nonzero(st["perm"] >= 0).flatten()
            st["inv"][st["perm"][slots].long()] = slots.to(torch.int32)
        return st
    # a residual stream has rows of very different size
    scale = torch.exp(_randn(g, rows, 1))
    st["X"] = (_randn(g, rows, C) * scale).to(dt)
    st["R"] = (_randn(g, rows, C) * scale).to(dt) if case["residual"] and op != "rms_norm_backward" else None
    st["w"] = 1 + 0.2 * _randn(g, C) if case["weight"] else None
    if op == "rms_norm_backward":
        st["dY"] = _randn(g, rows, C).to(dt)
        st["dH"] = _randn(g, rows, C).to(dt) if case["residual"] else None
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_attention_backward(st):
    c, perm = st["case"], st["perm"]
    m, H, d = c["m"], c["H"], c["d"]
    real = perm >= 0
    src = perm.clamp(min=0).long()
    keep = real.view(-1, 1, m)  # [balls, 1, m]
    # [balls, H, m, d] in float, dummies as zeros
    q, k, v, do = ((st[n][src].float() * real[:, None, None]).view(-1, m, H, d).transpose(1, 2)
                   for n in ("Q", "K", "V", "dO"))
    scale = 1 / math.sqrt(d)
    s = (q @ k.transpose(2, 3)) * scale
    s = s.masked_fill(~keep[:, :, None, :], -3.0e38)
    p = torch.exp(s - s.amax(3, keepdim=True)) * keep[:, :, None, :]
    p = p / p.sum(3, keepdim=True).clamp(min=1e-30)  # a ball of dummies has no weights
    dv = p.transpose(2, 3) @ do
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (p * dp).sum(3, keepdim=True)) * scale
    dq, dk = ds @ k, ds.transpose(2, 3) @ q
    out = []
    for t in (dq, dk, dv):
        o = torch.zeros_like(st["Q"])
        o[src[real]] = t.transpose(1, 2).reshape(-1, H, d)[real].to(o.dtype)
        out.append(o)
    return out


def _plain_norm(st):
    c = st["case"]
    # the residual stream is kept in the features' type, and the norm is that of the stored stream
    h = st["X"] if st["R"] is None else (st["X"].float() + st["R"].float()).to(st["X"].dtype)
    y = h.float()
    if c["norm"]:
        y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        y = y if st["w"] is None else y * st["w"]
    out = {} if st["R"] is None else {"h": h}
    if c["op"] == "rms_norm":
        return {"y": y.to(h.dtype), **out}
    s = y.abs().amax(1) / 127
    q = torch.round(y / torch.where(s > 0, s, 1)[:, None]).clamp(-127, 127)
    return {"y": _stands_for(q, s), "scale": s, **out}


def _stands_for(q, s):
    """8-bit values times their rows' scales, in one pass; bf16 holds 8 bits."""
    return torch.mul(q, s[:, None], out=torch.empty(q.shape, dtype=torch.bfloat16, device=q.device))


def _plain_norm_backward(st):
    x, dy = st["X"].float(), st["dY"].float()
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    g = dy if st["w"] is None else dy * st["w"]
    dx = r * (g - x * (r * r * (g * x).mean(1, keepdim=True)))
    if st["dH"] is not None:
        dx = dx + st["dH"].float()
    out = {"dx": dx.to(st["X"].dtype)}
    if st["w"] is not None:
        out["dw"] = (dy * x * r).double().sum(0).float()  # up to a million rows
    return out


def _plain_project(st):
    c, hd = st["case"], st["case"]["H"] * st["case"]["d"]
    # products of 8-bit values: a float sum is exact while C * 127^2 < 2^24, in 64 bits always
    t = torch.float32 if c["C"] <= 1040 else torch.float64
    y = (st["Xq"].to(t) @ st["Wq"].to(t).T).float() * st["Xs"][:, None] * st["Ws"][None, :]
    y = y.to(DTYPES[c["dt"]])
    if c["tree"]:
        o = torch.zeros(st["perm"].numel(), 3 * hd, dtype=y.dtype, device=y.device)
        o[st["inv"].long()] = y
        y = o
    return [y[:, i * hd:(i + 1) * hd].reshape(-1, c["H"], c["d"]) for i in range(3)]


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import ball_tree_sparse_b200 as bts
        if op == "attention_backward":
            return list(bts.bt_ball_attention_backward(state["Q"], state["K"], state["V"], state["dO"], state["perm"],
                                                       c["m"]))
        if op == "project_i8":
            return list(bts.bt_qkv_project_i8(state["Xq"], state["Xs"], state["Wq"], state["Ws"], c["H"], c["d"],
                                              dtype=DTYPES[c["dt"]], perm=state["perm"], inv=state["inv"]))
        if op == "rms_norm":
            y, h = bts.bt_rms_norm(state["X"], state["w"], residual=state["R"], eps=EPS)
            return {"y": y} if state["R"] is None else {"y": y, "h": h}
        if op == "rms_norm_i8":
            if not c["norm"]:
                q, s = bts.bt_quantize_i8(state["X"])
                return {"y": _stands_for(q, s), "scale": s}
            q, s, h = bts.bt_rms_norm_i8(state["X"], state["w"], residual=state["R"], eps=EPS)
            return {"y": _stands_for(q, s), "scale": s, **({} if state["R"] is None else {"h": h})}
        dx, dw = bts.bt_rms_norm_backward(state["dY"], state["X"], state["w"], dH=state["dH"], eps=EPS)
        return {"dx": dx} if dw is None else {"dx": dx, "dw": dw}
    if op == "attention_backward":
        return _plain_attention_backward(state)
    if op == "project_i8":
        return _plain_project(state)
    if op == "rms_norm_backward":
        return _plain_norm_backward(state)
    return _plain_norm(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, rows = case["op"], case["rows"]
    es = 4 if case["dt"] == "f32" else 2
    if op == "attention_backward":
        H, d, m = case["H"], case["d"], case["m"]
        sizes = _cloud_sizes(rows, case["clouds"])
        pairs = sum((n // m) * m * m + (n % m) ** 2 for n in sizes)
        return {"bytes": 7 * rows * H * d * es + 4 * sum(_padded(n, m) for n in sizes),
                "flops": 10 * pairs * H * d}  # S, dP, dV, dQ, dK: five products of 2 d per pair
    if op == "project_i8":
        nout, C = 3 * case["H"] * case["d"], case["C"]
        out, slots = rows, 0
        if case["tree"]:
            out = slots = sum(_padded(n, case["m"]) for n in _cloud_sizes(rows, case["clouds"]))
        return {"bytes": rows * (C + 4) + nout * (C + 4) + out * nout * es + (4 * slots + 4 * rows if slots else 0),
                "flops": 2 * rows * C * nout}
    n, C = rows * case["C"], case["C"]  # what the 8-bit output stands for is written by torch: not counted
    if op == "rms_norm_backward":
        return {"bytes": n * es * (3 + case["residual"]) + (8 * C if case["weight"] else 0), "flops": 10 * n}
    w = 4 * C if case["weight"] else 0
    moved = n * es * (3 if case["residual"] else 1)  # x, the residual, the new stream
    if op == "rms_norm":
        return {"bytes": moved + n * es + w, "flops": 5 * n}
    return {"bytes": moved + n + 4 * rows + w, "flops": 8 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_attention_backward(st):
    # the gradient of sum(O * dO) by differentiation of softmax(q k / sqrt(d)) v, a run of balls at a time
    c, perm = st["case"], st["perm"]
    m, H, d = c["m"], c["H"], c["d"]
    outs = [torch.zeros_like(st["Q"], dtype=torch.float64) for _ in range(3)]
    balls = perm.view(-1, m)
    some = (balls >= 0).any(1)
    balls = balls[some]
    step = max(1, (1 << 25) // (m * m * H))
    for b in range(0, balls.shape[0], step):
        idx = balls[b:b + step].long()
        real = idx >= 0
        x = [st[n][idx.clamp(min=0)].double().permute(0, 2, 1, 3) for n in ("Q", "K", "V", "dO")]
        x = [torch.where(real[:, None, :, None], t, 0.0) for t in x]
        q, k, v = (t.clone().requires_grad_(True) for t in x[:3])
        s = torch.einsum("bhqd,bhkd->bhqk", q, k) * d ** -0.5
        s = torch.where(real[:, None, None, :], s, -torch.inf)
        o = torch.einsum("bhqk,bhkd->bhqd", torch.softmax(s, dim=3), v)
        grads = torch.autograd.grad((o * x[3]).sum(), (q, k, v))
        for t, gr in zip(outs, grads):
            t[idx[real]] = gr.permute(0, 2, 1, 3)[real]
    return outs


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "attention_backward":
        return _exact_attention_backward(st)
    if op == "project_i8":
        hd = case["H"] * case["d"]
        a = st["Xq"].double() * st["Xs"].double().unsqueeze(1)
        b = st["Wq"].double() * st["Ws"].double().unsqueeze(1)
        parts = [torch.einsum("rc,nc->rn", a, b[i * hd:(i + 1) * hd]).view(-1, case["H"], case["d"]) for i in range(3)]
        if not case["tree"]:
            return parts
        slots = st["perm"].long()
        zero = torch.zeros(1, case["H"], case["d"], dtype=torch.float64, device="cuda")
        return [torch.cat((p, zero))[slots] for p in parts]  # slot -1: the zero row
    if op == "rms_norm_backward":
        x = st["X"].double().requires_grad_(True)
        w = torch.ones(case["C"], dtype=torch.float64, device="cuda") if st["w"] is None else st["w"].double()
        w.requires_grad_(True)
        y = w * x / torch.sqrt(x.square().sum(1, keepdim=True) / case["C"] + EPS)
        dx, dw = torch.autograd.grad((y * st["dY"].double()).sum(), (x, w))
        if st["dH"] is not None:
            dx = dx + st["dH"].double()
        return {"dx": dx, "dw": dw} if st["w"] is not None else {"dx": dx}
    h = st["X"].double()
    if st["R"] is not None:
        h = (h + st["R"].double()).to(DTYPES[case["dt"]]).double()  # the stream as it is stored
    y = h
    if case["norm"]:
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["C"] + EPS)
        y = y if st["w"] is None else y * st["w"].double()
    out = {} if st["R"] is None else {"h": h}
    if op == "rms_norm":
        return {"y": y, **out}
    s = y.abs().max(1).values / 127
    q = torch.round(y / torch.where(s > 0, s, 1.0).unsqueeze(1))
    return {"y": q * s.unsqueeze(1), "scale": s, **out}
