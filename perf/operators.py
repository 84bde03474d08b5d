"""Timed cases of the operators around the SwiGLU MLP step: layer norm
(forward and backward), the global gradient norm with clipping, and the
mixture-of-experts layer for a few tokens.

``run`` computes a case either in its plain form (elementary torch operations
in 32 bits, in 64 where a sum is long or a choice depends on it) or, with
``own`` set, through this package's entry points.  ``exact`` is the
definition in 64 bits, written apart from both.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token of a served block: the smallest call, latency only
        _norm("norm_fwd_token", "norm_fwd", 1, 4096, "bf16", "bf16", True),
        # the norm in front of the target-shape MLP step
        _norm("norm_fwd_target", "norm_fwd", 11136, 3584, "bf16", "fp32", True),
        # an odd width in fp32 (a small model's ragged batch): rows that are not 16-byte aligned
        _norm("norm_fwd_odd", "norm_fwd", 1999, 1001, "fp32", "fp32", True),
        # backward of the norm in front of the target-shape step, the residual branch's gradient joining
        _norm("norm_bwd_target", "norm_bwd", 11136, 3584, "bf16", "fp32", True, res=True),
        # a small block's backward (the small workload's width), fp16 training
        _norm("norm_bwd_small", "norm_bwd", 2048, 1024, "fp16", "fp32", True, res=True),
        # few rows of a wide, odd norm without bias, fp32
        _norm("norm_bwd_odd", "norm_bwd", 333, 8191, "fp32", "fp32", False),
        # the gradients of the tiny block: four tensors, latency only
        _clip("clip_tiny_block", "block", 1, 256, 512, "bf16", True),
        # the gradients of a stack of four target-shape blocks, clipped into another buffer
        _clip("clip_stack", "block", 4, 3584, 14336, "bf16", True),
        # 301 ragged tensors (adapters, biases, embeddings' rows) in one flat buffer, fp32, none clipped: in place
        _clip("norm_ragged", "ragged", 301, 1, 400_000, "fp32", False),
        # one token of a served expert layer (the MoE workload's layer)
        _moe("moe_token", 1, 3584, 2048, 16, 2, True),
        # a batch of decoded tokens of the same layer: every expert is hit
        _moe("moe_batch", 32, 3584, 2048, 16, 2, True),
        # an odd number of tokens over many small experts
        _moe("moe_many", 7, 2048, 1024, 60, 6, False),
    ]


def _norm(name, op, M, D, dtype, wdtype, bias, res=False):
    return {"name": name, "op": op, "M": M, "D": D, "dtype": dtype, "wdtype": wdtype, "bias": bias, "res": res}


def _clip(name, kind, n, D, I, dtype, clips):
    """kind "block": the gradients of n blocks (dW1 [D,2I], dW_down [I,D], the
    norm's weight and bias in fp32).  kind "ragged": n tensors of D to I
    elements, one after another in a flat buffer."""
    return {"name": name, "op": "clip", "kind": kind, "n": n, "D": D, "I": I, "dtype": dtype, "clips": clips}


def _moe(name, M, D, I, E, k, renorm):
    return {"name": name, "op": "moe", "M": M, "D": D, "I": I, "E": E, "k": k, "renorm": renorm}


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    """A case of the listed ones' ranges: rows 1 to 11136 and widths 64 to
    8192 (up to 40 M elements), 1 to 301 gradients of up to 1.2 GB together,
    1 to 64 tokens over 4 to 64 experts."""
    op = rng.choice(["norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd", "clip", "clip", "moe", "moe"])
    if op in ("norm_fwd", "norm_bwd"):
        D = _log(rng, 64, 8192)
        if rng.random() < 0.5:
            D = max(64, D // 64 * 64)
        M = min(_log(rng, 1, 11136), 40_000_000 // D)
        c = _norm("", op, M, D, rng.choice(["bf16", "bf16", "fp16", "fp32"]), "fp32", rng.random() < 0.7,
                  op == "norm_bwd" and rng.random() < 0.5)
        if rng.random() < 0.3:
            c["wdtype"] = c["dtype"]
    elif op == "clip":
        dt, clips = rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.random() < 0.6
        if rng.random() < 0.5:
            c = _clip("", "block", rng.randint(1, 4), 64 * _log(rng, 4, 56), 64 * _log(rng, 8, 112), dt, clips)
        else:
            n = _log(rng, 1, 301)
            c = _clip("", "ragged", n, 1, _log(rng, 100, 400_000), dt, clips)
    else:
        E = rng.randint(4, 64)
        c = _moe("", _log(rng, 1, 64), 64 * _log(rng, 4, 56), 64 * _log(rng, 4, 32), E, rng.randint(1, min(E, 8)),
                 rng.random() < 0.5)
    del c["name"]
    return c


def _clip_sizes(c):
    """(numbers of elements of the tensors of the case's type, of the fp32 ones)."""
    if c["kind"] == "block":
        D, I = c["D"], c["I"]
        return [D * 2 * I, I * D] * c["n"], [D, D] * c["n"]
    r = torch.Generator().manual_seed(c["n"] * 7919 + c["I"])
    u = torch.rand(c["n"], generator=r, dtype=torch.float64)
    lo, hi = c["D"], c["I"]
    return [max(1, int(lo * (hi / lo) ** v)) for v in u.tolist()], []


def work(c):
    if c["op"] == "moe":
        # the experts that c["M"] tokens' independent choices hit, on average
        hit = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["M"])
        per = 3 * c["D"] * c["I"] * 2
        return {"bytes": hit * per + c["M"] * c["D"] * 4 + c["D"] * c["E"] * 2 + c["M"] * c["k"] * 8,
                "flops": 6 * c["M"] * c["k"] * c["D"] * c["I"] + 2 * c["M"] * c["D"] * c["E"]}
    if c["op"] == "clip":
        typed, f32 = _clip_sizes(c)
        n, b = sum(typed) + sum(f32), sum(typed) * SIZE[c["dtype"]] + sum(f32) * 4
        return {"bytes": 2 * b if c["clips"] else b, "flops": (3 if c["clips"] else 2) * n}
    n, s, w = c["M"] * c["D"], SIZE[c["dtype"]], c["D"] * SIZE[c["wdtype"]]
    vecs = 2 if c["bias"] else 1
    if c["op"] == "norm_fwd":
        return {"bytes": 2 * n * s + vecs * w + 8 * c["M"], "flops": 8 * n}
    return {"bytes": (4 if c["res"] else 3) * n * s + w + vecs * w + 8 * c["M"], "flops": 14 * n}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def prepare(c, seed):
    g = _gen(seed)
    if c["op"] == "moe":
        M, D, I, E = c["M"], c["D"], c["I"], c["E"]
        bf = torch.bfloat16
        return {"case": c, "x": _randn((M, D), g, bf), "Wr": _randn((D, E), g, bf, D ** -0.5),
                "W1": _randn((E, D, 2 * I), g, bf, D ** -0.5), "Wd": _randn((E, I, D), g, bf, I ** -0.5)}
    if c["op"] == "clip":
        typed, f32 = _clip_sizes(c)
        st = {"case": c, "grads": [], "flat": [], "outs": None, "flat_out": []}
        for sizes, dtype in ((typed, DT[c["dtype"]]), (f32, torch.float32)):
            if not sizes:
                continue
            # a bucket: the tensors one after another in one flat buffer
            flat = _randn((sum(sizes),), g, dtype, 1e-2)
            st["flat"].append(flat)
            st["grads"] += list(flat.split(sizes))
            if c["clips"]:
                out = torch.zeros_like(flat)
                st["flat_out"].append(out)
                st["outs"] = (st["outs"] or []) + list(out.split(sizes))
        n = sum(typed) + sum(f32)
        st["max_norm"] = 1e-2 * n ** 0.5 * (0.4 if c["clips"] else 3.0) + 1e-3
        return st
    M, D, dt, wt = c["M"], c["D"], DT[c["dtype"]], DT[c["wdtype"]]
    # a residual stream: rows of different scale and offset, a few loud channels
    x = torch.randn((M, D), generator=g, device="cuda")
    x = x * (0.5 + 2 * torch.rand((M, 1), generator=g, device="cuda")) + 0.3 * torch.randn((M, 1), generator=g, device="cuda")
    x *= torch.where(torch.rand((D,), generator=g, device="cuda") < 0.003, 12.0, 1.0)
    st = {"case": c, "x": x.to(dt), "w": (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(wt),
          "b": (0.1 * torch.randn(D, generator=g, device="cuda")).to(wt) if c["bias"] else None}
    if c["op"] == "norm_bwd":
        xf = st["x"].double()
        mean = xf.mean(1)
        st["mean"] = mean.float()
        st["rstd"] = ((xf - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        st["dy"] = _randn((M, D), g, dt, 1e-1)
        st["res"] = _randn((M, D), g, dt, 1e-1) if c["res"] else None
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s, s["case"])


def _own(s, c):
    import bwd_gemm_epilogue_amd as sw
    if c["op"] == "norm_fwd":
        return sw.swiglu_layer_norm_fwd(s["x"], s["w"], s["b"], EPS)
    if c["op"] == "norm_bwd":
        dx, dw, db = sw.swiglu_layer_norm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], dres=s["res"],
                                              bias_grad=c["bias"])
        return (dx, dw, db) if c["bias"] else (dx, dw)
    if c["op"] == "clip":
        norm = sw.swiglu_clip_grad_norm(s["grads"], s["max_norm"], outs=s["outs"])
        return [norm] + (s["flat_out"] if c["clips"] else s["flat"])
    return sw.swiglu_moe_few_layer(s["x"], s["Wr"], s["W1"], s["Wd"], c["k"], renormalize=c["renorm"])


def _plain(s, c):
    if c["op"] == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = (xc.square().mean(1) + EPS).rsqrt()
        y = xc * rstd[:, None] * s["w"].float()
        if s["b"] is not None:
            y = y + s["b"].float()
        return y.to(s["x"].dtype), mean, rstd
    if c["op"] == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["w"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if s["res"] is not None:
            dx = dx + s["res"].float()
        dw = (dy * xh).sum(0).to(s["w"].dtype)
        out = (dx.to(s["x"].dtype), dw)
        return out + (dy.sum(0).to(s["w"].dtype),) if c["bias"] else out
    if c["op"] == "clip":
        total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
        coef = (s["max_norm"] / (total + 1e-6)).clamp(max=1.0).float()
        if c["clips"]:
            return [total.float()] + [torch.mul(f.float(), coef, out=o) if o.dtype == torch.float32
                                      else o.copy_(f.float() * coef) for f, o in zip(s["flat"], s["flat_out"])]
        # unclipped gradients are multiplied by one in place
        return [total.float()] + [f.mul_(coef) if f.dtype == torch.float32 else f.copy_(f.float() * coef)
                                  for f in s["flat"]]
    # experts: the chosen experts' matrices where that is fewer of them than all
    x, k, E = s["x"], c["k"], c["E"]
    logits = x.double() @ s["Wr"].double()          # 64 bits: a choice depends on it
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    top = torch.gather(torch.softmax(logits, 1), 1, ids)
    if c["renorm"]:
        top = top / top.sum(1, keepdim=True)
    top, I = top.float(), c["I"]
    xf = x.float()
    if ids.numel() < E:
        at = ids.reshape(-1)
        pre = torch.matmul(xf.repeat_interleave(k, 0)[:, None], s["W1"][at].float())
        h = pre[..., :I] * (pre[..., I:] / (1 + torch.exp(-pre[..., I:])))
        out = torch.matmul(h, s["Wd"][at].float()).reshape(x.shape[0], k, -1)
        y = (out * top[..., None]).sum(1)
    else:
        pre = torch.matmul(xf[None], s["W1"].float())
        h = pre[..., :I] * (pre[..., I:] / (1 + torch.exp(-pre[..., I:])))
        gates = torch.zeros(x.shape[0], E, device=x.device).scatter_(1, ids, top)
        y = (torch.matmul(h, s["Wd"].float()) * gates.t()[..., None]).sum(0)
    return y.to(x.dtype), ids.to(torch.int32), top


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm_fwd":
        x, D = s["x"].double(), c["D"]
        mu = x.sum(1) / D
        sigma2 = ((x - mu.unsqueeze(1)) ** 2).sum(1) / D
        r = 1 / torch.sqrt(sigma2 + EPS)
        y = torch.addcmul(torch.zeros((), dtype=torch.float64, device="cuda") if s["b"] is None else s["b"].double(),
                          (x - mu.unsqueeze(1)) * r.unsqueeze(1), s["w"].double())
        return y, mu, r
    if c["op"] == "norm_bwd":
        # the gradient of <dy, y(x, w, b)> (+ <res, x>), by differentiation of the definition
        x, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
        b = torch.zeros(c["D"], dtype=torch.float64, device="cuda", requires_grad=True)
        mu = x.sum(1, keepdim=True) / c["D"]
        sigma2 = ((x - mu) ** 2).sum(1, keepdim=True) / c["D"]
        loss = (((x - mu) / torch.sqrt(sigma2 + EPS) * w + b) * s["dy"].double()).sum()
        if s["res"] is not None:
            loss = loss + (s["res"].double() * x).sum()
        got = torch.autograd.grad(loss, (x, w, b))
        return got if c["bias"] else got[:2]
    if c["op"] == "clip":
        norm = sum(float(f.double().dot(f.double())) for f in s["flat"]) ** 0.5
        scale = min(1.0, s["max_norm"] / (norm + 1e-6))
        return [torch.tensor(norm, dtype=torch.float64)] + [f.double() * scale for f in s["flat"]]
    x, E, I = s["x"].double(), c["E"], c["I"]
    l = x @ s["Wr"].double()
    p = torch.exp(l - l.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True)
    # rank of each expert: how many are larger, or equal with a lower index
    e = torch.arange(E, device="cuda")
    ahead = (l[:, None, :] > l[:, :, None]) | ((l[:, None, :] == l[:, :, None]) & (e[None, None, :] < e[None, :, None]))
    rank = ahead.sum(2)
    order = torch.zeros_like(rank).scatter_(1, rank, e.expand_as(rank))[:, :c["k"]]
    chosen = torch.where(rank < c["k"], p, torch.zeros_like(p))
    if c["renorm"]:
        chosen = chosen / chosen.sum(1, keepdim=True)
    y = torch.zeros(c["M"], c["D"], dtype=torch.float64, device="cuda")
    for i in range(E):
        rows = (rank[:, i] < c["k"]).nonzero().flatten()
        if rows.numel() == 0:
            continue
        pre = x[rows] @ s["W1"][i].double()
        left, gate = pre[:, :I], pre[:, I:]
        y[rows] += chosen[rows, i, None] * ((left * gate * torch.sigmoid(gate)) @ s["Wd"][i].double())
    return y, order.to(torch.int32), torch.gather(chosen, 1, order)
