"""Timed cases of the operators at the two ends of a layer of packed experts:
between the residual stream and the experts, and between the last layer and
the loss.  Each with its plain form (elementary torch operations in 32 bits or
more, rounded once at the end), its definition in 64 bits and the library's
entry points:

* ``norm``        residual addition and root-mean-square norm, the normed rows
                  as 8-bit integers with one scale each, or in bf16
* ``norm_bwd``    its gradients: of the sum and of the norm's weight
* ``route``       top-k routing of tokens to experts: pairs, weights, per-expert
                  counts, the rows sorted by expert, and the balance loss
* ``route_bwd``   the gradient of the weights and of the balance loss at the
                  router's logits
* ``combine``     a token's expert rows added up with its weights
* ``combine_bwd`` its gradients: of the rows and of the weights
* ``head``        softmax cross entropy of an output head without keeping the
                  logits, the head in bf16 or in 8 bits
* ``head_bwd``    its gradients: of the hidden rows and, in bf16, of the head
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode token in front of an 8-bit projection: latency
        dict(name="norm_token", op="norm", rows=1, d=7168, x="bf16", res="bf16", q8=True),
        # prompt or scoring batch in front of an 8-bit projection
        dict(name="norm_prefill", op="norm", rows=8192, d=7168, x="bf16", res="bf16", q8=True),
        # a training step's gradient, ragged batch, the stream's own gradient joining it
        dict(name="norm_bwd_train", op="norm_bwd", rows=4099, d=7168, h="bf16", dy="bf16", joined=True),
        # one decode token's routing, 8 of 256 experts
        dict(name="route_token", op="route", tokens=1, experts=256, top_k=8, dtype="fp32", renorm=True, padded=0.0),
        # routing of a long prompt pass, some of its tokens padding
        dict(name="route_prefill", op="route", tokens=16384, experts=256, top_k=8, dtype="fp32", renorm=True, padded=0.02),
        # the router's gradient of a training step
        dict(name="route_bwd_train", op="route_bwd", tokens=8191, experts=256, top_k=8, dtype="bf16", renorm=True, padded=0.02),
        # 2048 prompt tokens, 8 expert rows each as the packed down product leaves them
        dict(name="combine_prefill", op="combine", tokens=2048, top_k=8, d=7168, z="fp32", y="fp32", weighted=True, padded=0.0),
        # its gradients in a training step of a narrower layer, ragged batch with padding
        dict(name="combine_bwd_train", op="combine_bwd", tokens=1021, top_k=8, d=4096, z="fp32", dy="bf16", dz="bf16", padded=0.02),
        # scoring one short text under an 8-bit head of odd vocabulary: the weights' stream
        dict(name="head_q8_score", op="head", rows=37, vocab=100003, d=7168, w="int8", ignored=0.0),
        # training forward under a bf16 head
        dict(name="head_train", op="head", rows=4096, vocab=131072, d=7168, w="bf16", ignored=0.05),
        # gradient through a frozen 8-bit head to the hidden rows
        dict(name="head_bwd_frozen", op="head_bwd", rows=2048, vocab=131072, d=7168, w="int8", ignored=0.05),
        # both gradients of a trained head, ragged batch, odd vocabulary
        dict(name="head_bwd_train", op="head_bwd", rows=4099, vocab=50021, d=7168, w="bf16", ignored=0.05),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "route", "route_bwd", "combine", "combine_bwd", "head", "head", "head_bwd",
                     "head_bwd"])
    kind = lambda: rng.choice(["bf16", "fp32"])  # noqa: E731
    if op == "norm":
        return dict(op=op, rows=_log_int(rng, 1, 8192), d=_log_int(rng, 64, 8192), x=kind(),
                    res=rng.choice(["none", "bf16", "fp32"]), q8=rng.random() < 0.6)
    if op == "norm_bwd":
        return dict(op=op, rows=_log_int(rng, 1, 8192), d=_log_int(rng, 64, 8192), h=kind(), dy=kind(), joined=rng.random() < 0.5)
    if op in ("route", "route_bwd"):
        experts = _log_int(rng, 2, 512)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts, top_k=rng.randint(1, min(8, experts)), dtype=kind(),
                    renorm=rng.random() < 0.6, padded=rng.choice([0.0, 0.02, 0.3]))
    if op in ("combine", "combine_bwd"):
        c = dict(op=op, tokens=_log_int(rng, 1, 4096), top_k=rng.randint(1, 8), d=_log_int(rng, 64, 8192), z=kind(),
                 padded=rng.choice([0.0, 0.02, 0.3]))
        return dict(c, y=kind(), weighted=rng.random() < 0.7) if op == "combine" else dict(c, dy=kind(), dz=kind())
    return dict(op=op, rows=_log_int(rng, 1, 4099), vocab=_log_int(rng, 500, 131072), d=_log_int(rng, 64, 7168),
                w=rng.choice(["bf16", "int8"]), ignored=rng.choice([0.0, 0.05, 0.5]))


def _size(kind):
    return {"none": 0.0, "int8": 1.0, "bf16": 2.0, "fp32": 4.0}[kind]


def work(c):
    op = c["op"]
    if op == "norm":
        out = (1.0 if c["q8"] else 2.0) + _size(c["res"])
        return {"bytes": c["rows"] * c["d"] * (_size(c["x"]) + _size(c["res"]) + out) + 4.0 * c["d"], "flops": 8.0 * c["rows"] * c["d"]}
    if op == "norm_bwd":
        n = _size(c["h"]) * (3 if c["joined"] else 2) + _size(c["dy"])
        return {"bytes": c["rows"] * c["d"] * n + 8.0 * c["d"], "flops": 10.0 * c["rows"] * c["d"]}
    if op in ("route", "route_bwd"):
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        logits = _size(c["dtype"]) * t * e
        if op == "route":
            return {"bytes": logits + 20.0 * t * k + 8.0 * e, "flops": 6.0 * t * e}
        return {"bytes": 2 * logits + 12.0 * t * k, "flops": 10.0 * t * e}
    if op in ("combine", "combine_bwd"):
        t, k, d = c["tokens"], c["top_k"], c["d"]
        if op == "combine":
            return {"bytes": t * d * (k * _size(c["z"]) + _size(c["y"])) + 8.0 * t * k, "flops": 2.0 * t * k * d}
        return {"bytes": t * d * (_size(c["dy"]) + k * (_size(c["z"]) + _size(c["dz"]))) + 12.0 * t * k, "flops": 3.0 * t * k * d}
    n, v, d = c["rows"], c["vocab"], c["d"]
    operands = _size(c["w"]) * (n + v) * d + 12.0 * n
    prod = 2.0 * n * v * d
    if op == "head":
        return {"bytes": operands, "flops": prod}
    # the logits are not kept: their product once more, then that of each gradient
    if c["w"] == "int8":
        return {"bytes": operands + 2.0 * n * d, "flops": 2 * prod}
    return {"bytes": operands + 2.0 * (n + v) * d, "flops": 3 * prod}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, shape, std=1.0):
    return torch.randn(shape, device="cuda", generator=gen) * std


def _rand(gen, shape):
    return torch.rand(shape, device="cuda", generator=gen)


def _rows(t, align):
    """`t` with rows that start on 16 bytes, as a program keeps them."""
    n, d = t.shape
    wide = torch.zeros((n, (d + align - 1) // align * align), dtype=t.dtype, device=t.device)
    wide[:, :d] = t
    return wide[:, :d]


def _pad_tokens(c):
    """How many tokens at the end are padding."""
    return int(c["tokens"] * c["padded"])


def _hidden(gen, rows, d, outliers=True):
    """Rows of a residual stream: a few channels many times the others."""
    x = _randn(gen, (rows, d))
    if outliers:
        x[:, :: 97] *= 8.0
    return x


def _quantize(x):
    scale = x.abs().amax(1) / 127.0
    return torch.round(x / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def _head_rows(s):
    """The head's operands as numbers in 32 bits: hidden rows, head, and the scales of the logits."""
    x, w = s["x"].float(), s["w"].float()
    return x, w, (s["x_scale"][:, None] * s["w_scale"] if s["x_scale"] is not None else 1.0)


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(c)
    op = c["op"]
    if op == "norm":
        rows, d = c["rows"], c["d"]
        s["x"] = _hidden(gen, rows, d).to(DTYPES[c["x"]])
        s["residual"] = None if c["res"] == "none" else (4.0 * _hidden(gen, rows, d)).to(DTYPES[c["res"]])
        s["weight"] = 1.0 + _randn(gen, d, 0.1)
    elif op == "norm_bwd":
        rows, d = c["rows"], c["d"]
        s["h"] = (4.0 * _hidden(gen, rows, d)).to(DTYPES[c["h"]])
        s["weight"] = 1.0 + _randn(gen, d, 0.1)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["dy"] = _randn(gen, (rows, d), 1e-3).to(DTYPES[c["dy"]])
        s["dh"] = _randn(gen, (rows, d), 1e-3).to(DTYPES[c["h"]]) if c["joined"] else None
    elif op in ("route", "route_bwd"):
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        # some experts better liked than others; the logits of padding are masked throughout
        x = _randn(gen, (t, e)) + _randn(gen, (e,), 0.7)
        pads = _pad_tokens(c)
        if pads:
            x[t - pads:] = float("-inf")
        s["logits"] = x.to(DTYPES[c["dtype"]])
        if op == "route_bwd":
            r = _plain_route(dict(s, op="route"))
            s["pair_expert"], s["pair_row"], s["counts"] = r["pair_expert"], r["pair_row"], r["counts"]
            s["grad_weight"] = _randn(gen, (t * k,), 1e-2)
            s["grad_balance"] = 1e-2 * (1.0 + _rand(gen, (1,)))
    elif op in ("combine", "combine_bwd"):
        t, k, d = c["tokens"], c["top_k"], c["d"]
        live = (t - _pad_tokens(c)) * k
        s["pair_row"] = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
        s["pair_row"][:live] = torch.randperm(live, device="cuda", generator=gen).int()
        s["z"] = _randn(gen, (live, d)).to(DTYPES[c["z"]])
        w = _rand(gen, (t, k)) + 0.05
        s["weight"] = (w / w.sum(1, keepdim=True)).reshape(-1) if c.get("weighted", True) else None
        if op == "combine_bwd":
            s["dy"] = _randn(gen, (t, d), 1e-3).to(DTYPES[c["dy"]])
    else:
        n, v, d = c["rows"], c["vocab"], c["d"]
        targets = torch.randint(0, v, (n,), device="cuda", generator=gen)
        w = _randn(gen, (v, d), 0.02)
        # hidden rows that lean towards their targets, from not at all to almost sure
        lean = 12.0 / (0.0004 * d) * _rand(gen, (n, 1))
        x = _randn(gen, (n, d), math.sqrt(min(1.0, 4.0 / (0.0004 * d)))) + lean * w[targets]
        if c["w"] == "int8":
            w, s["w_scale"] = _quantize(w)
            x, s["x_scale"] = _quantize(x)
            s["x"], s["w"] = _rows(x, 16), _rows(w, 16)
        else:
            s["x"], s["w"], s["x_scale"], s["w_scale"] = _rows(x.bfloat16(), 8), _rows(w.bfloat16(), 8), None, None
        targets[_rand(gen, (n,)) < c["ignored"]] = -1
        s["targets"] = targets.int()
        if op == "head_bwd":
            s["lse"] = torch.empty(n, device="cuda")
            x, w, scale = _head_rows(s)
            for r in range(0, n, 1024):
                part = scale if isinstance(scale, float) else scale[r:r + 1024]
                s["lse"][r:r + 1024] = torch.logsumexp((x[r:r + 1024] @ w.t()) * part, 1)
            s["grad_loss"] = (0.5 + _rand(gen, (n,))) / n
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is None:
        h = s["x"]
    else:
        h = (x + s["residual"].float()).to(s["residual"].dtype)
    f = h.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(1) + EPS)
    out = {"rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    if s["q8"]:
        v = f * s["weight"]
        step = (v.abs().amax(1).double() / 127.0).float()
        div = torch.where(step > 0, step, 1.0).double()
        q = torch.round(v.double() / div[:, None]).float()   # next to a half the quotient needs more than 32 bits
        scale = step * rstd
        out["scale"] = scale
        out["values"] = (q * scale[:, None]).bfloat16()
    else:
        out["y"] = (f * rstd[:, None] * s["weight"]).bfloat16()
    return out


def _plain_norm_bwd(s):
    f, dy = s["h"].float(), s["dy"].float()
    unit = f * s["rstd"][:, None]
    g = dy * s["weight"]
    dx = s["rstd"][:, None] * (g - unit * (g * unit).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dweight": (dy * unit).sum(0)}


def _plain_route(s):
    l = s["logits"].float()
    t, e, k = s["tokens"], s["experts"], s["top_k"]
    top = l.amax(1, keepdim=True)
    live = top > float("-inf")
    x = torch.exp(l - torch.where(live, top, 0.0))
    p = x / torch.where(live, x.sum(1, keepdim=True), 1.0)
    chosen = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(x, 1, chosen)
    w = w / torch.where(live, w.sum(1, keepdim=True), 1.0) if s["renorm"] else torch.gather(p, 1, chosen)
    pair_expert = torch.where(live, chosen, -1).reshape(-1)
    pair_weight = torch.where(live, w, 0.0).reshape(-1)
    bin_of = torch.where(pair_expert < 0, e, pair_expert)
    counts = torch.zeros(e + 1, dtype=torch.int64, device="cuda").scatter_add_(0, bin_of, torch.ones_like(bin_of))[:e]
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)])
    row_pair = torch.sort(bin_of, stable=True).indices
    at = torch.arange(t * k, device="cuda")
    used = at < offsets[-1]
    pair_row = torch.empty_like(at).scatter_(0, row_pair, torch.where(used, at, -1))
    f = counts.float() / torch.clamp(counts.sum(), min=1)
    mean_p = p.sum(0) / torch.clamp(live.sum(), min=1)
    return {"pair_expert": pair_expert.int(), "pair_weight": pair_weight, "counts": counts.int(), "offsets": offsets.int(),
            "pair_row": pair_row.int(), "row_token": torch.where(used, row_pair // k, 0).int(),
            "row_weight": torch.where(used, pair_weight[row_pair], 0.0), "balance": (e * (f * mean_p).sum()).reshape(1)}


def _plain_route_bwd(s):
    l = s["logits"].float()
    t, e, k = s["tokens"], s["experts"], s["top_k"]
    chosen = s["pair_expert"].long().view(t, k)
    live = chosen[:, :1] >= 0
    chosen = torch.where(live, chosen, 0)
    # the weights' gradient comes in the order of the sorted rows
    row = s["pair_row"].long().view(t, k)
    g = torch.where(row >= 0, s["grad_weight"][torch.clamp(row, min=0)], 0.0)
    top = torch.where(live, l.amax(1, keepdim=True), 0.0)
    x = torch.exp(l - top)
    p = x / torch.where(live, x.sum(1, keepdim=True), 1.0)
    if s["renorm"]:
        w = torch.gather(x, 1, chosen)
        w = w / torch.where(live, w.sum(1, keepdim=True), 1.0)
        d = torch.zeros_like(l).scatter_(1, chosen, w * (g - (g * w).sum(1, keepdim=True)))
    else:
        full = torch.zeros_like(l).scatter_(1, chosen, g)
        d = p * (full - (full * p).sum(1, keepdim=True))
    total = torch.clamp(s["counts"].sum(), min=1).float()
    c = s["grad_balance"] * e * (s["counts"].float() / total) / (total / k)
    d = d + p * (c - (c * p).sum(1, keepdim=True))
    return torch.where(live, d, 0.0).to(s["logits"].dtype)


def _plain_combine(s):
    t, k = s["tokens"], s["top_k"]
    row = s["pair_row"].long()
    z = s["z"].float()[torch.clamp(row, min=0)]
    z = z * s["weight"][:, None] if s["weight"] is not None else z
    z = torch.where(row[:, None] >= 0, z, 0.0)
    return z.view(t, k, -1).sum(1).to(DTYPES[s["y"]])


def _plain_combine_bwd(s):
    t, k, d = s["tokens"], s["top_k"], s["d"]
    live = s["pair_row"] >= 0
    row = s["pair_row"].long()[live]
    dy = s["dy"].float()[:, None, :].expand(t, k, d).reshape(t * k, d)[live]
    dz = torch.empty_like(s["z"], dtype=DTYPES[s["dz"]])
    dz[row] = (dy * s["weight"][live][:, None]).to(dz.dtype)
    dw = torch.zeros(t * k, device="cuda")
    dw[live] = (dy * s["z"].float()[row]).sum(1)
    return {"dz": dz, "dweight": dw}


def _plain_logits(s):
    x, w, scale = _head_rows(s)
    l = x @ w.t()
    return l if s["x_scale"] is None else l * scale


def _plain_head(s):
    l = _plain_logits(s)
    m = l.amax(1, keepdim=True)
    z = torch.exp(l - m).sum(1)
    lse = m[:, 0] + torch.log(z)
    kept = s["targets"] >= 0
    at = torch.where(kept, s["targets"], 0).long()
    hit = l[torch.arange(s["rows"], device="cuda"), at]
    return {"loss": torch.where(kept, torch.log(z) - (hit - m[:, 0]), 0.0), "lse": lse}


def _plain_head_bwd(s):
    x, w, _ = _head_rows(s)
    kept = s["targets"] >= 0
    g = torch.where(kept, s["grad_loss"], 0.0)
    d = torch.exp(_plain_logits(s) - s["lse"][:, None]) * g[:, None]
    at = torch.where(kept, s["targets"], 0).long()
    d[torch.arange(s["rows"], device="cuda"), at] -= g
    if s["w"].dtype == torch.int8:
        return {"dx": ((d * s["w_scale"]) @ w).bfloat16()}
    return {"dx": (d @ w).bfloat16(), "dw": (d.t() @ x).bfloat16()}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "route": _plain_route, "route_bwd": _plain_route_bwd,
          "combine": _plain_combine, "combine_bwd": _plain_combine_bwd, "head": _plain_head, "head_bwd": _plain_head_bwd}


def run(s):
    op = s["op"]
    if not own:
        return _PLAIN[op](s)
    import sparse_ternary_bit_amd as stq
    if op == "norm":
        r = stq.rmsnorm_rows(s["x"], s["weight"], eps=EPS, residual=s["residual"], need_q=s["q8"], need_y=not s["q8"])
        out = {"rstd": r.rstd}
        if s["residual"] is not None:
            out["h"] = r.h
        if s["q8"]:
            values = torch.empty(r.q.shape, dtype=torch.bfloat16, device="cuda")
            return dict(out, scale=r.scale, values=torch.mul(r.q, r.scale[:, None], out=values))
        return dict(out, y=r.y)
    if op == "norm_bwd":
        dx, dweight = stq.rmsnorm_rows_backward(s["h"], s["weight"], s["rstd"], s["dy"], dh=s["dh"])
        return {"dx": dx, "dweight": dweight}
    if op == "route":
        return stq.route_tokens(s["logits"], s["top_k"], renormalize=s["renorm"])._asdict()
    if op == "route_bwd":
        return stq.route_tokens_backward(s["logits"], s["pair_expert"], s["counts"], s["top_k"], renormalize=s["renorm"],
                                         grad_weight=s["grad_weight"], pair_row=s["pair_row"], grad_balance=s["grad_balance"])
    if op == "combine":
        return stq.combine_rows(s["z"], s["pair_row"], s["top_k"], weight=s["weight"], out_dtype=DTYPES[s["y"]])
    if op == "combine_bwd":
        dz, dweight = stq.combine_rows_backward(s["dy"], s["pair_row"], s["top_k"], s["z"], weight=s["weight"],
                                                dz_dtype=DTYPES[s["dz"]])
        return {"dz": dz, "dweight": dweight}
    if op == "head":
        loss, lse = stq.head_cross_entropy(s["x"], s["w"], s["targets"], x_scale=s["x_scale"], w_scale=s["w_scale"])
        return {"loss": loss, "lse": lse}
    dx, dw = stq.head_cross_entropy_backward(s["x"], s["w"], s["targets"], s["lse"], s["grad_loss"], x_scale=s["x_scale"],
                                             w_scale=s["w_scale"], need_dw=s["w"].dtype != torch.int8)
    return {"dx": dx} if dw is None else {"dx": dx, "dw": dw}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    dev = "cuda"
    if op == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            h = h + s["residual"].double()
            out["h"] = h
            # the norm is that of the stored sum
            h = h.float().to(s["residual"].dtype).double()
        rms = torch.sqrt(h.square().mean(1) + EPS)
        y = h / rms[:, None] * s["weight"].double()
        out["rstd"] = 1 / rms
        if c["q8"]:
            scale = y.abs().amax(1) / 127
            out["scale"] = scale
            return dict(out, values=torch.round(y / scale[:, None]) * scale[:, None])
        return dict(out, y=y)
    if op == "norm_bwd":
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()
        wdy = dy * s["weight"].double()
        dot = torch.linalg.vecdot(wdy, h) / c["d"]
        dx = r[:, None] * wdy - (r.pow(3) * dot)[:, None] * h
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dweight": torch.mv((dy * h).t(), r)}
    if op == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        n = t - _pad_tokens(c)
        l = s["logits"][:n].double()
        p = torch.softmax(l, 1)
        order = torch.argsort(-l, dim=1, stable=True)[:, :k]
        w = torch.gather(p, 1, order)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
        flat = order.reshape(-1)
        counts = torch.bincount(flat, minlength=e)
        by_expert = torch.argsort(flat, stable=True)
        weight, row_weight = (torch.zeros(t * k, dtype=torch.float64, device=dev) for _ in range(2))
        weight[:n * k] = w.reshape(-1)
        row_weight[:n * k] = w.reshape(-1)[by_expert]
        balance = e * torch.dot(counts.double() / max(1, n * k), p.mean(0)) if n else torch.zeros((), dtype=torch.float64, device=dev)
        return {"pair_expert": None, "pair_weight": weight, "counts": None, "offsets": None, "pair_row": None, "row_token": None,
                "row_weight": row_weight, "balance": balance.reshape(1)}
    if op == "route_bwd":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        n = t - _pad_tokens(c)
        d = torch.zeros((t, e), dtype=torch.float64, device=dev)
        with torch.enable_grad():
            l = s["logits"][:n].double().requires_grad_()
            p = torch.softmax(l, 1)
            w = torch.gather(p, 1, s["pair_expert"][:n * k].long().view(n, k))
            w = w / w.sum(1, keepdim=True) if c["renorm"] else w
            g = s["grad_weight"].double()[s["pair_row"][:n * k].long()].view(n, k)
            balance = e * torch.dot(s["counts"].double() / max(1, n * k), p.sum(0) / max(1, n))
            d[:n] = torch.autograd.grad((w * g).sum() + s["grad_balance"].double()[0] * balance, l)[0]
        return d
    if op in ("combine", "combine_bwd"):
        t, k, d = c["tokens"], c["top_k"], c["d"]
        live = (t - _pad_tokens(c)) * k
        row = s["pair_row"][:live].long()
        token = torch.arange(live, device=dev) // k
        w = s["weight"].double()[:live, None] if s["weight"] is not None else 1.0
        if op == "combine":
            y = torch.zeros((t, d), dtype=torch.float64, device=dev)
            return y.index_add_(0, token, s["z"].double()[row] * w)
        dy = s["dy"].double()[token]
        dz = torch.zeros((live, d), dtype=torch.float64, device=dev)
        dz[row] = dy * w
        dw = torch.zeros(t * k, dtype=torch.float64, device=dev)
        dw[:live] = torch.linalg.vecdot(dy, s["z"].double()[row])
        return {"dz": dz, "dweight": dw}
    n, v, d = c["rows"], c["vocab"], c["d"]
    x, w = s["x"].double(), s["w"].double()
    if s["x_scale"] is not None:
        x, w = x * s["x_scale"].double()[:, None], w * s["w_scale"].double()[:, None]
    kept = s["targets"] >= 0
    if op == "head":
        loss, lse = torch.zeros(n, dtype=torch.float64, device=dev), torch.empty(n, dtype=torch.float64, device=dev)
        for r in range(0, n, 512):
            b = slice(r, min(n, r + 512))
            l = torch.matmul(w, x[b].t().contiguous()).t()
            lse[b] = torch.logsumexp(l, 1)
            picked = torch.gather(l, 1, s["targets"][b].clamp(min=0).long()[:, None])[:, 0]
            loss[b] = torch.where(kept[b], lse[b] - picked, 0.0)
        return {"loss": loss, "lse": lse}
    dx = torch.empty((n, d), dtype=torch.float64, device=dev)
    dw = torch.zeros((v, d), dtype=torch.float64, device=dev) if c["w"] == "bf16" else None
    for r in range(0, n, 512):
        b = slice(r, min(n, r + 512))
        g = torch.where(kept[b], s["grad_loss"][b].double(), 0.0)
        p = torch.exp(torch.matmul(w, x[b].t().contiguous()) - s["lse"][b].double())       # [vocab, rows]
        column = torch.arange(p.shape[1], device=dev)[kept[b]]
        p[s["targets"][b][kept[b]].long(), column] -= 1.0
        p *= g
        dx[b] = torch.matmul(p.t().contiguous(), w)
        if dw is not None:
            dw += torch.matmul(p, x[b])
    return {"dx": dx} if dw is None else {"dx": dx, "dw": dw}
