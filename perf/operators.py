"""Timed cases of the prompt-pass and scoring operators.

Three operators around the packed STQ1_0 experts, each with its plain form
(elementary torch operations in 32 bits or more, rounded once at the end) and
the library's entry points:

* ``swiglu``      gated feed-forward over STQ1_0 experts, rows grouped by
                  expert: h = silu(Wg x) * (Wu x), optionally saving [g | u]
* ``swiglu_bwd``  its gradients: dx through the packed weights and, for
                  training, dW of every expert
* ``q8``          rows quantized to 8-bit integers with one scale each, times
                  an 8-bit matrix with one scale per output channel
* ``logprobs``    log probabilities of given tokens, log-sum-exp, entropy and
                  the most likely alternatives of each row of logits
* ``logprobs_bwd`` the gradient of those log probabilities and entropies
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

QK = 256           # weights per STQ1_0 block
BLOCK_BYTES = 42   # bytes per block
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # prompt pass of one layer: 2048 tokens, 8 of 256 experts each, gate/up 2 x 2048 rows of 7168
        dict(name="swiglu_prefill", op="swiglu", experts=256, d_model=7168, d_ff=2048, rows=16384, skew=0.0, save=False),
        # a 37-token prompt on the same layer: about one row per expert, many experts with none; the weights dominate
        dict(name="swiglu_short_prompt", op="swiglu", experts=256, d_model=7168, d_ff=2048, rows=296, skew=0.0, save=False),
        # training forward of a narrow layer with uneven routing, pre-activations saved for the backward pass
        dict(name="swiglu_train", op="swiglu", experts=32, d_model=4096, d_ff=1024, rows=8191, skew=1.0, save=True),
        # gradient back through frozen packed experts to the layer's input, the full prompt
        dict(name="swiglu_bwd_frozen", op="swiglu_bwd", experts=256, d_model=7168, d_ff=2048, rows=16384, skew=0.0, dw=False),
        # one training step's gradients (inputs and weights) of the experts one GPU holds, a ragged batch
        dict(name="swiglu_bwd_train", op="swiglu_bwd", experts=8, d_model=7168, d_ff=2048, rows=4099, skew=0.5, dw=True),
        # one decode token through a matrix kept in 8 bits: latency and the weights' stream
        dict(name="q8_token", op="q8", m=1, k=7168, n=4096, out="bf16"),
        # output head of a decode batch, odd vocabulary, logits in fp32
        dict(name="q8_head", op="q8", m=64, k=7168, n=100003, out="fp32"),
        # prompt or scoring batch through an 8-bit projection
        dict(name="q8_prefill", op="q8", m=8192, k=7168, n=4096, out="bf16"),
        # one sampled token's log probability with 20 alternatives
        dict(name="logprobs_token", op="logprobs", rows=1, vocab=131072, dtype="fp32", top=20, masked=0.0),
        # scoring a corpus batch, padded vocabulary masked out
        dict(name="logprobs_score", op="logprobs", rows=4096, vocab=131072, dtype="bf16", top=5, masked=0.02),
        # gradient of a small fine-tuning batch, odd vocabulary
        dict(name="logprobs_bwd_small", op="logprobs_bwd", rows=17, vocab=50021, dtype="fp32", masked=0.0),
        # gradient of a training batch
        dict(name="logprobs_bwd_batch", op="logprobs_bwd", rows=4096, vocab=131072, dtype="bf16", masked=0.02),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["swiglu", "swiglu_bwd", "q8", "q8", "logprobs", "logprobs_bwd"])
    if op in ("swiglu", "swiglu_bwd"):
        c = dict(op=op, experts=_log_int(rng, 1, 256), d_model=QK * _log_int(rng, 1, 28), d_ff=QK * _log_int(rng, 1, 8),
                 rows=_log_int(rng, 1, 16384), skew=rng.choice([0.0, 0.0, 0.5, 1.0]))
        if op == "swiglu":
            c["save"] = rng.random() < 0.5
        else:
            c["dw"] = rng.random() < 0.5
            if c["dw"]:   # weight gradients are dense: as many experts as keep them near half a gigabyte
                c["rows"] = min(c["rows"], 8192)
                c["experts"] = max(1, min(c["experts"], (1 << 28) // (2 * c["d_ff"] * c["d_model"])))
        return c
    if op == "q8":
        c = dict(op=op, m=_log_int(rng, 1, 8192), k=_log_int(rng, 64, 8192), n=_log_int(rng, 64, 100003),
                 out=rng.choice(["bf16", "fp32"]))
        while c["m"] * c["n"] > 1 << 25 or c["m"] * c["n"] * c["k"] > 8192 * 7168 * 4096:
            c["n"] = max(64, c["n"] // 2)
            if c["n"] == 64:
                break
        return c
    c = dict(op=op, rows=_log_int(rng, 1, 4096), vocab=_log_int(rng, 1000, 200000), dtype=rng.choice(["bf16", "fp32"]),
             masked=rng.choice([0.0, 0.02, 0.5]))
    while c["rows"] * c["vocab"] * (2 if c["dtype"] == "bf16" else 4) > 4096 * 131072 * 2:
        c["rows"] = max(1, c["rows"] // 2)
    if op == "logprobs":
        c["top"] = rng.choice([0, 1, 5, 8, 20])
    return c


def _experts_used(c):
    return c["experts"] * (1.0 - (1.0 - 1.0 / c["experts"]) ** c["rows"])


def work(c):
    op = c["op"]
    if op in ("swiglu", "swiglu_bwd"):
        rows, d, f = c["rows"], c["d_model"], c["d_ff"]
        table = _experts_used(c) * 2 * f * d / QK * BLOCK_BYTES
        prod = 2.0 * rows * 2 * f * d
        if op == "swiglu":
            return {"bytes": table + rows * d * 2 + rows * f * 2 * (3 if c["save"] else 1), "flops": prod}
        nbytes = table + rows * 3 * f * 2 + rows * d * 2
        if c["dw"]:
            return {"bytes": nbytes + rows * d * 2 + c["experts"] * 2.0 * f * d * 2, "flops": 2 * prod}
        return {"bytes": nbytes, "flops": prod}
    if op == "q8":
        m, k, n = c["m"], c["k"], c["n"]
        return {"bytes": 2.0 * m * k + n * (k + 4.0) + m * n * (2.0 if c["out"] == "bf16" else 4.0), "flops": 2.0 * m * n * k}
    size = (2 if c["dtype"] == "bf16" else 4) * float(c["rows"]) * c["vocab"]
    if op == "logprobs":
        return {"bytes": size + c["rows"] * (16 + 8.0 * c["top"]), "flops": 5.0 * c["rows"] * c["vocab"]}
    return {"bytes": 2 * size + c["rows"] * 20.0, "flops": 6.0 * c["rows"] * c["vocab"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _routing(c, seed):
    """Rows of each expert: every row's expert drawn with probability ~ 1 / rank**skew."""
    rng = np.random.default_rng(seed)
    p = 1.0 / np.arange(1, c["experts"] + 1) ** c["skew"]
    rng.shuffle(p)
    counts = rng.multinomial(c["rows"], p / p.sum())
    return [0] + np.cumsum(counts).tolist()


def _packed(gen, experts, n, k):
    """Random packed experts (n a multiple of 64): any code bits are a valid pattern; the block
    scales are those that N(0, 0.02) weights get."""
    blocks = experts * n * (k // QK)
    t = torch.randint(0, 256, (blocks, BLOCK_BYTES), dtype=torch.uint8, device="cuda", generator=gen)
    d = 0.02 * (0.8 + 0.4 * torch.rand(blocks, device="cuda", generator=gen))
    t[:, :2] = d.half().view(torch.uint8).view(blocks, 2)
    return t.view(-1)


def _randn(gen, shape, std=1.0):
    return torch.randn(shape, device="cuda", generator=gen) * std


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = c["op"]
    s = dict(c)
    if op in ("swiglu", "swiglu_bwd"):
        rows, d, f = c["rows"], c["d_model"], c["d_ff"]
        s["bounds"] = _routing(c, seed)
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
        s["table"] = _packed(gen, c["experts"], 2 * f, d)
        s["stride"] = 2 * f * (d // QK) * BLOCK_BYTES
        s["x"] = _randn(gen, (rows, d)).bfloat16()
        if op == "swiglu_bwd":
            # pre-activations of unit-variance inputs, and the gradient that arrives at h
            s["gate_up"] = _randn(gen, (rows, 2 * f), 0.0173 * math.sqrt(d)).bfloat16()
            s["dh"] = _randn(gen, (rows, f), 1e-3).bfloat16()
    elif op == "q8":
        s["x"] = _randn(gen, (c["m"], c["k"])).bfloat16()
        # N(0, 0.02) channels quantized to 8 bits, in rows of whole 16-byte units as a program keeps them
        w = torch.zeros((c["n"], (c["k"] + 15) // 16 * 16), dtype=torch.int8, device="cuda")
        w[:, :c["k"]] = _randn(gen, (c["n"], c["k"]), 32.0).round().clamp(-127, 127)
        s["w"] = w[:, :c["k"]]
        s["w_scale"] = 6e-4 * (0.8 + 0.4 * torch.rand(c["n"], device="cuda", generator=gen))
    else:
        rows, vocab = c["rows"], c["vocab"]
        # a broad background and, in most rows, a few likely tokens
        x = _randn(gen, (rows, vocab), 2.0)
        ids = torch.randint(0, vocab, (rows, 4), device="cuda", generator=gen)
        x.scatter_add_(1, ids, 10.0 * torch.rand((rows, 4), device="cuda", generator=gen))
        keep = vocab - int(vocab * c["masked"])
        x[:, keep:] = float("-inf")
        s["logits"] = x.to(DTYPES[c["dtype"]])
        s["targets"] = torch.randint(0, keep, (rows,), dtype=torch.int32, device="cuda", generator=gen)
        if op == "logprobs_bwd":
            lse, entropy = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            for r in range(0, rows, 512):
                l = s["logits"][r:r + 512].double()
                z = torch.logsumexp(l, 1)
                p = torch.exp(l - z[:, None])
                lse[r:r + 512] = z
                entropy[r:r + 512] = -(p * torch.where(p > 0, l - z[:, None], 0.0)).sum(1)
            s["lse"], s["entropy"] = lse, entropy
            s["g_logprob"] = _randn(gen, (rows,))
            s["g_entropy"] = _randn(gen, (rows,), 0.01)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _pattern_table():
    rows = []
    for code in range(32):
        signs = [-1.0 if code >> i & 1 else 1.0 for i in range(3)]
        signs.insert(code >> 3, 0.0)
        rows.append(signs)
    return rows


def _decode(table, n, k):
    """fp32 [n, k] of one packed expert (n a multiple of 64) through the 32-entry pattern table."""
    nb = k // QK
    blk = table.view(n // 64, nb, 64, BLOCK_BYTES).transpose(1, 2).reshape(n, nb, BLOCK_BYTES)
    d = blk[..., :2].contiguous().view(torch.float16).float()                       # [n, nb, 1]
    b = blk[..., 2:34].reshape(n, nb, 8, 1, 4)
    nib = torch.cat([b & 15, b >> 4], 3).reshape(n, nb, 64)
    bit = torch.arange(8, dtype=torch.uint8, device=table.device).view(1, 1, 1, 8, 1)
    sel = (blk[..., 34:42].reshape(n, nb, 2, 1, 4) >> bit & 1).reshape(n, nb, 64)
    code = (nib | sel << 4).int()
    pat = torch.tensor(_pattern_table(), device=table.device)
    return (pat[code].view(n, nb, QK) * d).view(n, k)


def _expert(s, e):
    return s["table"][e * s["stride"]:(e + 1) * s["stride"]]


def _plain_swiglu(s):
    rows, d, f = s["rows"], s["d_model"], s["d_ff"]
    h = torch.empty((rows, f), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((rows, 2 * f), dtype=torch.bfloat16, device="cuda") if s["save"] else None
    for e in range(s["experts"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if lo == hi:
            continue
        z = s["x"][lo:hi].float() @ _decode(_expert(s, e), 2 * f, d).t()
        g, u = z[:, :f], z[:, f:]
        h[lo:hi] = (g / (1.0 + torch.exp(-g)) * u).bfloat16()
        if gu is not None:
            gu[lo:hi] = z.bfloat16()
    return (h, gu) if s["save"] else (h,)


def _plain_swiglu_bwd(s):
    rows, d, f = s["rows"], s["d_model"], s["d_ff"]
    dx = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros((s["experts"], 2 * f, d), dtype=torch.bfloat16, device="cuda") if s["dw"] else None
    for e in range(s["experts"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if lo == hi:
            continue
        g, u, dh = s["gate_up"][lo:hi, :f].float(), s["gate_up"][lo:hi, f:].float(), s["dh"][lo:hi].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        dz = torch.cat([dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig], 1)
        dx[lo:hi] = (dz @ _decode(_expert(s, e), 2 * f, d)).bfloat16()
        if dw is not None:
            dw[e] = (dz.t().contiguous() @ s["x"][lo:hi].float()).bfloat16()
    return (dx, dw) if s["dw"] else (dx,)


def _plain_q8(s):
    x = s["x"].float()
    scale = (x.abs().amax(1).double() / 127.0).float()
    div = torch.where(scale > 0, scale, 1.0).double()
    q = torch.round(x.double() / div[:, None]).float()   # next to a half the quotient needs more than 32 bits
    y = (q @ s["w"].float().t()) * scale[:, None] * s["w_scale"]
    return y.to(DTYPES[s["out"]])


def _plain_logprobs(s):
    l = s["logits"].float()
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - m)
    z = e.sum(1)
    lse = m[:, 0] + torch.log(z)
    mean = (e * torch.where(e > 0, l - m, 0.0)).sum(1) / z
    entropy = torch.log(z) - mean
    row = torch.arange(s["rows"], device="cuda")
    logprob = (l[row, s["targets"].long()] - m[:, 0]) - torch.log(z)
    ids = torch.empty((s["rows"], s["top"]), dtype=torch.int32, device="cuda")
    top = torch.empty((s["rows"], s["top"]), device="cuda")
    if s["top"]:
        pos = torch.arange(s["vocab"], dtype=torch.int32, device="cuda")
        left = l.clone()
        for i in range(s["top"]):
            v = left.amax(1, keepdim=True)
            j = torch.where(left == v, pos, s["vocab"]).amin(1)
            ids[:, i] = j
            top[:, i] = (v[:, 0] - m[:, 0]) - torch.log(z)
            left.scatter_(1, j[:, None].long(), float("-inf"))
    return logprob, lse, entropy, ids, top


def _plain_logprobs_bwd(s):
    l = s["logits"].float()
    lp = l - s["lse"][:, None]
    p = torch.exp(lp)
    d = -p * (s["g_logprob"][:, None] + s["g_entropy"][:, None] * torch.where(p > 0, lp + s["entropy"][:, None], 0.0))
    row = torch.arange(s["rows"], device="cuda")
    d[row, s["targets"].long()] += s["g_logprob"]
    return d.to(s["logits"].dtype)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["op"]
    if not own:
        return {"swiglu": _plain_swiglu, "swiglu_bwd": _plain_swiglu_bwd, "q8": _plain_q8, "logprobs": _plain_logprobs,
                "logprobs_bwd": _plain_logprobs_bwd}[op](s)
    import sparse_ternary_bit_amd as stq
    if op == "swiglu":
        gu = torch.empty((s["rows"], 2 * s["d_ff"]), dtype=torch.bfloat16, device="cuda") if s["save"] else None
        h = stq.grouped_swiglu(s["table"], s["stride"], s["experts"], s["d_model"], s["d_ff"], s["x"], s["offsets"],
                               gate_up=gu)
        return (h, gu) if s["save"] else (h,)
    if op == "swiglu_bwd":
        dx, dw = stq.grouped_swiglu_backward(s["table"], s["stride"], s["experts"], s["d_model"], s["d_ff"], s["x"],
                                             s["offsets"], s["gate_up"], s["dh"], need_dw=s["dw"])
        return (dx, dw) if s["dw"] else (dx,)
    if op == "q8":
        q, scale = stq.q8_quantize_rows(s["x"])
        return stq.q8_matmul(q, scale, s["w"], s["w_scale"], out_dtype=DTYPES[s["out"]])
    if op == "logprobs":
        return stq.token_logprobs(s["logits"], s["targets"], top_n=s["top"])
    return stq.token_logprobs_backward(s["logits"], s["targets"], s["lse"], s["entropy"], s["g_logprob"], s["g_entropy"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _weights64(s, e):
    """Weights of expert e from the block format's bit rules, byte and bit positions worked out
    for every weight of a row block."""
    n, nb = 2 * s["d_ff"], s["d_model"] // QK
    dev = s["table"].device
    blocks = _expert(s, e).view(-1, BLOCK_BYTES)
    i = torch.arange(QK, device=dev)
    g, lane = i // 4, i % 4
    nib = blocks[:, 2 + 4 * (g >> 3) + (g & 3)].int() >> (4 * (g >> 2 & 1)).int() & 15
    sel = blocks[:, 34 + 4 * (g >> 5) + (g & 3)].int() >> (g >> 2 & 7).int() & 1
    code = nib + 16 * sel
    zero = code >> 3
    rank = lane.int() - (lane.int() > zero).int()
    value = torch.where(lane.int() == zero, 0, 1 - 2 * (code >> rank.clamp(min=0) & 1)).double()
    value *= blocks[:, :2].contiguous().view(torch.float16).double()
    return value.view(n // 64, nb, 64, QK).permute(0, 2, 1, 3).reshape(n, nb * QK)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    dev = "cuda"
    if op == "swiglu":
        f = c["d_ff"]
        z = torch.zeros((c["rows"], 2 * f), dtype=torch.float64, device=dev)
        for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if hi > lo:
                z[lo:hi] = torch.matmul(_weights64(s, e), s["x"][lo:hi].double().t()).t()
        h = z[:, :f] * torch.sigmoid(z[:, :f]) * z[:, f:]
        return (h, z) if c["save"] else (h,)
    if op == "swiglu_bwd":
        f, d = c["d_ff"], c["d_model"]
        g, u = s["gate_up"].double().split(f, 1)
        sig = torch.sigmoid(g)
        dh = s["dh"].double()
        dg = dh * u * (sig + g * sig * torch.sigmoid(-g))
        du = dh * (g * sig)
        dx = torch.zeros((c["rows"], d), dtype=torch.float64, device=dev)
        dw = torch.zeros((c["experts"], 2 * f, d), dtype=torch.float64, device=dev) if c["dw"] else None
        for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if hi == lo:
                continue
            w = _weights64(s, e)
            dx[lo:hi] = torch.matmul(dg[lo:hi], w[:f]) + torch.matmul(du[lo:hi], w[f:])
            if dw is not None:
                x = s["x"][lo:hi].double()
                dw[e, :f] = torch.matmul(dg[lo:hi].t().contiguous(), x)
                dw[e, f:] = torch.matmul(du[lo:hi].t().contiguous(), x)
        return (dx, dw) if c["dw"] else (dx,)
    if op == "q8":
        x = s["x"].double()
        scale = (x.abs().max(1).values / 127).float().double()
        q = torch.where(scale[:, None] > 0, torch.round(x / scale[:, None]), 0.0)
        w = s["w"].double() * s["w_scale"].double()[:, None]
        return torch.matmul(q * scale[:, None], w.t())
    rows, vocab = c["rows"], c["vocab"]
    row = torch.arange(rows, device=dev)
    if op == "logprobs":
        out = [torch.empty(rows, dtype=torch.float64, device=dev) for _ in range(3)]
        ids = torch.empty((rows, c["top"]), dtype=torch.int32, device=dev)
        top = torch.empty((rows, c["top"]), dtype=torch.float64, device=dev)
        for r in range(0, rows, 256):
            b = slice(r, min(rows, r + 256))
            l = s["logits"][b].double()
            lp = torch.log_softmax(l, 1)
            out[0][b] = lp.gather(1, s["targets"][b, None].long())[:, 0]
            out[1][b] = torch.logsumexp(l, 1)
            p = torch.exp(lp)
            out[2][b] = torch.special.entr(p).sum(1)
            if c["top"]:
                order = torch.sort(l, dim=1, descending=True, stable=True)
                ids[b] = order.indices[:, :c["top"]].int()
                top[b] = lp.gather(1, order.indices[:, :c["top"]])
        return out[0], out[1], out[2], ids, top
    d = torch.empty((rows, vocab), dtype=torch.float64, device=dev)
    for r in range(0, rows, 256):
        b = slice(r, min(rows, r + 256))
        p = torch.exp(s["logits"][b].double() - s["lse"][b].double()[:, None])
        ent = torch.special.xlogy(p, p) + p * s["entropy"][b].double()[:, None]
        d[b] = -s["g_logprob"][b].double()[:, None] * p - s["g_entropy"][b].double()[:, None] * ent
    d[row, s["targets"].long()] += s["g_logprob"].double()
    return d
