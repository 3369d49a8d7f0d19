"""The operators of a prompt pass as a program strings them together: routed
rows through the gated feed-forward and the packed down projection, the
combined tokens through an 8-bit head, scored, and the gradient back to the
experts' inputs and weights.  Every stage is held against 64-bit arithmetic
on the inputs it was given (the bounds of the stages' own tests; the down
product's is 2e-3 of the sum of its products' magnitudes), and the whole
sequence, captured into one graph, has to repeat the eager bits."""
import numpy as np
import pytest
import torch

import test_gpu_logprobs as TL
import test_gpu_q8 as TQ
import test_gpu_swiglu as TS
import synth_inputs as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_ternary_bit_amd as m
    return m


class Pass:
    """One layer and head: T tokens, top_k of E experts each, a vocabulary of odd size."""

    def __init__(self, stq, T, E, top_k, d, f, vocab, seed):
        self.stq, self.T, self.E, self.d, self.f = stq, T, E, d, f
        row_token, offsets = S.prefill_routing(seed, T, E, top_k)
        counts = np.diff(offsets)
        self.c = TS.Case(stq, counts, d, f, seed=seed)
        self.down = TS.Case(stq, counts, f, d // 2, seed=seed + 1)       # packed [d, f] matrices
        g = torch.Generator().manual_seed(seed)
        self.tokens = torch.randn((T, d), generator=g).bfloat16().cuda()
        self.row_token = torch.from_numpy(row_token).cuda()
        self.weight = torch.softmax(torch.randn((T * top_k,), generator=g), 0).cuda() * T
        self.head, self.head_scale = stq.q8_quantize_rows((torch.randn((vocab, d), generator=g) * 0.05).cuda())
        self.head_f = self.head.float() * self.head_scale[:, None]
        self.targets = torch.randint(0, vocab, (T,), generator=g, dtype=torch.int32).cuda()
        self.g = torch.randn(T, generator=g).cuda()
        self.down_w = torch.stack([self.down.weights(e) for e in range(E)]).float()
        # rows of the same expert share its matrix in the torch steps between the operators
        self.row_expert = torch.repeat_interleave(torch.arange(E), torch.from_numpy(counts.astype(np.int64))).cuda()
        self.top_k = top_k
        order = torch.argsort(self.row_token, stable=True)
        self.token_rows = order.view(T, top_k)                            # the rows of every token

    def run(self):
        stq, c = self.stq, self.c
        c.x = self.tokens.index_select(0, self.row_token)
        gate_up = torch.empty((c.m, 2 * self.f), dtype=torch.bfloat16, device="cuda")
        h = c.forward(gate_up=gate_up)
        z = stq.grouped_gemm(self.down.table, self.down.stride, self.E, self.d, self.f, h, c.offsets)
        zw = z * self.weight[:, None]
        y = zw[self.token_rows[:, 0]]
        for k in range(1, self.top_k):
            y = y + zw[self.token_rows[:, k]]
        q, s = stq.q8_quantize_rows(y)
        logits = stq.q8_matmul(q, s, self.head, self.head_scale, out_dtype=torch.float32)
        scored = stq.token_logprobs(logits, self.targets, top_n=5)
        d_logits = stq.token_logprobs_backward(logits, self.targets, scored[1], scored[2], self.g, 0.01 * self.g)
        dy = d_logits @ self.head_f                                       # the head's rows as they were rounded
        dz = dy.index_select(0, self.row_token) * self.weight[:, None]
        dh = torch.empty((c.m, self.f), dtype=torch.bfloat16, device="cuda")
        for e in range(self.E):
            lo, hi = self.down.bounds[e], self.down.bounds[e + 1]
            if hi > lo:
                dh[lo:hi] = dz[lo:hi] @ self.down_w[e]
        c.gu, c.dh = gate_up, dh
        dx, dw = c.backward()
        return dict(x=c.x, gate_up=gate_up, h=h, z=z, y=y, q=q, s=s, logits=logits, scored=scored, d_logits=d_logits,
                    dh=dh, dx=dx, dw=dw)


@pytest.mark.parametrize("T, E, top_k, d, f", [(96, 6, 2, 512, 256), (1, 4, 2, 512, 256), (70, 3, 1, 1024, 512)])
def test_prompt_pass(stq, T, E, top_k, d, f):
    p = Pass(stq, T, E, top_k, d, f, 1003, seed=T)
    o = p.run()
    p.c.check_forward(o["h"], o["gate_up"])
    for e in range(E):
        lo, hi = p.down.bounds[e], p.down.bounds[e + 1]
        if hi > lo:
            w, h = p.down_w[e].double(), o["h"][lo:hi].double()
            ref, A = h @ w.t().contiguous(), h.abs() @ w.abs().t().contiguous()
            assert bool(((o["z"][lo:hi].double() - ref).abs() <= 2e-3 * A).all())
    want_q, want_s = TQ._quant_ref(o["y"].cpu())
    assert np.array_equal(o["q"].cpu().numpy(), want_q) and np.array_equal(o["s"].cpu().numpy(), want_s)
    TQ._check(o["logits"], o["q"].cpu(), o["s"].cpu(), p.head.cpu(), p.head_scale.cpu())
    logits = o["logits"].cpu()
    TL._check(o["scored"], logits, p.targets.cpu(), 5)
    d, tol = TL._backward_ref(logits, p.targets.cpu(), o["scored"][1].cpu(), o["scored"][2].cpu(), p.g.cpu(), 0.01 * p.g.cpu())
    assert bool(((o["d_logits"].cpu().double() - d).abs() <= tol + 2.0 ** -126).all())
    p.c.check_backward(o["dx"], o["dw"])


def test_prompt_pass_in_one_graph(stq):
    p = Pass(stq, 64, 5, 2, 512, 256, 1003, seed=3)
    p.run()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            got = p.run()
    torch.cuda.synchronize()
    names = ("h", "z", "logits", "d_logits", "dx", "dw")
    for r in range(4):
        p.tokens.copy_(torch.randn(p.tokens.shape, generator=torch.Generator().manual_seed(r)).bfloat16())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        first = {n: got[n].clone() for n in names}
        want = p.run()
        torch.cuda.synchronize()
        assert all(torch.equal(first[n], want[n]) for n in names), r


def test_readme_example(stq):
    """The README's prompt pass runs as it stands, and its gradients are those of its stages.

    dh is PyTorch's: an fp32 sum of d products, at most 2 u (d + 2) of their magnitudes off in any order, and
    its rounding to bf16; d_tokens an fp32 sum of a token's top_k rows."""
    import os
    import re
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        text = f.read()
    part = text[text.index("\nA prompt pass."):]
    blocks = re.findall(r"(?:^    .*\n)+", part, flags=re.M)[:2]
    assert "token_logprobs(" in blocks[0] and "grouped_swiglu_backward(" in blocks[1]
    T, E, d, f = 50, 5, 512, 256
    p = Pass(stq, T, E, 2, d, f, 1003, seed=23)
    names = dict(torch=torch, stq=stq, tokens=p.tokens, row_token=p.row_token.long(), row_weight=p.weight,
                 offsets=p.c.offsets, bounds=p.c.bounds, gate_up=p.c.table, gate_up_stride=p.c.stride,
                 down=p.down.table, down_stride=p.down.stride, experts=E, d_model=d, d_ff=f, head=p.head,
                 head_scale=p.head_scale, targets=p.targets, g=p.g)
    for b in blocks:
        exec("".join(line[4:] for line in b.splitlines(True)), names)
    logits = names["logits"].cpu()
    TL._check(tuple(names[n] for n in ("logprob", "lse", "entropy", "ids", "alternatives")), logits, p.targets.cpu(), 5)
    p.c.x, p.c.gu, p.c.dh = names["x"], names["gu"], names["dh"]
    p.c.check_forward(names["h"], names["gu"])
    dz = names["dz"].double()
    for e in range(E):
        lo, hi = p.c.bounds[e], p.c.bounds[e + 1]
        w = p.down_w[e].double()
        ref, A = dz[lo:hi] @ w, dz[lo:hi].abs() @ w.abs()
        assert bool(((names["dh"][lo:hi].double() - ref).abs() <= 2 * TS.U * (d + 2) * A * (1 + TS.B) + TS.B * ref.abs()).all())
    p.c.check_backward(names["dx"], names["dw"])
    rows = names["dx"].double()[p.token_rows]                            # [T, top_k, d]
    assert bool(((names["d_tokens"].double() - rows.sum(1)).abs() <= 2 * TS.U * rows.abs().sum(1)).all())
