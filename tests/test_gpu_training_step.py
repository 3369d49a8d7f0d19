"""A training step of a layer and its head: norm rows, routing, the experts,
their combination, the head's loss, and back to the tokens, as the README
strings them together.  Every stage is held against 64-bit arithmetic on the
inputs it was given, with the bounds of the stage's own tests; the whole
sequence captured into one graph repeats the eager bits, the routing changing
from replay to replay."""
import os
import re

import pytest
import torch

import test_gpu_head as TH
import test_gpu_norm as TN
import test_gpu_route as TR
import test_gpu_swiglu as TS

pytestmark = pytest.mark.gpu
D, F, VOCAB = 512, 256, 1003


@pytest.fixture(scope="module")
def stq():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import sparse_ternary_bit_amd as m
    return m


class Step:
    """The names that the README's two blocks use."""

    def __init__(self, stq, T, E, top_k, seed):
        self.stq, self.T, self.E, self.k = stq, T, E, top_k
        g = torch.Generator().manual_seed(seed)
        self.randn = lambda *s: torch.randn(s, generator=g)
        self.gate_up, self.down = TS.Case(stq, [1] * E, D, F, seed=seed), TS.Case(stq, [1] * E, F, D // 2, seed=seed + 1)
        head, head_scale = stq.q8_quantize_rows((self.randn(VOCAB, D) * 0.05).cuda())
        targets = torch.randint(-1, VOCAB, (T,), generator=g, dtype=torch.int32).cuda()
        self.names = dict(
            torch=torch, stq=stq, tokens=self.randn(T, D).bfloat16().cuda(), residual=(3 * self.randn(T, D)).bfloat16().cuda(),
            w1=(1 + 0.1 * self.randn(D)).cuda(), w2=(1 + 0.1 * self.randn(D)).cuda(),
            router=(self.randn(E, D) * 0.1).bfloat16().cuda(), top_k=top_k, experts=E, d_model=D, d_ff=F,
            gate_up=self.gate_up.table, gate_up_stride=self.gate_up.stride, down=self.down.table, down_stride=self.down.stride,
            head=head, head_scale=head_scale, targets=targets, g=(self.randn(T) / T).cuda(),
            g_balance=torch.full((1,), 0.02, device="cuda"))
        self.down_w = torch.stack([self.down.weights(e) for e in range(E)])

    def check(self, o):
        T, k, a, b, route = self.T, self.k, o["a"], o["b"], o["route"]
        TN._check(a, o["tokens"].cpu(), o["residual"].cpu(), o["w1"].cpu())
        ref = TR._check(route, o["logits"].cpu(), k, True)
        c = self.gate_up
        c.bounds = [int(v) for v in ref["offsets"]]
        c.m, c.x, c.offsets, c.gu, c.dh = T * k, o["x"], route.offsets, o["gu"], o["dh"]
        assert torch.equal(o["x"], a.y[ref["token"].cuda()])
        c.check_forward(o["h"], o["gu"])
        for e, (lo, hi) in enumerate(zip(c.bounds, c.bounds[1:])):
            w, h, dz = self.down_w[e], o["h"][lo:hi].double(), o["dz"][lo:hi].double()
            assert bool(((o["z"][lo:hi].double() - h @ w.t().contiguous()).abs() <= 2e-3 * (h.abs() @ w.abs().t().contiguous())).all())
            want, A = dz @ w, dz.abs() @ w.abs()
            assert bool(((o["dh"][lo:hi].double() - want).abs() <= 2 * TS.U * (D + 2) * A * (1 + TS.B) + TS.B * want.abs()).all())
        y, tol = TR._combine_ref(o["z"].cpu(), route.pair_row.cpu(), route.pair_weight.cpu(), k, torch.float32)
        assert bool(((o["y"].cpu().double() - y).abs() <= tol).all())
        TN._check(b, o["y"].cpu(), a.h.cpu(), o["w2"].cpu())
        head = TH.Case.__new__(TH.Case)
        head.n, head.v, head.k, head.i8 = T, VOCAB, D, True
        head.x, head.w, head.targets, head.grad = b.q, o["head"], o["targets"], o["g"]
        head.x_scale, head.w_scale = b.scale, o["head_scale"]
        head.check_forward(o["loss"], o["lse"])
        head.check_backward(o["d_rows"], None, o["lse"])
        cpu = lambda *names: [t.cpu() for t in names]  # noqa: E731
        TN._bwd_check((o["d_y"], o["d_w2"]), cpu(b.h, o["w2"], b.rstd, o["d_rows"]) + [None])
        row, share = ref["row"], o["d_y"].cpu().double().repeat_interleave(k, 0)
        on = row >= 0
        dz = share[on] * route.pair_weight.cpu().double()[on, None]
        assert bool(((o["dz"].cpu().double()[row[on]] - dz).abs() <= TR.U * dz.abs() + TR.TINY).all())
        terms = torch.zeros(T * k, D, dtype=torch.float64)
        terms[on] = share[on] * o["z"].cpu().double()[row[on]]
        tol = (8 * -(-D // 512) + 24) * TR.U * terms.abs().sum(1) + TR.TINY
        assert bool(((o["d_weight"].cpu().double() - terms.sum(1)).abs() <= tol).all())
        c.check_backward(o["dx"], o["dw"])
        d, tol = TR._bwd_ref(o["logits"].cpu(), k, True, ref, o["d_weight"].cpu().double().view(T, k), float(o["g_balance"].item()))
        assert bool(((o["d_logits"].cpu().double() - d).abs() <= tol).all())
        TN._bwd_check((o["d_tokens"], o["d_w1"]), cpu(a.h, o["w1"], a.rstd, o["d_a"], o["d_y"]))


def _blocks():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        text = f.read()
    blocks = re.findall(r"(?:^    .*\n)+", text[text.index("A training step of one layer"):], flags=re.M)[:2]
    assert "head_cross_entropy(" in blocks[0] and "route_tokens_backward(" in blocks[1]
    return ["".join(line[4:] for line in b.splitlines(True)) for b in blocks]


@pytest.mark.parametrize("T, E, top_k", [(50, 5, 2), (1, 4, 3), (200, 9, 4)])
def test_readme_example(stq, T, E, top_k):
    s = Step(stq, T, E, top_k, seed=T)
    o = dict(s.names)
    for b in _blocks():
        exec(b, o)
    s.check(o)


def test_gradient_against_differences(stq):
    """The whole step's derivative along its own gradient, against the difference of its own loss.

    The roundings to bf16 and 8 bits make the loss a staircase, so the step is long (a tenth of the tokens' norm) and
    the comparison loose: it says that no stage's gradient is missing or of the wrong sign, the stages' own tests say
    the rest."""
    s = Step(stq, 40, 4, 4, seed=5)      # every expert is chosen: the choice cannot change
    s.names["targets"].clamp_(min=0)
    forward, backward = _blocks()
    o = dict(s.names)
    for b in (forward, backward):
        exec(b, o)

    def loss(delta):
        p = dict(s.names, tokens=(s.names["tokens"].float() + delta).bfloat16())
        exec(forward, p)
        return (p["loss"].double() @ p["g"].double()).item()
    # uphill along the gradient itself: what the difference has to show is |gradient|^2
    d = o["d_tokens"].float()
    d *= 0.1 * s.names["tokens"].float().norm() / d.norm()
    got = loss(d) - loss(-d)
    want = 2 * (o["d_tokens"].double() * d.double()).sum().item()
    assert 0.5 * want < got < 1.5 * want, (got, want)


def test_step_in_one_graph(stq):
    """Replays with other tokens, and so another routing, repeat the eager bits."""
    s = Step(stq, 70, 6, 2, seed=8)
    forward, backward = _blocks()
    # bounds on the host are the program's own: here every expert's gradient takes all rows, masked
    loop = backward[backward.index("bounds ="):backward.index("dx, dw =")]
    backward = backward.replace(loop, "dh.copy_((dz @ w_all.view(d_model, -1)).view(len(dz), experts, d_ff)[rows, row_expert(route)])\n")
    names = dict(s.names, w_all=s.down_w.float().permute(1, 0, 2).contiguous(), rows=torch.arange(140, device="cuda"),
                 row_expert=lambda r: (torch.arange(140, device="cuda")[:, None] >= r.offsets[1:-1]).sum(1))
    exec(forward, names)
    exec(backward, names)
    torch.cuda.synchronize()
    side, graph, o = torch.cuda.Stream(), torch.cuda.CUDAGraph(), dict(names)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            exec(forward, o)
            exec(backward, o)
    torch.cuda.synchronize()
    keys = ("loss", "lse", "d_rows", "d_y", "d_w2", "dz", "d_weight", "d_logits", "d_tokens", "d_w1")
    seen = set()
    for r in range(4):
        names["tokens"].copy_(torch.randn((70, D), generator=torch.Generator().manual_seed(r)).bfloat16())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        first = {n: o[n].clone() for n in keys}
        seen.add(tuple(o["route"].counts.tolist()))
        again = dict(names)
        exec(forward, again)
        exec(backward, again)
        torch.cuda.synchronize()
        assert torch.equal(o["route"].pair_row, again["route"].pair_row)
        for n in keys:
            assert torch.equal(first[n], again[n]), (r, n)
    assert len(seen) > 1
