"""A draft head's step as a program runs it: a projection (Int4Linear), its
experts one product at a time over the routing's tables (Int4GroupedLinear),
the vocabulary projection (Int4Linear, whose weights the library's quantizer
made), the rules on both heads' logits (LogitsRules), and the verification
(DraftVerifier); eagerly, against 64 bits, and captured as one graph.

Tolerance of the logits: every step rounds its output to bf16 (half a step,
2^-8 / 2 = 2^-9 relative to the value), and so does the plain form here, from
its own inputs; three roundings in a row (projection, experts' activation,
hidden state) and the kernels' fp32 sums leave a difference of at most 2^-9 of
each input's size, which a product of K terms turns into 2^-9 sqrt(sum w^2 x^2)
at one sigma: six sigma of three of them."""
import numpy as np
import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import DraftVerifier, Int4GroupedLinear, Int4Linear, LogitsRules, MoeInt4Layer
from test_gpu_int4_linear import generator, matrix64, weights
from test_gpu_verify import definition, host

pytestmark = pytest.mark.gpu

HIDDEN, EXPERTS, INTER, TOP_K, VOCAB, SEQS, WIDTH = 256, 16, 128, 4, 3001, 6, 3


class Head:
    def __init__(self, seed):
        g = generator(seed)
        self.proj = Int4Linear(*weights((HIDDEN,), HIDDEN, 128, g), 128)
        w13, s13 = weights((EXPERTS, 2 * INTER), HIDDEN, 128, g)
        w2, s2 = weights((EXPERTS, HIDDEN), INTER, 128, g)
        self.router = (torch.randn(EXPERTS, HIDDEN, device="cuda", generator=g) * 0.1).to(torch.bfloat16)
        self.layer = MoeInt4Layer({"router_w": self.router, "w13_packed": w13, "w13_scales": s13, "w2_packed": w2,
                                   "w2_scales": s2}, TOP_K)
        self.up, self.down = Int4GroupedLinear(w13, s13, 128), Int4GroupedLinear(w2, s2, 128)
        # the vocabulary projection: bf16 weights through the library's quantizer
        dense = (torch.randn(VOCAB, HIDDEN, device="cuda", generator=g) * 0.2).to(torch.bfloat16)
        packed = torch.empty(VOCAB, HIDDEN // 8, dtype=torch.int32, device="cuda")
        scales = torch.empty(VOCAB, HIDDEN // 128, dtype=torch.bfloat16, device="cuda")
        B.moe_int4_quantize(dense, VOCAB, HIDDEN, packed, scales)
        self.vocab = Int4Linear(packed, scales, 128)

    def logits(self, x):
        h = self.proj.forward(x, residual=x)
        r = self.layer.route(h)
        gate, lift = self.up.forward(h, r["offsets"], gather=r["sorted_slots"], gather_div=TOP_K,
                                     out_dtype=torch.float32).chunk(2, dim=1)
        a = (torch.nn.functional.silu(gate) * lift).to(torch.bfloat16)
        y = self.down.forward(a, r["offsets"], scatter=r["sorted_slots"], row_weights=r["weights"],
                              out_dtype=torch.float32)
        hidden = (h.float() + y.view(x.shape[0], TOP_K, HIDDEN).sum(1)).to(torch.bfloat16)
        return self.vocab.forward(hidden), (h, r)

    def plain(self, x, ids, w):
        """In 64 bits, rounded to bf16 where the step above rounds; the routing given."""
        def rounded(t):
            return t.to(torch.bfloat16).double()

        def product(t, layer, e=None):
            p, s = (layer.packed, layer.scales) if e is None else (layer.packed[e], layer.scales[e])
            return torch.mm(t, matrix64(p, s, 128).t().contiguous())

        h = rounded(product(x.double(), self.proj) + x.double())
        hidden = h.clone()
        for t in range(x.shape[0]):
            for j in range(TOP_K):
                e = int(ids[t, j])
                gate, lift = product(h[t:t + 1], self.up, e).chunk(2, dim=1)
                a = rounded(torch.nn.functional.silu(gate) * lift)
                hidden[t] += float(w[t, j]) * product(a, self.down, e)[0]
        hidden = rounded(hidden)
        spread = torch.mm(hidden.square(), matrix64(self.vocab.packed, self.vocab.scales, 128).square().t().contiguous()).sqrt()
        return product(hidden, self.vocab), spread


def step(target, draft, verifier, rules, xs, d):
    tl, _ = target.logits(xs[0])
    dl, _ = draft.logits(xs[1])
    tl, dl = rules[0].apply(tl), rules[1].apply(dl)
    tokens, accepted = verifier.verify(tl, d["drafted"], d["coins"], d["picks"], draft=dl, lengths=d["lengths"])
    return tl, dl, tokens, accepted


def inputs(seed):
    g = generator(seed)
    x = torch.randn(SEQS * (WIDTH + 1), HIDDEN, device="cuda", generator=g).to(torch.bfloat16)
    xd = x.view(SEQS, WIDTH + 1, HIDDEN)[:, :WIDTH].reshape(-1, HIDDEN).contiguous()
    d = {"drafted": torch.randint(0, VOCAB, (SEQS, WIDTH), device="cuda", generator=g).to(torch.int32),
         "coins": torch.rand(SEQS, WIDTH, device="cuda", generator=g), "picks": torch.rand(SEQS, device="cuda", generator=g),
         "lengths": torch.tensor([3, 2, 3, 0, 1, 3], dtype=torch.int32, device="cuda")}
    return (x, xd), d


def make():
    target, draft = Head(1), Head(1)   # a draft head of the target's own weights: half its drafts pass
    temperature = torch.tensor([0.8, 0.0, 1.0, 1.2, 0.0, 0.6], device="cuda")
    mask = torch.full((SEQS, (VOCAB + 31) // 32), -1, dtype=torch.int32, device="cuda")
    mask[2, 20:] = 0

    def rules(rows):
        return LogitsRules(VOCAB, temperature=temperature.repeat_interleave(rows),
                           mask=mask.repeat_interleave(rows, 0).contiguous())

    return target, draft, DraftVerifier(VOCAB, temperature=temperature), (rules(WIDTH + 1), rules(WIDTH)), temperature


def test_step_against_64_bits():
    target, draft, verifier, rules, temperature = make()
    xs, d = inputs(5)
    logits, (h, r) = target.logits(xs[0])
    want, spread = target.plain(xs[0], r["ids"], r["weights"])
    err = (logits.double() - want).abs()
    limit = 3 * 6 * 2.0 ** -9 * spread + 2.0 ** -9 * want.abs()
    assert (err <= limit).all(), (err / limit).max().item()
    # the greedy sequences draft what the target would say, the others what the draft head would
    best = rules[0].apply(logits).view(SEQS, WIDTH + 1, VOCAB)[:, :WIDTH].argmax(2).to(torch.int32)
    d["drafted"][1], d["drafted"][4], d["drafted"][0] = best[1], best[4], best[0]
    tl, dl, tokens, accepted = step(target, draft, verifier, rules, xs, d)
    t, a = definition(host(tl), host(dl), host(d["drafted"]), host(d["lengths"]), host(d["coins"]), host(d["picks"]),
                      host(temperature), WIDTH, VOCAB)
    assert np.array_equal(host(tokens), t) and np.array_equal(host(accepted), a)
    assert a[1] == 2 and a[4] == 1 and a[3] == 0


def test_step_as_one_graph():
    target, draft, verifier, rules, _ = make()
    xs, d = inputs(6)
    for _ in range(2):
        step(target, draft, verifier, rules, xs, d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(target, draft, verifier, rules, xs, d)
    for i in range(4):
        nx, nd = inputs(10 + i)
        for old, new in list(zip(xs, nx)) + [(d[k], nd[k]) for k in d]:
            old.copy_(new)
        want = [t.clone() for t in step(target, draft, verifier, rules, xs, d)]
        torch.cuda.synchronize()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(out, want):
            assert torch.equal(got, w), f"replay {i}"
