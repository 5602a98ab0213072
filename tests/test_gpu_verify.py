"""moe_int4_verify_drafts on the GPU against its definition in 64 bits: tokens
and counts are whole numbers and have to be equal.

The kernels' probabilities and sums are within 2^-40 of the definition's; a pick
falls that close to one of 248320 borders with a probability below 10^-6, and the
inputs here are fixed, so equality is what is tested."""
import math
import sys

import numpy as np
import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import DraftVerifier, LogitsRules

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.lib()
    yield


def softmax(l):
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    e = np.exp(np.where(l == top, 0.0, l - top)) if np.isfinite(top) else (l == top).astype(np.float64)
    return e / e.sum()


def definition(target, draft, drafted, lengths, coins, picks, temperature, width, vocab):
    seqs = len(picks)
    tokens, accepted = np.full((seqs, width + 1), -1, np.int32), np.zeros(seqs, np.int32)
    for b in range(seqs):
        n, drafts = 0, width if lengths is None else min(max(int(lengths[b]), 0), width)
        greedy = temperature is not None and not temperature[b] > 0
        while True:
            row = target[b * (width + 1) + n]
            p = softmax(row)
            x = int(drafted[b, n]) if n < drafts else -1
            if greedy:
                clean = np.where(np.isnan(row), -np.inf, row)
                best = int(clean.argmax()) if clean.max() > -np.inf else -1
                if n < drafts and best >= 0 and x == best:
                    tokens[b, n], n = x, n + 1
                    continue
                tokens[b, n] = best
                break
            q = np.zeros(vocab)
            if n < drafts:
                if draft is not None:
                    q = softmax(draft[b * width + n])
                elif 0 <= x < vocab:
                    q[x] = 1.0
                if 0 <= x < vocab and float(coins[b, n]) * q[x] < p[x]:
                    tokens[b, n], n = x, n + 1
                    continue
            r = np.maximum(p - q, 0.0)
            c = np.cumsum(r if r.sum() > 0 else p)
            if c[-1] > 0:
                tokens[b, n] = int(np.searchsorted(c, float(picks[b]) * c[-1], side="right"))
            break
        accepted[b] = n
    return tokens, accepted


def host(t):
    if t is None:
        return None
    return t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def case(seqs, width, vocab, tt="fp32", dt="fp32", seed=0, noise=0.4, spread=2.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def uniform(*s):
        return torch.rand(*s, device="cuda", generator=g)

    target = torch.randn(seqs, width + 1, vocab, device="cuda", generator=g) * spread
    draft = target[:, :width] + noise * torch.randn(seqs, width, vocab, device="cuda", generator=g)
    gumbel = -torch.log(-torch.log(uniform(seqs, width, vocab).clamp(1e-9, 1 - 1e-7)))
    d = {"drafted": (draft + gumbel).argmax(2).to(torch.int32) if width else
         torch.zeros(seqs, 0, dtype=torch.int32, device="cuda")}
    d["target"] = target.view(-1, vocab).to(TYPES[tt])
    d["draft"] = draft.reshape(-1, vocab).to(TYPES[dt]) if dt else None
    d["coins"], d["picks"] = uniform(seqs, width), uniform(seqs)
    d["lengths"], d["temperature"] = None, None
    return d


def verify(d, vocab, what=""):
    width = d["drafted"].shape[1]
    tokens, accepted = DraftVerifier(vocab, temperature=d["temperature"]).verify(
        d["target"], d["drafted"], d["coins"], d["picks"], draft=d["draft"], lengths=d["lengths"])
    want = definition(*(host(d[k]) for k in ("target", "draft", "drafted", "lengths", "coins", "picks", "temperature")),
                      width, vocab)
    assert np.array_equal(host(accepted), want[1]), what
    assert np.array_equal(host(tokens), want[0]), what
    return want


@pytest.mark.parametrize("tt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dt", [None, "bf16", "fp16", "fp32"])
@pytest.mark.parametrize("seqs,width,vocab", [(1, 1, 1), (3, 2, 7), (2, 4, 1000), (5, 3, 8192), (9, 8, 8193), (40, 1, 33)])
def test_against_definition(seqs, width, vocab, tt, dt):
    say(f"seqs={seqs} width={width} vocab={vocab} {tt} {dt}")
    for seed in range(3):
        verify(case(seqs, width, vocab, tt, dt, seed), vocab)


@pytest.mark.parametrize("seqs,width,vocab,tt,dt", [(1, 3, 248320, "fp32", "bf16"), (3, 2, 151937, "bf16", "fp32"),
                                                   (2, 0, 248320, "fp16", None), (1, 1, 1000003, "fp32", "fp32"),
                                                   (20, 7, 32003, "fp16", None)])
def test_large_vocabularies(seqs, width, vocab, tt, dt):
    say(f"seqs={seqs} width={width} vocab={vocab}")
    for seed in range(2):
        verify(case(seqs, width, vocab, tt, dt, seed), vocab)


def test_flat_rows_and_many_picks():
    """Rows of nearly equal probabilities, whose borders lie close: every pick's own token."""
    for vocab in (50257, 248320):
        verify(case(48, 0, vocab, seed=3, spread=0.01), vocab)
        verify(case(24, 1, vocab, seed=4, spread=0.5, noise=0.05), vocab)


def test_widest_and_many_sequences():
    verify(case(4, 64, 1001, "bf16", "bf16", noise=0.01), 1001)
    verify(case(3000, 2, 50, "fp32", "bf16"), 50)


def test_lengths_and_greedy():
    d = case(64, 5, 3001, "fp32", "bf16", seed=7)
    d["lengths"] = torch.randint(-2, 8, (64,), device="cuda").to(torch.int32)
    d["temperature"] = torch.ones(64, device="cuda")
    d["temperature"][::3], d["temperature"][1::6], d["temperature"][2] = 0.0, -1.0, math.nan
    best = d["target"].view(64, 6, 3001)[:, :5].argmax(2).to(torch.int32)
    d["drafted"][::3, :3] = best[::3, :3]
    d["drafted"][6] = best[6]
    want = verify(d, 3001)
    assert want[1].max() >= 3


def test_ties_go_to_the_first():
    vocab = 20000
    d = case(4, 2, vocab, "bf16", None, seed=1)
    d["temperature"] = torch.zeros(4, device="cuda")
    t = d["target"].view(4, 3, vocab)
    t[:, :, 17000] = 30.0
    t[:, :, 9001] = 30.0
    t[2, 0, 12] = 30.0
    d["drafted"][:] = 9001
    want = verify(d, vocab)
    assert want[1].tolist() == [2, 2, 0, 2] and want[0][2, 0] == 12


@pytest.mark.parametrize("greedy", [False, True])
def test_masked_rows(greedy):
    """Rows that leave nothing, one token, or few; NaN; +infinities."""
    vocab = 9000
    d = case(12, 2, vocab, "fp32", "fp32", seed=2)
    t, q = d["target"].view(12, 3, vocab), d["draft"].view(12, 2, vocab)
    inf = math.inf
    t[0] = -inf                                     # nothing anywhere
    t[1, 1:] = -inf                                 # nothing behind the first draft
    t[2, :, :8999] = -inf                           # the last token alone
    t[3, :, 1:] = -inf                              # the first token alone
    q[4] = -inf                                     # a draft head that allows nothing
    t[5, :, ::2] = math.nan
    t[6, 0, 500], t[6, 0, 8500] = inf, inf
    q[7, 0, 31] = inf
    t[8] = torch.finfo(torch.float32).min           # the type's lowest value everywhere: equal logits
    t[9, :, 5000:] = -inf
    q[9, :, :5000] = -inf                           # target and draft share no token
    d["drafted"][2], d["drafted"][3] = 8999, 0
    d["drafted"][10], d["drafted"][11, 0] = -1, vocab   # ids outside the vocabulary
    t[11, 0, :] = q[11, 0, :]
    if greedy:
        d["temperature"] = torch.zeros(12, device="cuda")
    want = verify(d, vocab)
    assert want[0][0].tolist() == [-1, -1, -1]
    d["draft"] = None
    verify(d, vocab)


def test_extreme_random_numbers():
    vocab = 5000
    for coin, pick in ((0.0, 0.0), (1 - 2 ** -24, 1 - 2 ** -24), (0.5, 2 ** -126)):
        d = case(16, 3, vocab, seed=5)
        d["coins"].fill_(coin)
        d["picks"].fill_(pick)
        verify(d, vocab, (coin, pick))
        # equal distributions: everything is accepted
        d["draft"] = d["target"].view(16, 4, vocab)[:, :3].reshape(-1, vocab).contiguous()
        want = verify(d, vocab)
        assert (want[1] == 3).all()


def test_strides_and_alignment():
    """Rows inside wider ones, at addresses that share no aligned word."""
    for extra, off in ((29, 0), (8, 1), (3, 3)):
        for tt, dt in (("fp16", "bf16"), ("fp32", "fp16"), ("bf16", None)):
            d = case(6, 3, 9001, tt, dt, seed=6)
            want = verify(d, 9001)
            for k in ("target", "draft"):
                if d[k] is not None:
                    w = torch.full((d[k].shape[0], 9001 + extra + off), math.nan, dtype=d[k].dtype, device="cuda")
                    w[:, off:off + 9001] = d[k]
                    d[k] = w[:, off:off + 9001]
            again = verify(d, 9001)
            assert np.array_equal(again[0], want[0])


def test_distribution_of_tokens():
    """Over many random numbers the answered token follows the target's
    probabilities, whatever the draft's are: with n sequences a share is within
    five standard deviations, 5 sqrt(p (1 - p) / n)."""
    n, vocab = 60000, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    t = torch.tensor([1.0, 0.0, -1.0, 2.0, -math.inf, 0.5], device="cuda")
    q = torch.tensor([0.0, 1.0, 1.0, -1.0, 0.0, 0.0], device="cuda")
    target = t.expand(n, 2, vocab).reshape(-1, vocab).contiguous()
    draft = q.expand(n, vocab).contiguous()
    drafted = torch.multinomial(torch.softmax(q, 0), n, replacement=True, generator=g).to(torch.int32).view(n, 1)
    tokens, accepted = DraftVerifier(vocab).verify(target, drafted, torch.rand(n, 1, device="cuda", generator=g),
                                                   torch.rand(n, device="cuda", generator=g), draft=draft)
    p = torch.softmax(t.double(), 0).cpu()
    share = torch.bincount(tokens[:, 0].long(), minlength=vocab).double().cpu() / n
    assert ((share - p).abs() <= 5 * (p * (1 - p) / n).sqrt() + 1e-12).all(), (share, p)
    behind = tokens[accepted == 1, 1].long()
    share = torch.bincount(behind, minlength=vocab).double().cpu() / behind.numel()
    assert ((share - p).abs() <= 5 * (p * (1 - p) / behind.numel()).sqrt() + 1e-12).all()


def test_behind_the_rules():
    """Logits through LogitsRules, target and draft alike, then the verification."""
    seqs, width, vocab = 6, 3, 4000
    d = case(seqs, width, vocab, "bf16", "bf16", seed=9)
    temperature = torch.tensor([0.7, 0.0, 1.0, 1.3, 0.0, 0.2], device="cuda")
    mask = torch.full((seqs, (vocab + 31) // 32), -1, dtype=torch.int32, device="cuda")
    mask[2, 10:] = 0
    mask[4] = 0

    def rules(rows):
        return LogitsRules(vocab, temperature=temperature.repeat_interleave(rows),
                           mask=mask.repeat_interleave(rows, 0).contiguous())

    d["target"] = rules(width + 1).apply(d["target"])
    d["draft"] = rules(width).apply(d["draft"])
    d["temperature"] = temperature
    want = verify(d, vocab)
    assert want[0][4].tolist() == [-1] * (width + 1)


def test_repeated_and_captured():
    vocab = 30000
    d = case(10, 3, vocab, "fp32", "bf16", seed=12)
    v = DraftVerifier(vocab)
    tokens = torch.empty(10, 4, dtype=torch.int32, device="cuda")
    accepted = torch.empty(10, dtype=torch.int32, device="cuda")

    def call():
        v.verify(d["target"], d["drafted"], d["coins"], d["picks"], draft=d["draft"], tokens=tokens, accepted=accepted)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        other = case(10, 3, vocab, "fp32", "bf16", seed=20 + i)
        for k in ("target", "draft", "drafted", "coins", "picks"):
            d[k].copy_(other[k])
        want = verify(d, vocab)
        tokens.fill_(5), accepted.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(tokens), want[0]) and np.array_equal(host(accepted), want[1]), f"replay {i}"


def test_two_streams():
    vocab = 60000
    ds = [case(6, 3, vocab, "fp32", "bf16", seed=30 + i) for i in range(2)]
    want = [verify(d, vocab) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    v = DraftVerifier(vocab)
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                d = ds[i]
                got.append((i, v.verify(d["target"], d["drafted"], d["coins"], d["picks"], draft=d["draft"])))
    torch.cuda.synchronize()
    for i, (tokens, accepted) in got:
        assert np.array_equal(host(tokens), want[i][0]) and np.array_equal(host(accepted), want[i][1])
