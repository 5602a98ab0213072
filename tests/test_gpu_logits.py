"""moe_int4_logits_process on the GPU against the rules written out in fp64,
row by row and token by token.

Tolerance, from the arithmetic (u = 2^-24, half a step of fp32): the rules are
at most a quotient or product, a product and two sums, one sum and one
quotient, so at most eight roundings, each of a value no larger than the sum
of the operands' magnitudes M (the division by the temperature scales both);
the store rounds once more, by half a step of the output's type.  -inf, +inf
and NaN have to come out where the definition has them."""
import math
import sys

import numpy as np
import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd import synth
from quantized_moe_router_amd.layer import Int8Linear, LogitsRules

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FILL = 55.0


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.lib()
    yield


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def expected(logits, rules):
    """(fp64 values, magnitudes M) of the rules given as LogitsRules' arguments."""
    y = host(logits).copy()
    m = np.abs(y)
    rows, vocab = y.shape
    r = {k: host(v) for k, v in rules.items() if v is not None}
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(rows):
            if "history" in r:
                width = r["history"].shape[1]
                n = int(np.clip(r["history_lengths"][i], 0, width)) if "history_lengths" in r else width
                p = int(np.clip(r["prompt_lengths"][i], 0, n)) if "prompt_lengths" in r else 0
                h = r["history"][i, :n].astype(np.int64)
                seen = np.unique(h[(h >= 0) & (h < vocab)])
                rep = r["repetition"][i] if "repetition" in r else 1.0
                y[i, seen] = np.where(y[i, seen] > 0, y[i, seen] / rep, y[i, seen] * rep)
                m[i, seen] = m[i, seen] * max(rep, 1 / rep, 1)
                a = h[p:]
                ids, c = np.unique(a[(a >= 0) & (a < vocab)], return_counts=True)
                f = r["frequency"][i] if "frequency" in r else 0.0
                q = r["presence"][i] if "presence" in r else 0.0
                y[i, ids] -= f * c + q
                m[i, ids] += np.abs(f * c) + abs(q)
            if "bias_ids" in r:
                width = r["bias_ids"].shape[1]
                n = int(np.clip(r["bias_lengths"][i], 0, width)) if "bias_lengths" in r else width
                last = {int(v): r["bias_values"][i, j] for j, v in enumerate(r["bias_ids"][i, :n]) if 0 <= v < vocab}
                for v, b in last.items():
                    y[i, v] += b
                    m[i, v] += abs(b)
            if "temperature" in r and r["temperature"][i] > 0:
                y[i] /= r["temperature"][i]
                m[i] /= r["temperature"][i]
            if "mask" in r:
                mask = r["mask"] if r["mask"].ndim == 2 else r["mask"][None]
                bits = np.unpackbits(mask[i if len(mask) > 1 else 0].view(np.uint8), bitorder="little")[:vocab]
                y[i, bits == 0] = -np.inf
    return y, m


def check(got, want, m, label):
    dtype = got.dtype
    g = host(got)
    f = torch.finfo(dtype)
    with np.errstate(invalid="ignore"):
        # beyond the type's largest value (plus half its step) a store gives infinity
        want = np.where(np.abs(want) >= f.max * (1 + f.eps / 4), np.sign(want) * np.inf, want)
        fine = np.isfinite(want)
        assert np.array_equal(np.isnan(g), np.isnan(want)), f"{label}: NaN elsewhere"
        odd = ~fine & ~np.isnan(want)
        assert np.array_equal(g[odd], want[odd]), f"{label}: infinities differ"
        err = 8 * U * np.where(fine, m, 0)
        o = np.abs(np.where(fine, want, 0)) + err
        bound = err + np.exp2(np.floor(np.log2(np.maximum(o, f.tiny)))) * f.eps / 2
        off = np.abs(np.where(fine, g, 0) - np.where(fine, want, 0))
    bad = np.argwhere(off > bound)
    assert bad.size == 0, (f"{label}: {len(bad)} of {off.size} off, first {bad[0].tolist()}: "
                           f"{g[tuple(bad[0])]} for {want[tuple(bad[0])]} +- {bound[tuple(bad[0])]}")


def inside(t, extra, fill):
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide, wide[:, :t.shape[1]]


def make(rows, vocab, width, biases, mask, seed, strided=False, in_type="bf16", repeats=1.0):
    """Logits and rules.  Lengths run from none to more than the width, ids
    from below zero to beyond the vocabulary, biased tokens come twice."""
    rng = np.random.default_rng(seed)
    logits = torch.from_numpy(rng.standard_normal((rows, vocab)) * 3).to(TYPES[in_type]).cuda()
    c32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    cf = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()  # noqa: E731
    u = {}
    if width:
        ids = (rng.random((rows, width)) ** (2 * repeats) * vocab).astype(np.int64)
        ids[rng.random((rows, width)) < 0.05] = -1
        ids[rng.random((rows, width)) < 0.05] = vocab
        ids[rng.random((rows, width)) < 0.01] = 2**31 - 1
        u["history"] = c32(ids)
        n = rng.integers(0, width + 1, rows)
        n[0] = width
        n[1::5] = 0
        n[2::5] = 1
        n[3::7] = width + 9      # taken as the width
        n[4::9] = -3             # taken as none
        u["history_lengths"] = c32(n)
        u["prompt_lengths"] = c32(rng.integers(-1, width + 5, rows))
        u["repetition"] = cf(rng.uniform(0.7, 1.6, rows))
        u["frequency"] = cf(rng.uniform(-0.5, 1, rows))
        u["presence"] = cf(rng.uniform(-0.5, 1, rows))
    if biases:
        ids = rng.integers(-2, vocab + 2, (rows, biases))
        ids[:, -1] = ids[:, 0]   # the first id again: the last entry holds
        u["bias_ids"] = c32(ids)
        u["bias_values"] = cf(rng.standard_normal((rows, biases)) * 4)
        u["bias_values"][:, 1::4] = -math.inf
        n = rng.integers(0, biases + 3, rows)
        n[0] = biases
        u["bias_lengths"] = c32(n)
    t = rng.uniform(0.3, 2, rows)
    t[1::3] = 0
    t[2::7] = -1
    u["temperature"] = cf(t)
    if mask:
        words = (vocab + 31) // 32
        w = rng.integers(-2**31, 2**31, (rows, words))
        w[rng.random((rows, words)) < 0.6] = 0
        w[1::4] = -1
        w[3::4] = 0              # nothing left
        u["mask"] = c32(w)
    if strided:
        logits = inside(logits, 13, math.nan)[1]
        for k in ("history", "mask"):
            if k in u:
                u[k] = inside(u[k], 3, 1)[1]
        if biases:
            u["bias_ids"], u["bias_values"] = inside(u["bias_ids"], 5, 0)[1], inside(u["bias_values"], 5, 1e9)[1]
    return logits, u


CASES = [
    # (rows, vocab, history width, biases, mask, in, out, strided)
    (1, 1, 1, 1, True, "fp32", "fp32", False),
    (1, 7, 0, 0, True, "bf16", "fp32", False),
    (2, 31, 3, 2, True, "fp16", "bf16", False),
    (3, 32, 40, 0, True, "bf16", "bf16", True),
    (5, 33, 1, 5, False, "fp32", "fp16", True),
    (4, 1000, 0, 0, False, "bf16", "fp32", False),
    (8, 8191, 300, 20, True, "bf16", "fp32", True),
    (8, 8192, 1023, 64, True, "fp16", "fp32", False),
    (8, 8193, 1024, 64, True, "fp32", "fp32", False),
    (9, 20000, 1025, 0, True, "bf16", "bf16", False),
    (17, 32003, 700, 40, True, "fp16", "fp16", True),
    (6, 50001, 5000, 300, False, "fp32", "bf16", False),
    (33, 16384, 64, 7, True, "bf16", "fp16", False),
    (3, 248320, 2000, 100, True, "bf16", "fp32", False),
    (2, 248320, 1, 0, False, "fp32", "fp32", True),
]


@pytest.mark.parametrize("rows,vocab,width,biases,mask,tin,tout,strided", CASES)
def test_rules_small(rows, vocab, width, biases, mask, tin, tout, strided):
    label = f"rules {rows}x{vocab} history {width} biases {biases} mask {mask} {tin}->{tout} {strided}"
    say(label)
    logits, u = make(rows, vocab, width, biases, mask, rows + vocab, strided, tin)
    out = torch.full((rows, vocab), FILL, dtype=TYPES[tout], device="cuda")
    wide = None
    if strided:
        wide, out = inside(out, 9, FILL)
    LogitsRules(vocab, **u).apply(logits, out=out)
    torch.cuda.synchronize()
    check(out, *expected(logits, u), label)
    if strided:
        assert bool((wide[:, vocab:] == FILL).all())


@pytest.mark.parametrize("keep", [("history", "repetition"), ("history", "frequency"), ("history", "presence"),
                                  ("history", "history_lengths", "prompt_lengths", "repetition", "presence"),
                                  ("bias_ids", "bias_values"), ("bias_ids", "bias_values", "bias_lengths"),
                                  ("temperature",), ("mask",), ()])
@pytest.mark.parametrize("rows", [1, 6])
def test_rules_each_alone(keep, rows):
    say(f"only {keep}, {rows} rows")
    logits, u = make(rows, 9001, 500, 30, True, 3)
    u = {k: v for k, v in u.items() if k in keep}
    out = LogitsRules(9001, **u).apply(logits)
    torch.cuda.synchronize()
    check(out, *expected(logits, u), f"only {keep}")


@pytest.mark.parametrize("rows,vocab", [(1, 500), (5, 20000)])
def test_rules_one_token_throughout(rows, vocab):
    # a row that says one token again and again: one counter takes them all
    say(f"one token {rows}x{vocab}")
    logits, u = make(rows, vocab, 60000, 0, False, 8)
    u["history"].fill_(vocab - 1)
    u["prompt_lengths"].fill_(17)
    out = LogitsRules(vocab, **u).apply(logits)
    torch.cuda.synchronize()
    check(out, *expected(logits, u), "one token")


@pytest.mark.parametrize("rows,width", [(1, 131072), (2, 262144), (40, 20011)])
def test_rules_long_history(rows, width):
    say(f"long history {rows} x {width}")
    vocab = 40000
    logits, u = make(rows, vocab, width, 10, True, width)
    out = LogitsRules(vocab, **u).apply(logits)
    torch.cuda.synchronize()
    check(out, *expected(logits, u), f"{rows} x {width}")


@pytest.mark.parametrize("rows,vocab,tin,tout", [(5, 30000, "fp32", "fp32"), (8, 30000, "bf16", "bf16"),
                                                 (9, 300000, "fp32", "fp32"), (9, 300000, "fp16", "fp16")])
def test_rules_long_history_edges(rows, vocab, tin, tout):
    # lengths and prompts that end at, before and behind whole runs of 16384
    # ids (1024 threads, four groups of four each), of which the scan keeps one ahead
    say(f"long history edges {rows}x{vocab} {tin}->{tout}")
    edges = [0, 1, 3, 16383, 16384, 16385, 32767, 32768, 32769, 49152, 49155, 65536, 65539]
    for width in (16384, 32769, 65539):
        logits, u = make(rows, vocab, width, 7, False, rows + width, in_type=tin)
        rng = np.random.default_rng(width)
        u["history_lengths"].copy_(torch.from_numpy(rng.choice(edges, rows).astype(np.int32)))
        u["prompt_lengths"].copy_(torch.from_numpy(rng.choice(edges, rows).astype(np.int32)))
        out = LogitsRules(vocab, **u).apply(logits, out_dtype=TYPES[tout])
        torch.cuda.synchronize()
        check(out, *expected(logits, u), f"{rows} x {width}")


@pytest.mark.parametrize("tin", ["bf16", "fp16", "fp32"])
def test_rules_special_values(tin):
    rows, vocab = 8, 4100
    logits, u = make(rows, vocab, 200, 8, True, 5, in_type=tin)
    for j, v in enumerate((math.inf, -math.inf, math.nan, torch.finfo(TYPES[tin]).min, torch.finfo(TYPES[tin]).max, 0.0)):
        logits[:, j::61] = v     # in allowed and in masked places
    # no rule that takes the largest finite values beyond fp32 on the way
    u["repetition"].fill_(1.0)
    u["temperature"].clamp_(min=1.0)
    # an infinity and a bias of the other sign make NaN, in the definition too
    out = LogitsRules(vocab, **u).apply(logits)
    torch.cuda.synchronize()
    check(out, *expected(logits, u), tin)
    assert bool((out[3] == -math.inf).all())     # a row whose mask leaves nothing


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_rules_in_place_and_fewer_rows_than_tables(t):
    logits, u = make(9, 12345, 300, 20, True, 6, in_type=t)
    rules = LogitsRules(12345, **u)
    few = logits[:4].clone()
    want = expected(few, {k: v[:4] for k, v in u.items()})
    got = rules.apply(few, out=few)
    torch.cuda.synchronize()
    assert got.data_ptr() == few.data_ptr()
    check(few, *want, "in place")


def test_rules_one_mask_for_all_rows():
    logits, u = make(7, 10001, 0, 0, True, 4)
    for mask in (u["mask"][0], u["mask"][:1]):
        out = LogitsRules(10001, mask=mask).apply(logits)
        torch.cuda.synchronize()
        check(out, *expected(logits, {"mask": mask}), "one mask")


def test_rules_no_rows_and_repeat_is_deterministic():
    logits, u = make(6, 30000, 4000, 50, True, 2)
    rules = LogitsRules(30000, **u)
    out = torch.full((6, 30000), FILL, device="cuda")
    rules.apply(logits[:0], out=out[:0])
    torch.cuda.synchronize()
    assert bool((out == FILL).all())
    a, b = rules.apply(logits), rules.apply(logits)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_rules_graph_sees_what_the_tables_hold_and_another_stream():
    rows, vocab = 3, 20001
    logits, u = make(rows, vocab, 64, 8, True, 7)
    u["history_lengths"].copy_(torch.tensor([5, 0, 20], dtype=torch.int32))
    u["prompt_lengths"].fill_(3)
    rules = LogitsRules(vocab, **u)
    out = torch.zeros(rows, vocab, device="cuda")
    rules.apply(logits, out=out)   # loaded before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rules.apply(logits, out=out)
    for step in range(4):
        # the program's own work between replays: a token more, another mask
        for r in range(rows):
            u["history"][r, int(u["history_lengths"][r])] = 100 * step + r
        u["history_lengths"] += 1
        u["mask"].copy_(torch.roll(u["mask"], 1, 0))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(out, *expected(logits, u), f"replay {step}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = rules.apply(logits)
    side.synchronize()
    assert torch.equal(other, out)


@pytest.mark.parametrize("seed", range(12))
def test_rules_random(seed):
    rng = np.random.default_rng(seed + 60)
    rows, vocab = int(np.exp(rng.uniform(0, 4))), int(np.exp(rng.uniform(0, 11)))
    width, biases = int(rng.choice([0, 1, 50, 3000])), int(rng.choice([0, 1, 200]))
    tin, tout = rng.choice(["bf16", "fp16", "fp32"], 2)
    mask, strided = bool(rng.integers(2)), bool(rng.integers(2))
    label = f"random {seed}: {rows}x{vocab} history {width} biases {biases} mask {mask} {tin}->{tout} {strided}"
    say(label)
    logits, u = make(rows, vocab, width, biases, mask, seed, strided, tin)
    out = LogitsRules(vocab, **u).apply(logits, out_dtype=TYPES[tout])
    torch.cuda.synchronize()
    check(out, *expected(logits, u), label)


def test_rules_refusals():
    logits, u = make(4, 1000, 20, 6, True, 1)
    with pytest.raises(ValueError, match="at most 4 rows"):
        LogitsRules(1000, **u).apply(torch.zeros(5, 1000, device="cuda"))
    with pytest.raises(ValueError, match="logits must be on the GPU"):
        LogitsRules(1000, **u).apply(logits.cpu())
    with pytest.raises(ValueError, match="GPU"):
        LogitsRules(1000).apply(logits.cpu())
    with pytest.raises(ValueError, match="presence must be on the GPU"):
        LogitsRules(1000, **{**u, "presence": u["presence"].cpu()})
    with pytest.raises(B.MoeError, match="out overlaps logits"):
        wide = torch.zeros(4, 1500, device="cuda")
        LogitsRules(1000, **u).apply(wide[:, :1000], out=wide[:, 500:])
    with pytest.raises(B.MoeError, match="out overlaps mask"):
        mask = torch.zeros(4, 1000, dtype=torch.int32, device="cuda")
        LogitsRules(1000, mask=mask).apply(logits, out=mask.view(torch.float32))


def test_head_of_a_decode_step_eager_and_in_a_graph():
    """Hidden states through a mixer pair with its residual, lm_head and the
    rules, each stage against fp64 from the stage before it, then the whole
    step captured and replayed while the program appends tokens."""
    T, wide, low, hidden, vocab = 5, 1024, 128, 256, 20011
    rng = np.random.default_rng(0)

    def weights(n, k, group, seed):
        h = synth.make_int8_linear(1, n, k, group, seed=seed)
        f = 0.0135 / math.sqrt(k) / synth.INT8_SCALE_STD
        s = torch.from_numpy(h["scales"].view(np.int16)).view(torch.bfloat16).float().mul(f).to(torch.bfloat16)
        p = torch.from_numpy(h["packed"])
        w = (p.view(torch.uint8).double() - 128) * s.double().repeat_interleave(group, 1)
        return p.cuda(), s.cuda(), w

    dp, ds, dw = weights(low, wide, 64, 1)
    up, us, uw = weights(wide, low, 64, 2)
    hp, hs, hw = weights(vocab, hidden, 128, 3)
    down, upl = Int8Linear(dp, ds, 64, activation="silu"), Int8Linear(up, us, 64)
    head = Int8Linear(hp, hs, 128)
    stream = torch.from_numpy(rng.standard_normal((T, wide))).to(torch.bfloat16).cuda()
    _, u = make(T, vocab, 40, 6, True, 3)
    u["history_lengths"].fill_(10)
    rules = LogitsRules(vocab, **u)

    def step():
        low_ = down.forward(stream)
        mixed = upl.forward(low_, residual=stream)
        logits = head.forward(mixed[:, :hidden], out_dtype=torch.float32)   # a column range: strided rows
        return low_, mixed, logits, rules.apply(logits)

    low_, mixed, logits, out = step()
    torch.cuda.synchronize()
    b16 = 2.0 ** -8      # half a bf16 step, relative; the fp32 sums below add far less than 1e-4
    v = stream.double().cpu() @ dw.T
    assert torch.allclose(low_.double().cpu(), v * torch.sigmoid(v), rtol=b16, atol=1e-4)
    assert torch.allclose(mixed.double().cpu(), stream.double().cpu() + low_.double().cpu() @ uw.T, rtol=b16, atol=1e-4)
    assert torch.allclose(logits.double().cpu(), mixed[:, :hidden].double().cpu() @ hw.T, rtol=1e-5, atol=1e-4)
    check(out, *expected(logits, u), "rules of the step")

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(3):
        u["history"][:, 10 + i] = torch.randint(0, vocab, (T,), dtype=torch.int32, device="cuda")
        u["history_lengths"] += 1
        stream.mul_(-1.25)
        g.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {i}"
