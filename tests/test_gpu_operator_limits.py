"""moe_int8_linear_fused and moe_int4_logits_process at the ends of what their
documentation allows: rows 2^24 elements apart, 2^24 weight rows, K = 65536,
more than 2^32 logits, vocabularies and histories of 2^24, 65536 rows; two
threads and two branches of one graph at once.

The INT8 layer's outputs are compared at sampled places with sums in fp64, by
the tolerance of test_gpu_int8_fused.py; the rules with the fp64 form of
test_gpu_logits.py."""
import sys
import threading

import numpy as np
import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import Int8Linear, LogitsRules
from test_gpu_int8_fused import U, half_step
from test_gpu_int8_plans import EVERY, kernel
from test_gpu_logits import check as check_rules
from test_gpu_logits import expected, make

pytestmark = pytest.mark.gpu

MOST = 1 << 24


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def layer(N, K, G, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    packed = torch.randint(-2**31, 2**31 - 1, (N, K // 4), dtype=torch.int32, device="cuda", generator=g)
    scales = (torch.randn(N, K // G, device="cuda", generator=g).abs() * (0.0135 / K ** 0.5)).to(torch.bfloat16)
    return packed, scales


def far(t, stride, fill):
    """t with its rows `stride` elements apart, `fill` between them."""
    wide = torch.full(((t.shape[0] - 1) * stride + t.shape[1],), fill, dtype=t.dtype, device="cuda")
    v = wide.as_strided(t.shape, (stride, 1))
    v.copy_(t)
    return wide, v


def compare(got, x, packed, scales, G, residual, rows, toks, label):
    """Sampled outputs residual + x W^T against fp64."""
    K = x.shape[1]
    r, t = torch.as_tensor(rows, device="cuda"), torch.as_tensor(toks, device="cuda")
    w = (packed[r].view(torch.uint8).double() - 128) * scales[r].double().repeat_interleave(G, 1)
    xs = x[t].double()
    want = xs @ w.t().contiguous()
    err = (G + 2 * K // G + 32) * U * (xs.abs() @ w.abs().t().contiguous()) + w.abs().sum(1) * 2.0 ** -24
    want, err = want.cpu().numpy(), err.cpu().numpy()
    if residual is not None:
        want = want + residual[t][:, r].double().cpu().numpy()
        err = err + U * np.abs(want)
    g = got[t][:, r].double().cpu().numpy()
    bad = np.argwhere(~(np.abs(g - want) <= err + half_step(np.abs(want) + err, got.dtype)))
    assert bad.size == 0, f"{label}: {len(bad)} off, first {bad[0]}: {g[tuple(bad[0])]} for {want[tuple(bad[0])]}"


FAR = {**EVERY, "gemm": (129, 13000, 384, 64), "gemm split": (129, 13000, 640, 64)}


@pytest.mark.parametrize("name", FAR)
def test_rows_two_to_the_24_elements_apart(name):
    T, N, K, G = FAR[name]
    assert kernel(T, N, K, G) == name
    say(f"{name}: T={T} N={N} K={K}, rows 2^24 apart")
    packed, scales = layer(N, K, G, 1)
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    res = torch.randn(T, N, device="cuda").to(torch.bfloat16)
    plain = Int8Linear(packed, scales, G).forward(x, residual=res, out_dtype=torch.float32)
    _, xf = far(x, MOST, 3.0)
    _, rf = far(res, MOST, 4.0)
    wide, out = far(torch.zeros(T, N, device="cuda"), MOST, 55.0)
    Int8Linear(packed, scales, G).forward(xf, residual=rf, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, plain)
    out.fill_(55.0)
    assert bool((wide == 55.0).all())    # what lies between the rows is as it was
    compare(plain, x, packed, scales, G, res, np.unique(np.linspace(0, N - 1, 300).astype(np.int64)),
            np.unique(np.linspace(0, T - 1, 20).astype(np.int64)), name)


@pytest.mark.parametrize("T", [1, 4, 7, 16, 20, 100])
def test_two_to_the_24_weight_rows(T):
    say(f"T={T} N=2^24 K=64")
    packed, scales = layer(MOST, 64, 64, T)
    x = torch.randn(T, 64, device="cuda").to(torch.bfloat16)
    out = Int8Linear(packed, scales, 64).forward(x, out_dtype=torch.float16)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([np.linspace(0, MOST - 1, 4001).astype(np.int64), np.arange(MOST - 300, MOST)]))
    compare(out, x, packed, scales, 64, None, rows, np.arange(T), f"T={T}")


@pytest.mark.parametrize("T,N,G", [(1, 8195, 64), (3, 8195, 128), (4, 8189, 64), (16, 8197, 64), (33, 1001, 128),
                                   (200, 8193, 64)])
def test_k_of_65536(T, N, G):
    K = 65536
    say(f"T={T} N={N} K={K} G={G}: {kernel(T, N, K, G)}")
    packed, scales = layer(N, K, G, T)
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    out = Int8Linear(packed, scales, G).forward(x, out_dtype=torch.float32)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([np.linspace(0, N - 1, 200).astype(np.int64), np.arange(N - 20, N)]))
    compare(out, x, packed, scales, G, None, rows, np.unique(np.linspace(0, T - 1, 16).astype(np.int64)), f"T={T}")


@pytest.mark.parametrize("T,N,G", [(1 << 20, 3, 64), ((1 << 20) - 5, 130, 128), (300000, 7000, 64)])
def test_a_million_tokens(T, N, G):
    K = 128
    say(f"T={T} N={N} K={K} G={G}: {kernel(T, N, K, G)}")
    packed, scales = layer(N, K, G, N)
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    out = Int8Linear(packed, scales, G).forward(x)
    torch.cuda.synchronize()
    toks = np.unique(np.concatenate([np.linspace(0, T - 1, 2000).astype(np.int64), np.arange(T - 200, T)]))
    compare(out, x, packed, scales, G, None, np.unique(np.linspace(0, N - 1, 60).astype(np.int64)), toks, f"T={T}")


@pytest.mark.parametrize("rows,vocab,t", [(17300, 248321, "bf16"), (65536, 66000, "fp16")])
def test_more_than_two_to_the_32_logits(rows, vocab, t):
    say(f"rules {rows}x{vocab} {t}, in place")
    assert rows * vocab > 1 << 32
    some, u = make(8, vocab, 50, 5, True, rows, in_type=t)
    want = expected(some, u)
    # eight kinds of rows over and over
    at = (torch.arange(rows, device="cuda") * 5) % 8
    logits = torch.empty(rows, vocab, dtype=some.dtype, device="cuda")
    for r in range(8):
        logits[at == r] = some[r]
    rules = LogitsRules(vocab, **{k: v[at].contiguous() for k, v in u.items()})
    rules.apply(logits, out=logits)
    torch.cuda.synchronize()
    # every kind's first row against fp64, every other row against its first
    firsts = torch.stack([logits[int((at == r).nonzero()[0])] for r in range(8)])
    check_rules(firsts, *want, f"{rows}x{vocab}")
    for lo in range(0, rows, 1024):
        same = logits[lo:lo + 1024].view(torch.int16) == firsts.view(torch.int16)[at[lo:lo + 1024]]
        nan = logits[lo:lo + 1024].isnan()
        assert bool((same | nan).all()), f"rows from {lo}"


def test_vocabulary_and_history_of_two_to_the_24():
    say("rules 2 x 2^24, history 2^24")
    logits, u = make(2, MOST, MOST, 300, True, 3)
    u["history_lengths"].copy_(torch.tensor([MOST, MOST - 3], dtype=torch.int32))
    u["prompt_lengths"].copy_(torch.tensor([5, MOST - 9], dtype=torch.int32))
    out = LogitsRules(MOST, **u).apply(logits)
    torch.cuda.synchronize()
    check_rules(out, *expected(logits, u), "2^24")


def test_rows_of_logits_two_to_the_24_elements_apart():
    say("rules 70 x 40001, every table's rows 2^24 apart")
    rows, vocab = 70, 40001
    logits, u = make(rows, vocab, 300, 9, True, 4, in_type="fp32")
    plain = LogitsRules(vocab, **u).apply(logits)
    _, lf = far(logits, MOST, 1.0)
    wide, out = far(torch.zeros(rows, vocab, device="cuda"), MOST, 55.0)
    for k in ("history", "mask", "bias_ids", "bias_values"):
        u[k] = far(u[k], MOST, 7)[1]
    LogitsRules(vocab, **u).apply(lf, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int32), plain.view(torch.int32))
    out.fill_(55.0)
    assert bool((wide == 55.0).all())


def test_two_threads_on_two_streams():
    # one layer whose partial sums pass through a workspace, one set of rules
    T, N, K, G = EVERY["kwaves split"]
    assert kernel(T, N, K, G) == "kwaves split"
    packed, scales = layer(N, K, G, 5)
    lin = Int8Linear(packed, scales, G, activation="silu")
    xs = [torch.randn(T, K, device="cuda").to(torch.bfloat16) for _ in range(2)]
    logits, u = make(2 * T, N, 40, 6, True, 6)
    rules = LogitsRules(N, **u)
    want = [rules.apply(lin.forward(x, out_dtype=torch.float32)) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    bad, bits = [], lambda t: t.view(torch.int32)  # noqa: E731

    def program(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(50):
                    got = rules.apply(lin.forward(xs[i], out_dtype=torch.float32))
                    if i == 1:   # this thread's refusals are its own
                        with pytest.raises(B.MoeError, match="out: stride 0"):
                            rules.apply(got, out=got[:1].expand(T, N))
                    same = torch.equal(bits(got), bits(want[i]))
                    if not same:
                        bad.append(i)
        except BaseException as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=program, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad


def test_two_branches_of_one_graph():
    T, N, K, G = EVERY["gemm split"]
    packed, scales = layer(N, K, G, 7)
    lin = Int8Linear(packed, scales, G, activation="gelu")
    xs = [torch.randn(T, K, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [lin.forward(x, out_dtype=torch.float32) for x in xs]
    outs = [torch.zeros_like(w) for w in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lin.forward(xs[1], out=outs[1])
        lin.forward(xs[0], out=outs[0])
        torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        for o in outs:
            o.zero_()
        lin.forward(xs[i % 2])   # eager work between the replays
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), f"replay {i}"


def test_one_step_beyond_the_limits_is_refused():
    logits, u = make(2, 1000, 20, 6, True, 1)
    rules = LogitsRules(1000, **u)
    with pytest.raises(B.MoeError, match="stride"):
        rules.apply(torch.empty(MOST + 1001, device="cuda").as_strided((2, 1000), (MOST + 1, 1)))
    packed, scales = layer(16, 64, 64, 1)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.MoeError, match="out: stride"):
        Int8Linear(packed, scales, 64).forward(x, out=torch.empty(MOST + 17, device="cuda").as_strided((2, 16), (MOST + 1, 1)))
    with pytest.raises(B.MoeError, match="x: stride"):
        xf = torch.zeros(MOST + 72, dtype=torch.bfloat16, device="cuda").as_strided((2, 64), (MOST + 8, 1))
        Int8Linear(packed, scales, 64).forward(xf)
