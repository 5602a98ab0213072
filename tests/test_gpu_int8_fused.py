"""moe_int8_linear_fused on the GPU against the fp64 oracle of the INT8 linear
layer followed by the epilogue in fp64.

Tolerance, from the arithmetic (u = 2^-24, half a step of fp32):
  * the products code * x are exact (fp16 operands); one output's sum passes
    through at most G roundings within a group, two per group to fold it in
    and 32 to join lanes, waves and K splits, each at most u times the sum of
    the terms' magnitudes; an activation below fp16's normal range (2^-14)
    is off by at most 2^-24;
  * the activations have slopes of at most 1.13; exp, erfc, the division and
    the products around them take at most 16 roundings of the result, and a
    rounding of the argument of exp(-2 u) or erfc(z) moves the result by
    2 |u| or 2 z^2 of its ulps;
  * the addition of the residual is one more rounding of its result;
  * the store rounds once: half a step of the output's type."""
import math
import sys

import numpy as np
import pytest
import torch

import oracle
from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd import synth
from quantized_moe_router_amd.layer import Int8Linear

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.lib()
    yield


def half_step(o, dtype):
    """Half a step of the type at each value of o (its subnormal step near zero)."""
    f = torch.finfo(dtype)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(o), f.tiny)))) * f.eps
    return step / 2


def erfc(z):
    return torch.special.erfc(torch.from_numpy(z)).numpy()


def sigmoid(v):
    return torch.sigmoid(torch.from_numpy(v)).numpy()


def act64(v, kind):
    """(act(v), the bound of its own rounding errors)."""
    if kind == "relu":
        return np.maximum(v, 0), np.zeros_like(v)
    if kind == "silu":
        a, amp = v * sigmoid(v), 0.0
    elif kind == "gelu":
        a, amp = 0.5 * v * erfc(-v / math.sqrt(2)), v * v
    elif kind == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        a, amp = v * sigmoid(2 * u), 10 * np.abs(u)
    elif kind == "sigmoid":
        a, amp = sigmoid(v), 0.0
    else:
        return v, np.zeros_like(v)
    # a sigmoid below fp32's normal range, 2^-126, comes out as zero: that much
    # of the factor v, and of the result itself where there is none
    return a, (16 + amp) * U * np.abs(a) + 2.0 ** -126 * np.maximum(np.abs(v), 1)


def inside(t, extra, fill):
    """t in rows `extra` elements wider, the rest holding `fill`."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide, wide[:, :t.shape[1]]


def case(T, N, K, G, bias, residual, out, strided, seed, scale=None):
    layer = synth.make_int8_linear(T, N, K, G, seed=seed)
    rng = np.random.default_rng(seed + 5)
    # sums of about unit size, which the activations bend
    f = (0.0135 / math.sqrt(K) if scale is None else scale) / synth.INT8_SCALE_STD
    scales = torch.from_numpy(layer["scales"].view(np.int16)).view(torch.bfloat16).float() * f
    layer["scales"] = synth.bf16_bits(scales.numpy())
    d = {"x": torch.from_numpy(layer["x"].view(np.int16)).cuda().view(torch.bfloat16),
         "packed": torch.from_numpy(layer["packed"]).cuda(),
         "scales": torch.from_numpy(layer["scales"].view(np.int16)).cuda().view(torch.bfloat16),
         "bias": None, "residual": None, "group": G}
    if bias:
        d["bias"] = torch.from_numpy(rng.standard_normal(N)).to(TYPES[bias]).cuda()
    if residual:
        d["residual"] = torch.from_numpy(rng.standard_normal((T, N))).to(TYPES[residual]).cuda()
    d["out"] = torch.full((T, N), 77.0, dtype=TYPES[out], device="cuda")
    d["wide"] = {}
    if strided:
        d["wide"]["x"], d["x"] = inside(d["x"], 24, math.nan)
        d["wide"]["out"], d["out"] = inside(d["out"], 5, 55.0)
        if residual:
            d["wide"]["residual"], d["residual"] = inside(d["residual"], 3, math.nan)
    return layer, d


def expected(layer, d, kind, tokens=None):
    """(fp64 value, bound before the store) of every output of the tokens."""
    pick = slice(None) if tokens is None else tokens
    G = d["group"]
    x = np.ascontiguousarray(layer["x"][pick])
    o = oracle.int8_linear(x, layer["packed"], layer["scales"], G)
    xf = np.abs((x.astype(np.uint32) << 16).view(np.float32)).astype(np.float64)
    q = np.abs(layer["packed"].view(np.uint8).astype(np.int16) - 128).astype(np.float64)
    s = (layer["scales"].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    w = q * np.repeat(np.abs(s), G, axis=1)
    K = w.shape[1]
    err = (G + 2 * K // G + 32) * U * (xf @ w.T) + (w.sum(1) * 2.0 ** -24)[None, :]
    v = o
    if d["bias"] is not None:
        v = o + d["bias"].double().cpu().numpy()
        err = err + U * np.abs(v)
    a, own = act64(v, kind)
    err = 1.13 * err + own
    if d["residual"] is not None:
        a = a + d["residual"][pick].double().cpu().numpy()
        err = err + U * np.abs(a)
    return a, err


def check(got, want, err, dtype, label):
    bound = err + half_step(np.abs(want) + err, dtype)
    off = np.abs(got.double().cpu().numpy() - want)
    bad = np.argwhere(~(off <= bound))
    assert bad.size == 0, (f"{label}: {len(bad)} of {off.size} off, first {bad[0].tolist()}: "
                           f"{got[tuple(bad[0])].item()} for {want[tuple(bad[0])]} +- {bound[tuple(bad[0])]}")


def run(d, kind, **kw):
    need = B.moe_int8_linear_fused_workspace_bytes(*d["x"].shape[:1], *d["packed"].shape[:1], d["x"].shape[1], d["group"])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    T, K = d["x"].shape
    B.moe_int8_linear_fused(d["x"], d["packed"], d["scales"], T, d["packed"].shape[0], K, d["group"], d["out"],
                            d["bias"], d["residual"], kind, ws, **kw)
    return d["out"]


CASES = [
    # (T, N, K, G, bias, activation, residual, out, strided): every plan,
    # one token to many, ragged and odd sizes, each type in each place
    (1, 37, 128, 64, "bf16", "silu", None, "fp32", False),
    (1, 9, 64, 64, None, "none", "fp32", "bf16", False),
    (1, 1, 64, 64, "fp32", "sigmoid", "bf16", "fp16", False),
    (2, 130, 320, 64, "fp32", "gelu", "bf16", "fp32", True),
    (3, 8193, 2048, 64, None, "gelu_tanh", "fp16", "fp16", True),
    (4, 10240, 320, 64, None, "none", "bf16", "bf16", False),
    (4, 9000, 2560, 128, "fp16", "none", None, "fp32", False),
    (1, 320, 10240, 64, None, "silu", None, "bf16", False),
    (1, 300, 2560, 128, "fp16", "relu", "bf16", "fp32", True),
    (3, 77, 1152, 128, "bf16", "gelu", None, "fp16", True),
    (4, 320, 4096, 64, "fp32", "silu", "fp32", "fp32", False),
    (2, 7, 65536, 128, "bf16", "none", None, "fp32", False),
    (5, 777, 448, 64, "bf16", "silu", "bf16", "bf16", True),
    (7, 9001, 1152, 128, None, "none", "fp32", "fp32", False),
    (16, 2001, 320, 64, "fp32", "gelu_tanh", "fp16", "fp16", True),
    (12, 8200, 2560, 128, "fp16", "none", None, "fp32", False),
    (5, 320, 10240, 64, "bf16", "silu", None, "bf16", False),
    (5, 8189, 512, 64, "bf16", "silu", "fp16", "fp32", True),
    (3, 131072, 512, 64, "bf16", "none", None, "bf16", False),
    (4, 33000, 2048, 128, None, "silu", "bf16", "fp32", True),
    (6, 8200, 640, 64, None, "gelu", "bf16", "fp16", False),
    (9, 33001, 768, 128, "fp32", "none", "fp32", "fp32", True),
    (13, 70000, 512, 64, None, "relu", None, "bf16", False),
    (16, 8192, 2560, 128, "bf16", "none", "bf16", "fp32", False),
    (8, 8190, 4096, 64, None, "sigmoid", None, "fp32", False),
    (16, 66000, 256, 64, None, "none", None, "fp32", False),
    (7, 10240, 320, 64, None, "none", "bf16", "bf16", False),
    (11, 8195, 4224, 64, "bf16", "none", "bf16", "fp32", True),
    (40, 77, 8192, 64, "bf16", "silu", "bf16", "fp32", True),
    (300, 40, 16384, 128, None, "silu", "fp16", "fp16", False),
    (6, 320, 2048, 64, "bf16", "silu", "bf16", "bf16", False),
    (9, 317, 2048, 64, "bf16", "silu", "fp32", "fp32", True),
    (16, 33, 4096, 128, None, "relu", "fp16", "fp32", False),
    (1, 5, 65536, 64, None, "none", "fp32", "fp32", False),
    (33, 129, 1024, 128, "fp32", "relu", "fp32", "fp32", True),
    (77, 1003, 1152, 128, "fp32", "gelu", "fp16", "fp16", True),
    (130, 332, 1024, 64, "bf16", "sigmoid", "bf16", "fp32", False),
    (200, 96, 4096, 64, None, "silu", "bf16", "bf16", False),
    (200, 95, 4096, 64, "fp16", "silu", "bf16", "fp32", False),
    (64, 1000, 2560, 128, "bf16", "none", "fp32", "fp32", True),
    (17, 9, 64, 64, "bf16", "silu", "bf16", "fp32", True),
    (129, 130, 128, 128, "fp32", "gelu", "fp16", "bf16", False),
    (200, 333, 192, 64, None, "gelu_tanh", "fp32", "fp16", True),
    (300, 256, 256, 128, "fp16", "silu", "fp32", "fp32", False),
    (96, 300, 320, 64, "bf16", "relu", "bf16", "bf16", False),
    (260, 513, 256, 64, None, "none", "bf16", "fp32", False),
]


@pytest.mark.parametrize("T,N,K,G,bias,kind,residual,out,strided", CASES)
def test_fused_small(T, N, K, G, bias, kind, residual, out, strided):
    label = f"fused T={T} N={N} K={K} G={G} {bias} {kind} {residual} -> {out} {strided}"
    say(label)
    layer, d = case(T, N, K, G, bias, residual, out, strided, seed=1000 * T + N)
    got = run(d, kind)
    torch.cuda.synchronize()
    want, err = expected(layer, d, kind)
    check(got, want, err, TYPES[out], label)
    if strided:   # what lies between the rows stays
        assert bool((d["wide"]["out"][:, N:] == 55.0).all())


@pytest.mark.parametrize("T,N,K,G,bias,kind,residual,out", [
    (5000, 1283, 64, 64, "bf16", "silu", "fp32", "fp16"), (3000, 2051, 320, 64, None, "none", "bf16", "fp32"),
    (4500, 1025, 256, 128, "fp32", "gelu", "fp16", "bf16"), (4900, 1154, 192, 64, "fp16", "none", None, "fp32"),
    (2500, 1283, 128, 128, None, "sigmoid", "fp32", "fp32"), (1100, 711, 384, 64, "bf16", "gelu", "fp32", "fp32"),
    (2100, 1283, 640, 128, "fp32", "silu", "bf16", "fp16"), (2000, 1030, 448, 64, None, "none", "fp16", "bf16")])
@pytest.mark.parametrize("strided", [False, True])
def test_fused_many_tokens_of_unaligned_rows(T, N, K, G, bias, kind, residual, out, strided):
    # several token tiles to a workgroup, columns that share no aligned word
    label = f"unaligned T={T} N={N} K={K} {kind} {residual}->{out} {strided}"
    say(label)
    layer, d = case(T, N, K, G, bias, residual, out, strided, seed=T)
    got = run(d, kind)
    torch.cuda.synchronize()
    want, err = expected(layer, d, kind)
    check(got, want, err, TYPES[out], label)


@pytest.mark.parametrize("which,T", [("down", 512), ("up", 512), ("up", 2000)])
def test_fused_mixer_shapes(which, T):
    N, K = (320, 10240) if which == "down" else (10240, 320)
    label = f"mixer {which} T={T}"
    say(label)
    kind, residual = ("silu", None) if which == "down" else ("none", "bf16")
    layer, d = case(T, N, K, 64, "bf16", residual, "fp32", False, seed=T)
    got = run(d, kind)
    torch.cuda.synchronize()
    toks = np.unique(np.concatenate([[0, T - 1], np.random.default_rng(T).choice(T, 30, replace=False)]))
    want, err = expected(layer, d, kind, toks)
    check(got[torch.from_numpy(toks).cuda()], want, err, torch.float32, label)


@pytest.mark.parametrize("T", [1, 3, 8, 40])
@pytest.mark.parametrize("N,K", [(64, 128), (64, 1024)])
@pytest.mark.parametrize("kind", sorted(B.ACTIVATIONS))
def test_fused_activations_over_their_range(kind, T, N, K):
    # sums up to a few hundred: both saturated ends of every activation
    label = f"{kind} T={T} N={N} K={K}"
    say(label)
    layer, d = case(T, N, K, 64, None, None, "fp32", False, seed=T + K, scale=1.0 / math.sqrt(K))
    got = run(d, kind)
    torch.cuda.synchronize()
    want, err = expected(layer, d, kind)
    check(got, want, err, torch.float32, label)
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("T,N,K,G", [(1, 64, 128, 64), (2, 320, 1024, 64), (8, 900, 256, 128), (40, 96, 4096, 64),
                                     (130, 260, 256, 64), (64, 1000, 1280, 128)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_fused_residual_in_place(T, N, K, G, out):
    label = f"in place T={T} N={N} K={K} {out}"
    say(label)
    layer, d = case(T, N, K, G, "bf16", out, out, False, seed=T + N)
    want, err = expected(layer, d, "silu")
    d["out"] = d["residual"]
    got = run(d, "silu")
    torch.cuda.synchronize()
    check(got, want, err, TYPES[out], label)


@pytest.mark.parametrize("T", [1, 8, 100])
def test_fused_rows_interleaved_with_x_and_residual(T):
    # x, residual and out as column ranges of one wide buffer
    N, K, G = 72, 128, 64
    layer, d = case(T, N, K, G, None, "bf16", "bf16", False, seed=T)
    buf = torch.full((T, K + 2 * N + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    buf[:, :K] = d["x"]
    buf[:, K:K + N] = d["residual"]
    d["x"], d["residual"], d["out"] = buf[:, :K], buf[:, K:K + N], buf[:, K + N:K + 2 * N]
    want, err = expected(layer, d, "none")
    got = run(d, "none")
    torch.cuda.synchronize()
    check(got, want, err, torch.bfloat16, f"interleaved T={T}")
    assert bool((buf[:, K + 2 * N:] == 3.0).all())


@pytest.mark.parametrize("T,N,K", [(1, 40, 128), (2, 40, 1024), (8, 40, 128), (40, 40, 128), (40, 40, 1024)])
def test_fused_infinities_nan_and_fp16_overflow(T, N, K):
    say(f"specials T={T} N={N} K={K}")
    layer, d = case(T, N, K, 64, "fp32", "fp32", "fp16", False, seed=T)
    d["bias"][3] = 1e6          # beyond fp16: infinite after the store
    d["bias"][4] = -1e6
    d["bias"][5] = math.nan
    d["residual"][:, 6] = math.inf
    d["residual"][:, 7] = math.nan
    d["residual"][0, 8] = -math.inf
    got = run(d, "none").float()
    torch.cuda.synchronize()
    assert bool((got[:, 3] == math.inf).all()) and bool((got[:, 4] == -math.inf).all())
    assert bool(got[:, 5].isnan().all()) and bool((got[:, 6] == math.inf).all())
    assert bool(got[:, 7].isnan().all()) and got[0, 8].item() == -math.inf
    rest = [i for i in range(N) if i not in (3, 4, 5, 6, 7, 8)]
    want, err = expected(layer, d, "none")
    check(got[:, rest], want[:, rest], err[:, rest], torch.float16, "the other columns")


@pytest.mark.parametrize("T,N,K,G", [(1, 320, 10240, 64), (3, 4100, 320, 64), (8, 9001, 1152, 128), (9, 320, 10240, 64),
                                     (16, 8200, 2560, 128), (5, 40000, 512, 64), (2000, 256, 1024, 64),
                                     (512, 320, 10240, 64), (100, 10240, 320, 64), (70, 1000, 1152, 128)])
def test_fused_graph_replay_and_another_stream(T, N, K, G):
    label = f"graph T={T} N={N} K={K}"
    say(label)
    _, d = case(T, N, K, G, "bf16", "fp32", "fp32", False, seed=9)
    eager = run(d, "gelu").clone()
    torch.cuda.synchronize()
    lin = Int8Linear(d["packed"], d["scales"], G, bias=d["bias"], activation="gelu")
    out = torch.zeros(T, N, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin.forward(d["x"], residual=d["residual"], out=out)
    for i in range(3):
        out.zero_()
        junk = torch.randn(1 << 16, device="cuda") * (i + 1)   # eager work between replays
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), f"{label}: replay {i} differs"
        del junk
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = lin.forward(d["x"], residual=d["residual"], out_dtype=torch.float32)
    side.synchronize()
    assert torch.equal(other, eager), f"{label}: another stream differs"


def test_fused_two_graphs_at_once():
    # two captured calls of one layer, replayed on two streams at a time:
    # each has partial sums of its own
    T, N, K, G = 256, 320, 10240, 64
    _, d = case(T, N, K, G, None, None, "fp32", False, seed=4)
    _, d2 = case(T, N, K, G, None, None, "fp32", False, seed=5)
    lin = Int8Linear(d["packed"], d["scales"], G, activation="silu")
    want = [lin.forward(v["x"], out_dtype=torch.float32).clone() for v in (d, d2)]
    outs, graphs = [], []
    for v in (d, d2):
        out = torch.zeros(T, N, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lin.forward(v["x"], out=out)
        outs.append(out)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out, w), f"replay {i}"
            out.zero_()
        torch.cuda.synchronize()


def test_fused_zero_tokens_and_no_epilogue():
    layer, d = case(33, 130, 320, 64, None, None, "bf16", False, seed=2)
    before = d["out"].clone()
    B.moe_int8_linear_fused(d["x"][:0], d["packed"], d["scales"], 0, 130, 320, 64, d["out"][:0])
    torch.cuda.synchronize()
    assert torch.equal(d["out"], before)
    got = run(d, "none")
    plain = torch.empty(33, 130, dtype=torch.bfloat16, device="cuda")
    need = B.moe_int8_linear_workspace_bytes(33, 130, 320, 64)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    B.moe_int8_linear(d["x"], d["packed"], d["scales"], 33, 130, 320, 64, plain, ws)
    torch.cuda.synchronize()
    want, err = expected(layer, d, "none")
    check(got, want, err, torch.bfloat16, "no epilogue")
    check(plain, want, err, torch.bfloat16, "moe_int8_linear")


@pytest.mark.parametrize("seed", range(40))
def test_fused_random_shapes(seed):
    rng = np.random.default_rng(seed + 300)
    G = int(rng.choice([64, 128]))
    T = int(np.exp(rng.uniform(0, np.log(400))))
    K = G * int(rng.integers(1, 2048 // G + 1))
    N = int(np.exp(rng.uniform(np.log(3), np.log(2500))))
    pick = lambda *a: a[int(rng.integers(len(a)))]  # noqa: E731
    c = (pick(None, "bf16", "fp16", "fp32"), pick(*sorted(B.ACTIVATIONS)), pick(None, "bf16", "fp16", "fp32"),
         pick("bf16", "fp16", "fp32"), bool(rng.integers(2)))
    label = f"random {seed}: T={T} N={N} K={K} G={G} {c}"
    say(label)
    bias, kind, residual, out, strided = c
    layer, d = case(T, N, K, G, bias, residual, out, strided, seed=seed)
    got = run(d, kind)
    torch.cuda.synchronize()
    want, err = expected(layer, d, kind)
    check(got, want, err, TYPES[out], label)


def test_fused_refuses_host_tensors_and_bad_shapes():
    _, d = case(3, 16, 64, 64, None, None, "fp32", False, seed=1)
    lin = Int8Linear(d["packed"], d["scales"], 64)
    with pytest.raises(ValueError, match="GPU"):
        Int8Linear(d["packed"].cpu(), d["scales"].cpu(), 64).forward(d["x"].cpu())
    with pytest.raises(ValueError, match="x is"):
        lin.forward(d["x"][:, :32])
    with pytest.raises(ValueError, match="residual must be on the GPU"):
        lin.forward(d["x"], residual=torch.zeros(3, 16))
    with pytest.raises(ValueError, match="consecutive"):
        lin.forward(d["x"], out=torch.empty(16, 3, device="cuda").t())
    with pytest.raises(B.MoeError, match="x is not 16-byte aligned"):
        lin.forward(torch.zeros(3, 72, dtype=torch.bfloat16, device="cuda")[:, 1:65])
    with pytest.raises(B.MoeError, match="out overlaps x"):
        buf = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
        lin.forward(buf, out=buf[:, :16])
    with pytest.raises(B.MoeError, match="out overlaps residual"):
        buf = torch.zeros(3, 40, device="cuda")
        lin.forward(d["x"], residual=buf[:, :16], out=buf[:, 8:24])
