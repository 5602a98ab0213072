"""moe_int4_linear and moe_int4_grouped_linear on the GPU against their formula
in 64 bits.

Tolerance, from the arithmetic (u = 2^-24, half a step of fp32):
  * products x (code + 24) and 24 x are exact; a group of G inputs takes at most
    2 G additions in fp32, whose partial sums are sums of independent terms of
    at most 40 |x| each: at most 3 sigma, 120 |x_g| (2-norm).  2 G independent
    roundings of u times that come to 6 sqrt(2 G) u 120 |x_g| at six sigma.
    The group's scale multiplies it, and groups add up (each within the bound;
    taken as independent, by squares);
  * folding the groups in and joining waves and K splits is at most one rounding
    per group and 32 more, of u times the partial sums of the groups: 3 sigma of
    what the scaled groups add up to, sqrt(sum of squares of s_g 8 |x_g|);
  * the activations have slopes of at most 1.13; exp, erfc, the division and the
    products around them take at most 16 roundings of the result, and a rounding
    of the argument of exp(-2 u) or erfc(z) moves the result by 2 |u| or 2 z^2
    of its ulps;
  * the row's weight and the residual are one more rounding each;
  * the store rounds once: half a step of the output's type."""
import math
import sys

import numpy as np
import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd import synth
from quantized_moe_router_amd.layer import Int4GroupedLinear, Int4Linear, MoeInt4Layer

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


def matrix64(packed, scales, group):
    shifts = torch.arange(0, 32, 4, device=packed.device, dtype=torch.int32)
    q = (((packed.unsqueeze(-1) >> shifts) & 15) - 8).double().view(*packed.shape[:-1], -1, group)
    return (q * scales.double().unsqueeze(-1)).view(*packed.shape[:-1], -1)


def bound(x, scales, group):
    """The bound of the sums' errors, [rows, n] (see above)."""
    norm2 = x.double().view(x.shape[0], -1, group).square().sum(2)      # |x_g|^2
    s2 = scales.double().square()
    both = torch.mm(norm2, s2.t().contiguous()).sqrt()                  # sqrt(sum s_g^2 |x_g|^2)
    ng = scales.shape[1]
    return U * both * (6 * math.sqrt(2 * group) * 120 + (ng + 32) * 3 * 8)


def act64(v, kind):
    if kind == "relu":
        return v.clamp(min=0), torch.zeros_like(v)
    if kind == "silu":
        a, amp = v * torch.sigmoid(v), 0.0
    elif kind == "gelu":
        a, amp = 0.5 * v * torch.special.erfc(-v / math.sqrt(2)), v * v
    elif kind == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        a, amp = v * torch.sigmoid(2 * u), 10 * u.abs()
    elif kind == "sigmoid":
        a, amp = torch.sigmoid(v), 0.0
    else:
        return v, torch.zeros_like(v)
    return a, (16 + amp) * U * a.abs() + 2.0 ** -126 * v.abs().clamp(min=1)


def half_step(o, dtype):
    f = torch.finfo(dtype)
    return torch.exp2(torch.floor(torch.log2(o.abs().clamp(min=f.tiny)))) * f.eps / 2


def formula(x, packed, scales, group, kind, bias=None, weight=None, residual=None):
    """(value, bound of its error before the store) in 64 bits; weight [rows]."""
    v = torch.mm(x.double(), matrix64(packed, scales, group).t().contiguous())
    tol = bound(x, scales, group)
    if bias is not None:
        v = v + bias.double()
        tol = tol + U * v.abs()
    v, own = act64(v, kind)
    tol = 1.13 * tol + own
    if weight is not None:
        v = v * weight.double().unsqueeze(1)
        tol = tol * weight.double().abs().unsqueeze(1) + U * v.abs()
    if residual is not None:
        v = v + residual.double()
        tol = tol + U * v.abs()
    return v, tol


def check(got, want, tol, dtype, what):
    err = (got.double() - want).abs()
    limit = tol + half_step(want, dtype)
    limit = limit + half_step(want.abs() + limit, dtype) - half_step(want, dtype)   # the step of what is rounded
    share = (err / limit).max().item() if err.numel() else 0.0
    say(f"{what}: max share of the bound {share:.3f}")
    assert torch.isfinite(got).all() and share <= 1, f"{what}: {share}"


def inside(t, extra, fill):
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide, wide[:, :t.shape[1]]


def weights(shape, K, G, g):
    packed = torch.randint(-2**31, 2**31 - 1, (*shape, K // 8), dtype=torch.int32, device="cuda", generator=g)
    scales = (torch.randn(*shape, K // G, device="cuda", generator=g) * (0.27 / math.sqrt(K))).to(torch.bfloat16)
    return packed, scales


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


LINEAR = [
    # T, N, K, G, bias, activation, residual, out, strided
    (1, 2560, 2560, 128, None, "none", None, "bf16", False),
    (1, 1, 64, 64, None, "none", None, "fp32", False),
    (1, 33, 128, 128, "fp32", "silu", "fp32", "fp32", True),
    (2, 320, 640, 64, "bf16", "none", "bf16", "bf16", False),
    (3, 17, 192, 64, None, "gelu", "fp16", "fp16", True),
    (4, 10240, 320, 64, None, "none", "bf16", "bf16", False),
    (5, 1003, 1152, 128, "fp16", "relu", None, "fp32", True),
    (8, 4096, 2560, 128, None, "none", None, "fp32", False),
    (15, 257, 10240, 128, None, "sigmoid", None, "fp32", False),
    (16, 640, 2560, 128, "bf16", "gelu_tanh", "fp32", "bf16", False),
    (17, 640, 2560, 64, "bf16", "none", "fp32", "fp32", False),
    (31, 96, 64, 64, None, "none", None, "fp32", False),
    (32, 1000, 640, 128, None, "none", None, "fp32", False),
    (33, 2560, 640, 64, "fp32", "silu", "bf16", "fp16", True),
    (64, 511, 2560, 128, None, "none", None, "fp32", False),
    (65, 512, 2560, 128, None, "none", "fp32", "fp32", False),
    (77, 1003, 1152, 64, "fp32", "gelu", "fp16", "fp16", True),
    (128, 1280, 2560, 128, None, "none", None, "fp32", False),
    (129, 300, 192, 64, None, "none", None, "fp32", True),
    (200, 2562, 1088, 64, "fp32", "none", "fp32", "fp32", True),
    (300, 2560, 128, 128, None, "silu", "bf16", "bf16", False),
    (512, 10240, 2560, 128, None, "none", "bf16", "bf16", False),
    (1000, 700, 64, 64, None, "none", None, "fp32", False),
    (2049, 1281, 640, 128, "bf16", "none", None, "fp32", False),
]


@pytest.mark.parametrize("T,N,K,G,bias,kind,residual,out,strided", LINEAR)
def test_linear(T, N, K, G, bias, kind, residual, out, strided):
    g = generator(T * 1000 + N)
    say(f"linear T={T} N={N} K={K} G={G}")
    packed, scales = weights((N,), K, G, g)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
    b = torch.randn(N, device="cuda", generator=g).to(TYPES[bias]) if bias else None
    r = torch.randn(T, N, device="cuda", generator=g).to(TYPES[residual]) if residual else None
    o = torch.full((T, N), 77.0, dtype=TYPES[out], device="cuda")
    wide = None
    want, tol = formula(x, packed, scales, G, kind, b, None, r)
    if strided:
        _, x = inside(x, 24, math.nan)
        wide, o = inside(o, 5, 55.0)
        if residual:
            _, r = inside(r, 3, math.nan)
    layer = Int4Linear(packed, scales, G, bias=b, activation=kind)
    assert layer.forward(x, residual=r, out=o) is o
    check(o, want, tol, TYPES[out], f"T={T} N={N} K={K} G={G} {out}")
    if strided:
        assert (wide[:, N:] == 55.0).all()
    again = layer.forward(x, residual=r, out_dtype=TYPES[out])
    assert torch.equal(again, o)
    if residual == out:   # in place
        layer.forward(x, residual=r, out=r)
        assert torch.equal(r, o)


def test_linear_random_sweep():
    rng = np.random.default_rng(11)
    for i in range(40):
        T = int(np.exp(rng.uniform(0, np.log(700))))
        G = int(rng.choice([64, 128]))
        K = G * int(np.exp(rng.uniform(0, np.log(3000 // G))))
        N = int(np.exp(rng.uniform(0, np.log(3000))))
        out = str(rng.choice(["bf16", "fp16", "fp32"]))
        say(f"sweep {i}: T={T} N={N} K={K} G={G} {out}")
        g = generator(i)
        packed, scales = weights((N,), K, G, g)
        x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
        want, tol = formula(x, packed, scales, G, "none")
        check(Int4Linear(packed, scales, G).forward(x, out_dtype=TYPES[out]), want, tol, TYPES[out], f"sweep {i}")


@pytest.mark.parametrize("T", [1, 7, 40, 300])
@pytest.mark.parametrize("G", [64, 128])
def test_linear_wide_range_and_nonfinite(T, G):
    """Activations and scales over most of bf16's range; a NaN or an infinity of
    one token shows in that token alone."""
    N, K = 200, 640
    g = generator(5)
    packed, scales = weights((N,), K, G, g)
    scales = (scales.float() * torch.exp2(torch.randint(-30, 30, (N, 1), device="cuda", generator=g).float())).bfloat16()
    x = torch.randn(T, K, device="cuda", generator=g)
    x = (x * torch.exp2(torch.randint(-60, 60, (T, 1), device="cuda", generator=g).float())).bfloat16()
    want, tol = formula(x, packed, scales, G, "none")
    layer = Int4Linear(packed, scales, G)
    clean = layer.forward(x, out_dtype=torch.float32)
    check(clean, want, tol, torch.float32, f"wide range T={T}")
    if T > 2:
        x[1, 3], x[T - 1, K - 1] = math.nan, math.inf
        y = layer.forward(x, out_dtype=torch.float32)
        assert y[1].isnan().all() and y[T - 1].isnan().all()
        keep = [t for t in range(T) if t not in (1, T - 1)]
        assert torch.equal(y[keep], clean[keep])


def tables(counts, first=0, behind=0, top_k=1, seed=0):
    """offsets, a permutation of slots and the number of places of a routing with these counts."""
    off = np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)
    places = int(off[-1]) + behind
    slots = np.random.default_rng(seed).permutation(places).astype(np.int32)
    return torch.from_numpy(off).cuda(), torch.from_numpy(slots).cuda(), places


GROUPED = [
    # counts, N, K, G, out, how many places before and behind
    ([1], 40, 64, 64, "fp32", 0, 0),
    ([0, 3, 0, 1], 33, 128, 128, "fp32", 0, 0),
    ([0, 0, 0], 33, 128, 128, "fp32", 0, 4),
    ([1] * 10, 1280, 2560, 128, "bf16", 0, 0),
    ([2, 0, 5, 16, 17, 1], 100, 640, 64, "fp32", 3, 2),
    ([1, 2, 0, 33, 64, 65, 15], 257, 192, 64, "fp16", 0, 5),
    ([0] * 50 + [7] + [0] * 461, 640, 640, 128, "fp32", 0, 0),
    ([4] * 160, 64, 256, 128, "fp32", 0, 0),
    ([300, 1, 0, 129, 40], 513, 640, 64, "bf16", 1, 0),
    ([700], 300, 256, 128, "fp32", 0, 0),
    ([0, 193, 0, 192, 5, 1000], 256, 320, 64, "fp32", 0, 7),
    ([1] * 1024, 48, 64, 64, "fp32", 0, 0),
]


@pytest.mark.parametrize("counts,N,K,G,out,first,behind", GROUPED)
def test_grouped(counts, N, K, G, out, first, behind):
    E = len(counts)
    g = generator(E * 77 + N)
    off, slots, P = tables(counts, first, behind, seed=N)
    say(f"grouped E={E} places={P} N={N} K={K} G={G}")
    packed, scales = weights((E, N), K, G, g)
    top_k = 3
    x = torch.randn((P + top_k - 1) // top_k, K, device="cuda", generator=g).to(torch.bfloat16)
    xd = torch.randn(P, K, device="cuda", generator=g).to(torch.bfloat16)
    bias = torch.randn(E, N, device="cuda", generator=g)
    rw = torch.randn(P, device="cuda", generator=g)
    res = torch.randn(P, N, device="cuda", generator=g).to(TYPES[out])
    layer = Int4GroupedLinear(packed, scales, G)
    biased = Int4GroupedLinear(packed, scales, G, bias=bias, activation="silu")

    def filled():
        return inside(torch.full((P, N), 77.0, dtype=TYPES[out], device="cuda"), 3, 55.0)

    wu, up = filled()
    layer.forward(x, off, gather=slots, gather_div=top_k, out=up)
    wd, down = filled()
    layer.forward(xd, off, scatter=slots, row_weights=rw, out=down)
    wp, plain = filled()
    biased.forward(xd, off, residual=res, out=plain)
    for w in (wu, wd, wp):
        assert (w[:, N:] == 55.0).all()
    ends = off.tolist()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        mine = slots[a:b].long()
        want, tol = formula(x[mine // top_k], packed[e], scales[e], G, "none")
        check(up[a:b], want, tol, TYPES[out], f"gathered, expert {e} of {b - a}")
        want, tol = formula(xd[a:b], packed[e], scales[e], G, "none", weight=rw[mine])
        check(down[mine], want, tol, TYPES[out], f"scattered, expert {e}")
        want, tol = formula(xd[a:b], packed[e], scales[e], G, "silu", bias[e], None, res[a:b])
        check(plain[a:b], want, tol, TYPES[out], f"biased, expert {e}")
    for p in list(range(ends[0])) + list(range(ends[-1], P)):
        assert (up[p] == 77.0).all() and (plain[p] == 77.0).all() and (down[int(slots[p])] == 77.0).all()


@pytest.mark.parametrize("counts", [[1, 2, 0, 5], [40, 3, 0, 90]])
def test_grouped_rows_outside(counts):
    """A gathered row outside x counts as zeros, a scattered one outside out is not written; x may
    have more rows than there are places."""
    E, N, K, G = len(counts), 70, 256, 128
    g = generator(3)
    off, _, P = tables(counts)
    packed, scales = weights((E, N), K, G, g)
    x = torch.randn(3 * P, K, device="cuda", generator=g).to(torch.bfloat16)
    gather = torch.randint(0, 3 * P, (P,), device="cuda", generator=g).to(torch.int32)
    gather[0], gather[P // 2], gather[P - 1] = -1, 3 * P, 2**31 - 1
    scatter = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
    scatter[1], scatter[P - 2] = -5, P
    bias = torch.randn(E, N, device="cuda", generator=g)
    layer = Int4GroupedLinear(packed, scales, G, bias=bias)
    out = torch.full((P, N), 77.0, device="cuda")
    layer.forward(x, off, gather=gather, scatter=scatter, out=out)
    touched = set()
    for p in range(P):
        e = int((off[1:] <= p).sum())
        o = int(scatter[p])
        if not 0 <= o < P:
            continue
        touched.add(o)
        i = int(gather[p])
        row = x[i:i + 1] if 0 <= i < 3 * P else torch.zeros_like(x[:1])
        want, tol = formula(row, packed[e], scales[e], G, "none", bias[e])
        check(out[o:o + 1], want, tol, torch.float32, f"place {p}")
    rest = [o for o in range(P) if o not in touched]
    assert rest and (out[rest] == 77.0).all()


def test_experts_one_product_at_a_time():
    """The routing's tables, gate and up, SiLU, down and the weighted sum, against the fused layer."""
    shape = synth.TINY
    host = synth.make_layer(shape, seed=4)
    dev = synth.to_device(host, "cuda:0")
    top_k = host["top_k"]
    layer = MoeInt4Layer(dev, top_k)
    whole = layer.forward(dev["x"]).view(torch.bfloat16).float()
    r = layer.route(dev["x"])
    T = dev["x"].shape[0]
    x = dev["x"].view(torch.bfloat16)
    up = Int4GroupedLinear(dev["w13_packed"], dev["w13_scales"].view(torch.bfloat16), 128)
    down = Int4GroupedLinear(dev["w2_packed"], dev["w2_scales"].view(torch.bfloat16), 128)
    h = up.forward(x, r["offsets"], gather=r["sorted_slots"], gather_div=top_k, out_dtype=torch.float32)
    gate, lift = h.chunk(2, dim=1)
    a = (torch.nn.functional.silu(gate) * lift).to(torch.bfloat16)
    y = down.forward(a.contiguous(), r["offsets"], scatter=r["sorted_slots"], row_weights=r["weights"],
                     out_dtype=torch.float32)
    y = y.view(T, top_k, -1).sum(1)
    # the activation is rounded to bf16 here (half a step of 2^-8), to fp16 there, and out to bf16
    rms = y.square().mean().sqrt()
    err = (y - whole).abs()
    assert (err <= 2 ** -8 * (y.abs() + 4 * rms)).all(), (err.max() / rms).item()
    assert err.mean() <= 2 ** -8 * rms


def replayed(make, inputs, outs):
    """make() captured; replays with new inputs and eager work between them equal the eager results."""
    make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        make()
    for i in range(4):
        for t in inputs:
            t.copy_(torch.randn(t.shape, device="cuda", generator=generator(50 + i)).to(t.dtype))
        make()
        want = [o.clone() for o in outs]
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), f"replay {i}"


@pytest.mark.parametrize("T,N,K", [(1, 640, 640), (40, 640, 2560), (300, 512, 640)])
def test_linear_captured(T, N, K):
    g = generator(8)
    packed, scales = weights((N,), K, 128, g)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
    out = torch.empty(T, N, device="cuda")
    layer = Int4Linear(packed, scales, 128)
    replayed(lambda: layer.forward(x, out=out), [x], [out])


@pytest.mark.parametrize("counts", [[1, 0, 2], [40, 3, 0, 90] * 8])
def test_grouped_captured(counts):
    E, N, K = len(counts), 200, 256
    g = generator(9)
    off, slots, P = tables(counts)
    packed, scales = weights((E, N), K, 128, g)
    x = torch.randn(P, K, device="cuda", generator=g).to(torch.bfloat16)
    out = torch.empty(P, N, device="cuda")
    layer = Int4GroupedLinear(packed, scales, 128)
    replayed(lambda: layer.forward(x, off, scatter=slots, out=out), [x], [out])


def test_two_streams():
    """Calls in flight on two streams, each with its own workspace."""
    g = generator(10)
    N, K, T = 1024, 2560, 200
    layers = [Int4Linear(*weights((N,), K, 128, g), 128) for _ in range(2)]
    xs = [torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    want = [l.forward(x, out_dtype=torch.float32) for l, x in zip(layers, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layers[i].forward(xs[i], out_dtype=torch.float32))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
