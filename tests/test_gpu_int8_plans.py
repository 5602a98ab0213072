"""moe_int8_linear_fused kernel by kernel: shapes that provably run each of
them (the plan is asked of the built library) where a shape chosen by size
alone might come to another, and what only some shapes of a kernel reach.

Tolerances as in test_gpu_int8_fused.py."""
import ctypes
import math
import sys

import numpy as np
import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import Int8Linear
from test_gpu_int8_fused import TYPES, U, case, check, expected, inside, run

gpu = pytest.mark.gpu
CUS = 256


def say(*a):
    print(*a, file=sys.stderr, flush=True)


class Plan(ctypes.Structure):
    """Int8Plan of csrc/common.h."""
    _fields_ = ([(f, ctypes.c_bool) for f in ("gemv", "rowsplit", "mfma", "short_k")]
                + [(f, ctypes.c_int) for f in ("mtiles", "ntiles", "ksplit", "kslice")]
                + [(f, ctypes.c_size_t) for f in ("pstride", "part_bytes")]
                + [(f, ctypes.c_bool) for f in ("wide", "kwaves")])


def plan(T, N, K, G):
    f = B.lib()._ZN3moe15int8_fused_planEiiii
    f.restype, f.argtypes = Plan, [ctypes.c_int] * 4
    return f(T, N, K, G)


def kernel(T, N, K, G):
    p = plan(T, N, K, G)
    if p.wide:
        return "wide"
    if p.gemv:
        return "rowsplit" if p.rowsplit else "mfma" if p.mfma else "gemv"
    if p.short_k:
        return "short"
    return ("kwaves" if p.kwaves else "gemm") + (" split" if p.ksplit > 1 else "")


def wide_blocks(T, N, K):
    """Row blocks of the wave that has most (two workgroups of eight waves to a
    CU, one where the activations take most of its LDS)."""
    most = (2 if T * (K // 8 + 1) * 16 <= 57344 else 1) * CUS * 8
    return -(-(-(-N // 16)) // most)


# ---------------------------------------------------------------------------
# The GEMM of many tiles, rows with aligned words: ragged last tiles of one to
# four runs of 32 tokens, columns of a last tile that is not full, every
# activation, each type in each place, more scale groups than are staged at a
# time, and K over workgroups.
# ---------------------------------------------------------------------------
GEMM = [
    # (T, N, K, G, bias, activation, residual, out, strided)
    (1100, 1280, 384, 64, "bf16", "silu", "fp32", "fp32", False),
    (1030, 1284, 384, 128, "fp32", "gelu", "fp16", "bf16", False),
    (1024, 1152, 384, 64, None, "none", "bf16", "bf16", True),
    (1061, 1156, 384, 128, "fp16", "gelu_tanh", None, "fp16", True),
    (1217, 1408, 384, 64, None, "sigmoid", "fp32", "fp16", False),
    (1249, 1028, 384, 128, "bf16", "relu", "bf16", "fp32", True),
    (2100, 2048, 640, 128, None, "none", None, "fp32", False),
    (2050, 2052, 512, 64, "fp32", "none", "fp32", "fp32", True),
    (2100, 2048, 4224, 64, "bf16", "silu", "bf16", "fp32", False),
]
SPLIT = [
    (1024, 320, 10240, 64, "bf16", "silu", None, "bf16", False),
    (1024, 320, 10240, 64, None, "none", "fp32", "fp32", True),
    (900, 324, 10240, 128, "fp32", "gelu", "fp16", "fp16", False),
    (600, 968, 2688, 64, "fp16", "sigmoid", "bf16", "fp32", True),
    (1500, 1280, 1280, 128, None, "gelu_tanh", "fp32", "bf16", False),
]
# more blocks than waves; the steps of 128 inputs no multiple of the four that
# are on their way; a second, partial chunk of 16 scale groups
WIDE = [
    (5, 70003, 640, 64, "bf16", "silu", "bf16", "fp32"),
    (8, 66001, 2560, 128, None, "none", None, "fp32"),
    (16, 70001, 640, 128, "fp32", "none", "fp32", "bf16"),
    (16, 66003, 2688, 64, None, "gelu", None, "fp32"),
    (5, 140001, 1408, 64, "fp16", "none", "fp16", "fp16"),
    (3, 66004, 1152, 128, None, "sigmoid", None, "fp32"),
    (12, 35001, 4224, 64, "bf16", "none", "bf16", "fp32"),
    (8, 131104, 896, 128, "bf16", "relu", None, "bf16"),
]


@pytest.mark.parametrize("shape", sorted({c[:4] for c in GEMM + SPLIT + WIDE}))
def test_the_shapes_run_the_kernels_they_are_here_for(shape):
    T, N, K, G = shape
    if any(c[:4] == shape for c in WIDE):
        assert kernel(*shape) == "wide"
        assert wide_blocks(T, N, K) > 1
    else:
        assert kernel(*shape) == ("gemm" if any(c[:4] == shape for c in GEMM) else "gemm split")
        assert N % 4 == 0
    if shape == (2100, 2048, 4224, 64):
        assert K // G > 64


def aligned_rows(d, T, N):
    """x, residual and out inside wider rows that keep four columns on a word."""
    wide_x, d["x"] = inside(d["x"], 24, math.nan)
    wide, d["out"] = inside(d["out"], 12, 55.0)
    if d["residual"] is not None:
        _, d["residual"] = inside(d["residual"], 8, math.nan)
    return wide


@gpu
@pytest.mark.parametrize("T,N,K,G,bias,kind,residual,out,strided", GEMM + SPLIT)
def test_gemm_aligned_rows(T, N, K, G, bias, kind, residual, out, strided):
    label = f"{kernel(T, N, K, G)} T={T} N={N} K={K} G={G} {bias} {kind} {residual}->{out} {strided}"
    say(label)
    layer, d = case(T, N, K, G, bias, residual, out, False, seed=T + N)
    wide = aligned_rows(d, T, N) if strided else None
    got = run(d, kind)
    torch.cuda.synchronize()
    # the first, the last and both sides of the tiles' and passes' edges
    toks = np.unique(np.concatenate([[0, 31, 32, 63, 64, 127, 128, T - 2, T - 1, T // 128 * 128 - 1, T // 128 * 128],
                                     np.random.default_rng(T).choice(T, 24, replace=False)]).clip(0, T - 1))
    want, err = expected(layer, d, kind, toks)
    check(got[torch.from_numpy(toks).cuda()], want, err, TYPES[out], label)
    assert bool(torch.isfinite(got).all()) and not bool((got == 77.0).all(1).any())
    if strided:
        assert bool((wide[:, N:] == 55.0).all())


@gpu
@pytest.mark.parametrize("T,N,K,G", [(1100, 1280, 384, 64), (1030, 1284, 384, 128), (1024, 320, 10240, 64),
                                     (8, 66001, 2560, 128), (100, 1284, 320, 64), (2100, 1284, 320, 64)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_residual_in_place(T, N, K, G, out):
    label = f"in place, {kernel(T, N, K, G)} T={T} N={N} K={K} {out}"
    say(label)
    layer, d = case(T, N, K, G, "bf16", out, out, False, seed=T + 2 * N)
    rows = np.unique(np.random.default_rng(N).choice(N, min(N, 1200), replace=False))
    toks = np.unique(np.random.default_rng(T).choice(T, min(T, 30), replace=False))
    sub, ds = pick_rows(layer, d, rows)
    want, err = expected(sub, ds, "silu", toks)
    d["out"] = d["residual"]
    got = run(d, "silu")
    torch.cuda.synchronize()
    check(got[torch.from_numpy(toks).cuda()][:, torch.from_numpy(rows).cuda()], want, err, TYPES[out], label)


def pick_rows(layer, d, rows):
    """The layer and its data of some weight rows alone."""
    at = torch.from_numpy(rows).cuda()
    sub = {**layer, "packed": np.ascontiguousarray(layer["packed"][rows]),
           "scales": np.ascontiguousarray(layer["scales"][rows])}
    ds = {**d, "bias": None if d["bias"] is None else d["bias"][at],
          "residual": None if d["residual"] is None else d["residual"][:, at].clone()}
    return sub, ds


@gpu
@pytest.mark.parametrize("T,N,K,G,bias,kind,residual,out", WIDE)
def test_wide_gemv_of_several_blocks_per_wave(T, N, K, G, bias, kind, residual, out):
    label = f"wide T={T} N={N} K={K} G={G} {bias} {kind} {residual}->{out}"
    say(label)
    layer, d = case(T, N, K, G, bias, residual, out, False, seed=N)
    got = run(d, kind)
    torch.cuda.synchronize()
    # a row of every block of 16, each place in turn, and the last blocks whole
    rows = np.unique(np.concatenate([(np.arange(0, N, 16) + np.arange(-(-N // 16)) % 16).clip(max=N - 1),
                                     np.arange(max(0, N - 200), N)]))
    sub, ds = pick_rows(layer, d, rows)
    want, err = expected(sub, ds, kind)
    check(got[:, torch.from_numpy(rows).cuda()], want, err, TYPES[out], label)
    assert bool(torch.isfinite(got).all())


# ---------------------------------------------------------------------------
# Every kernel
# ---------------------------------------------------------------------------
EVERY = {"rowsplit": (3, 72, 1152, 128), "gemv": (4, 260, 320, 64), "mfma": (9, 260, 320, 64),
         "wide": (9, 8196, 640, 128), "short": (150, 2600, 320, 64), "kwaves": (70, 260, 1152, 128),
         "kwaves split": (64, 160, 10240, 64), "gemm": (1100, 1280, 384, 64), "gemm split": (1024, 320, 5120, 64)}


@pytest.mark.parametrize("name", EVERY)
def test_every_kernel_has_a_shape(name):
    assert kernel(*EVERY[name]) == name


@gpu
@pytest.mark.parametrize("name", EVERY)
def test_repeated_calls_agree_in_every_bit(name):
    T, N, K, G = EVERY[name]
    say(name)
    _, d = case(T, N, K, G, "fp32", "fp32", "fp32", False, seed=3)
    first = run(d, "silu").clone()
    for i in range(20):
        d["out"].fill_(float(i))
        if i % 3 == 0:
            torch.randn(1 << 18, device="cuda").sort()   # other kernels leave LDS and caches otherwise
        assert torch.equal(run(d, "silu"), first), f"{name}: call {i} differs"


def as_fp16_toward_zero(x):
    """What the activations are taken as: fp16, rounded toward zero, at most
    65504 in magnitude."""
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -60))), -14) - 10)
    return np.clip(np.trunc(x / step) * step, -65504, 65504)


@gpu
@pytest.mark.parametrize("name", EVERY)
def test_activations_beyond_the_normal_range_of_fp16(name):
    T, N, K, G = EVERY[name]
    say(name)
    layer, d = case(T, N, K, G, None, None, "fp32", False, seed=11)
    rng = np.random.default_rng(T)
    x = d["x"].double().cpu().numpy()
    x[0] = rng.standard_normal(K) * 2.0 ** -18                      # fp16's subnormal numbers
    x[1] = np.exp2(rng.uniform(-30, 20, K)) * rng.choice([-1, 1], K)   # all of its range and beyond
    d["x"] = torch.from_numpy(x).to(torch.bfloat16).cuda()
    x = d["x"].double().cpu().numpy()
    got = run(d, "none")
    torch.cuda.synchronize()
    toks = np.unique(np.concatenate([[0, 1, 2, T - 1], rng.choice(T, min(T, 20), replace=False)]))
    rows = np.unique(rng.choice(N, min(N, 600), replace=False))
    q = layer["packed"][rows].view(np.uint8).astype(np.float64) - 128
    s = (layer["scales"][rows].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    w = q * np.repeat(s, G, axis=1)
    h = as_fp16_toward_zero(x[toks])
    # fp16 values this time: only the sums' roundings are left
    err = (G + 2 * K // G + 32) * U * (np.abs(h) @ np.abs(w).T)
    check(got[torch.from_numpy(toks).cuda()][:, torch.from_numpy(rows).cuda()], h @ w.T, err, torch.float32, name)


@gpu
@pytest.mark.parametrize("name", EVERY)
def test_infinities_and_nan_stay_in_their_token(name):
    T, N, K, G = EVERY[name]
    say(name)
    _, d = case(T, N, K, G, None, None, "fp32", False, seed=12)
    clean = run(d, "none").clone()
    d["x"][0, 1::7] = math.nan
    d["x"][T - 1, K - 1] = math.inf
    got = run(d, "none")
    torch.cuda.synchronize()
    assert bool(got[0].isnan().all())
    assert not bool(torch.isfinite(got[T - 1]).any())    # infinite, or NaN where the code is zero
    assert torch.equal(got[1:T - 1], clean[1:T - 1])


@gpu
@pytest.mark.parametrize("name", EVERY)
def test_graph_replays_of_every_kernel_in_place(name):
    # the residual stream updated in place by replays: out is the residual
    T, N, K, G = EVERY[name]
    say(name)
    _, d = case(T, N, K, G, "bf16", "fp32", "fp32", False, seed=13)
    lin = Int8Linear(d["packed"], d["scales"], G, bias=d["bias"], activation="gelu_tanh")
    stream, start = d["residual"].clone(), d["residual"].clone()
    lin.forward(d["x"], residual=stream, out=stream)
    stream.copy_(start)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin.forward(d["x"], residual=stream, out=stream)
    want = start.clone()
    for i in range(4):
        want = lin.forward(d["x"], residual=want, out_dtype=torch.float32)   # eager work between the replays
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(stream, want), f"{name}: replay {i}"
