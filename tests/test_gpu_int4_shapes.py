"""moe_int4_linear and moe_int4_grouped_linear at the sizes that their kernels
part at: many rows (chunks of up to 128 or 192 rows, through a copy of x), long
K, wide matrices, memory past 4 GiB, tables that are out of order.  Formula and
tolerance as in test_gpu_int4_linear."""
import math

import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import Int4GroupedLinear, Int4Linear
from test_gpu_int4_linear import TYPES, check, formula, generator, inside, replayed, say, tables, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.lib()
    yield


@pytest.mark.parametrize("T,N,K,G,out,kind,residual,strided", [
    (257, 10240, 64, 64, "fp32", "none", None, False),      # one stage, half of it
    (300, 6913, 192, 64, "fp32", "silu", "fp32", True),     # odd columns, a stage and a half
    (641, 5000, 128, 128, "bf16", "none", "bf16", False),
    (1281, 2305, 320, 64, "fp16", "gelu", "fp16", True),
    (2000, 1281, 640, 128, "fp32", "none", None, True),
    (1030, 2561, 384, 128, "fp32", "relu", None, False),    # three stages
    (4097, 700, 512, 128, "fp32", "sigmoid", "bf16", False),
    (8191, 513, 896, 64, "bf16", "gelu_tanh", None, False),   # seven stages
    (1153, 2300, 4160, 64, "fp32", "none", None, False),    # more inputs than a wave holds of a row
    (16385, 257, 128, 128, "fp32", "none", None, False),
])
def test_many_rows(T, N, K, G, out, kind, residual, strided):
    assert B.moe_int4_linear_workspace_bytes(T, N, K, G) > 0
    g = generator(T + N)
    say(f"many rows T={T} N={N} K={K} G={G}")
    packed, scales = weights((N,), K, G, g)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
    b = torch.randn(N, device="cuda", generator=g)
    r = torch.randn(T, N, device="cuda", generator=g).to(TYPES[residual]) if residual else None
    want, tol = formula(x, packed, scales, G, kind, b, None, r)
    o, wide = torch.full((T, N), 77.0, dtype=TYPES[out], device="cuda"), None
    if strided:
        _, x = inside(x, 8, math.nan)
        wide, o = inside(o, 3, 55.0)
    layer = Int4Linear(packed, scales, G, bias=b, activation=kind)
    layer.forward(x, residual=r, out=o)
    check(o, want, tol, TYPES[out], f"T={T} N={N} K={K} G={G} {out}")
    if strided:
        assert (wide[:, N:] == 55.0).all()
    again = layer.forward(x, residual=r, out_dtype=TYPES[out])
    assert torch.equal(again, o)


@pytest.mark.parametrize("T,N,K,G", [(3, 40, 65536, 64), (16, 33, 65536, 128), (1, 130, 8256, 64), (40, 2100, 4096, 128),
                                     (1, 70001, 128, 128), (2, 70001, 64, 64), (20, 40000, 192, 64)])
def test_long_and_wide(T, N, K, G):
    g = generator(K)
    packed, scales = weights((N,), K, G, g)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
    want, tol = formula(x, packed, scales, G, "none")
    check(Int4Linear(packed, scales, G).forward(x, out_dtype=torch.float32), want, tol, torch.float32, f"T={T} N={N} K={K}")


@pytest.mark.parametrize("T,N", [(5, 300), (40, 2600), (400, 7000)])
@pytest.mark.parametrize("G", [64, 128])
def test_scales_of_a_row_far_apart(T, N, G):
    """Groups of a row whose scales lie up to 2^20 apart, tokens whose inputs do, and rows of all-zero scales."""
    K = 1280
    g = generator(17)
    packed, scales = weights((N,), K, G, g)
    far = torch.exp2(torch.randint(-10, 11, scales.shape, device="cuda", generator=g).float())
    scales = (scales.float() * far).bfloat16()
    scales[3], scales[N - 1] = 0.0, 0.0
    scales[5, 1:] = 0.0
    x = torch.randn(T, K, device="cuda", generator=g)
    x = (x * torch.exp2(torch.randint(-10, 11, (T, K // 64), device="cuda", generator=g).float()).repeat_interleave(64, 1)).bfloat16()
    x[T - 1] = 0.0
    want, tol = formula(x, packed, scales, G, "none")
    check(Int4Linear(packed, scales, G).forward(x, out_dtype=torch.float32), want, tol, torch.float32, f"T={T} G={G}")


@pytest.mark.parametrize("T,N", [(9, 500), (300, 9000)])
def test_inputs_of_one_sign(T, N):
    """x >= 0, as behind an activation: what the codes' offset of 24 adds is taken off before
    anything else is added.  Its sums are at most 24 sum |x| of a group, and 2 G roundings of them
    come to at most 6 sqrt(2 G) u times that, against the codes' own few."""
    K, G = 2560, 128
    g = generator(23)
    packed, scales = weights((N,), K, G, g)
    x = torch.randn(T, K, device="cuda", generator=g).abs().to(torch.bfloat16)
    want, tol = formula(x, packed, scales, G, "none")
    sums = x.double().view(T, -1, G).sum(2).square()
    extra = 6 * math.sqrt(2 * G) * 2.0 ** -24 * 24 * torch.mm(sums, scales.double().square().t().contiguous()).sqrt()
    check(Int4Linear(packed, scales, G).forward(x, out_dtype=torch.float32), want, tol + extra, torch.float32, f"T={T}")


@pytest.mark.parametrize("T,N", [(300, 9000), (700, 5001)])
def test_nonfinite_tokens_of_many(T, N):
    K = 256
    g = generator(29)
    packed, scales = weights((N,), K, 128, g)
    x = (torch.randn(T, K, device="cuda", generator=g) * torch.exp2(
        torch.randint(-100, 90, (T, 1), device="cuda", generator=g).float())).bfloat16()
    want, tol = formula(x, packed, scales, 128, "none")
    layer = Int4Linear(packed, scales, 128)
    clean = layer.forward(x, out_dtype=torch.float32)
    check(clean, want, tol + 2.0 ** -149, torch.float32, f"T={T}")   # down to fp32's smallest
    x[1, 3], x[T - 1, K - 1] = math.nan, -math.inf
    y = layer.forward(x, out_dtype=torch.float32)
    assert y[1].isnan().all() and y[T - 1].isnan().all()
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("counts,N,K,G,out,first,behind", [
    ([300, 0, 129, 700], 2560, 320, 64, "fp32", 3, 5),       # chunks of up to 192 rows
    ([193, 192, 97, 96, 95, 33, 0, 1], 3100, 128, 128, "bf16", 0, 0),
    ([60, 0, 31, 33, 129, 64, 1, 0] * 4, 1800, 192, 64, "fp32", 0, 9),
    ([40] * 64, 1100, 256, 128, "fp16", 0, 0),
    ([1000], 2900, 448, 64, "fp32", 2, 0),
    ([20] * 30, 700, 384, 128, "fp32", 0, 3),                # listed, sixteen rows a tile
])
def test_grouped_many_rows(counts, N, K, G, out, first, behind):
    E = len(counts)
    g = generator(E * 5 + N)
    off, slots, P = tables(counts, first, behind, seed=K)
    say(f"grouped E={E} places={P} N={N} K={K} G={G}")
    packed, scales = weights((E, N), K, G, g)
    top_k = 4
    x = torch.randn((P + top_k - 1) // top_k, K, device="cuda", generator=g).to(torch.bfloat16)
    xd = torch.randn(P, K, device="cuda", generator=g).to(torch.bfloat16)
    bias = torch.randn(E, N, device="cuda", generator=g)
    rw = torch.randn(P, device="cuda", generator=g)
    layer = Int4GroupedLinear(packed, scales, G, bias=bias)
    up = torch.full((P, N), 77.0, dtype=TYPES[out], device="cuda")
    down = up.clone()
    layer.forward(x, off, gather=slots, gather_div=top_k, out=up)
    layer.forward(xd, off, scatter=slots, row_weights=rw, out=down)
    ends = off.tolist()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        mine = slots[a:b].long()
        want, tol = formula(x[mine // top_k], packed[e], scales[e], G, "none", bias[e])
        check(up[a:b], want, tol, TYPES[out], f"gathered, expert {e} of {b - a}")
        want, tol = formula(xd[a:b], packed[e], scales[e], G, "none", bias[e], rw[mine])
        check(down[mine], want, tol, TYPES[out], f"scattered, expert {e}")
    for p in list(range(ends[0])) + list(range(ends[-1], P)):
        assert (up[p] == 77.0).all() and (down[int(slots[p])] == 77.0).all()


@pytest.mark.parametrize("more", [0, 5000])
def test_grouped_many_rows_outside(more):
    """Rows of x and out outside their operands, in the kernel of many rows; x with more rows than places."""
    counts, N, K, G = [200, 0, 300, 77], 4100, 256, 128
    E = len(counts)
    g = generator(31)
    off, _, P = tables(counts)
    rows = P + more
    packed, scales = weights((E, N), K, G, g)
    x = torch.randn(rows, K, device="cuda", generator=g).to(torch.bfloat16)
    gather = torch.randint(0, rows, (P,), device="cuda", generator=g).to(torch.int32)
    gather[0], gather[P // 2], gather[P - 1] = -1, rows, 2**31 - 1
    scatter = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
    scatter[1], scatter[P - 2] = -5, P
    layer = Int4GroupedLinear(packed, scales, G)
    out = torch.full((P, N), 77.0, device="cuda")
    layer.forward(x, off, gather=gather, scatter=scatter, out=out)
    inside_x = (gather >= 0) & (gather < rows)
    taken = x[gather.clamp(0, rows - 1).long()] * inside_x.unsqueeze(1)
    ends = off.tolist()
    untouched = torch.ones(P, dtype=torch.bool, device="cuda")
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        want, tol = formula(taken[a:b], packed[e], scales[e], G, "none")
        to = scatter[a:b].long()
        ok = (to >= 0) & (to < P)
        check(out[to[ok]], want[ok], tol[ok], torch.float32, f"expert {e}")
        untouched[to[ok]] = False
    assert untouched.any() and (out[untouched] == 77.0).all()


def test_a_row_of_x_for_many_places():
    """Every place gathers the same row."""
    counts, N, K = [100, 30, 0, 70], 1000, 256
    g = generator(37)
    off, _, P = tables(counts)
    packed, scales = weights((4, N), K, 128, g)
    x = torch.randn(3, K, device="cuda", generator=g).to(torch.bfloat16)
    gather = torch.full((P,), 2, dtype=torch.int32, device="cuda")
    out = Int4GroupedLinear(packed, scales, 128).forward(x, off, gather=gather, out_dtype=torch.float32)
    ends = off.tolist()
    for e in (0, 1, 3):
        want, tol = formula(x[2:3], packed[e], scales[e], 128, "none")
        check(out[ends[e]:ends[e + 1]], want.expand(counts[e], -1), tol.expand(counts[e], -1), torch.float32, f"expert {e}")


@pytest.mark.parametrize("E,P,N", [(6, 40, 100), (40, 300, 200), (5, 900, 3000)])
def test_offsets_out_of_order(E, P, N):
    """Offsets that decrease, pass the places or are negative: rows beside the operands stay as they were."""
    K = 128
    g = generator(41)
    packed, scales = weights((E, N), K, 128, g)
    x = torch.randn(P, K, device="cuda", generator=g).to(torch.bfloat16)
    layer = Int4GroupedLinear(packed, scales, 128)
    for seed in range(4):
        off = torch.randint(-P, 2 * P, (E + 1,), device="cuda", generator=generator(seed)).to(torch.int32)
        off[seed % (E + 1)] = (2**31 - 1, -2**31, 0, P)[seed]
        guard = torch.full((P + 8, N), 55.0, device="cuda")
        layer.forward(x, off, out=guard[4:P + 4])
        torch.cuda.synchronize()
        assert (guard[:4] == 55.0).all() and (guard[P + 4:] == 55.0).all()


def test_matrices_past_4_gib():
    """The last of 40 experts, whose codes lie more than 4 GiB behind the first's."""
    E, N, K, G = 40, 16384, 16384, 128
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of GPU memory")
    g = generator(43)
    packed = torch.empty(E, N, K // 8, dtype=torch.int32, device="cuda")
    for e in range(E):
        packed[e] = torch.randint(-2**31, 2**31 - 1, (N, K // 8), dtype=torch.int32, device="cuda", generator=g)
    scales = (torch.randn(E, N, K // G, device="cuda", generator=g) * 0.002).to(torch.bfloat16)
    layer = Int4GroupedLinear(packed, scales, G)
    for rows in (3, 200):
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = rows
        x = torch.randn(rows, K, device="cuda", generator=g).to(torch.bfloat16)
        out = layer.forward(x, off, out_dtype=torch.float32)
        pick = torch.arange(0, N, 97, device="cuda")
        want, tol = formula(x, packed[E - 1][pick], scales[E - 1][pick], G, "none")
        check(out[:, pick], want, tol, torch.float32, f"{rows} rows")


@pytest.mark.parametrize("T,N,K", [(512, 6000, 640), (20, 30000, 256)])
def test_more_captured(T, N, K):
    g = generator(47)
    packed, scales = weights((N,), K, 128, g)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
    res = torch.randn(T, N, device="cuda", generator=g)
    out = torch.empty(T, N, device="cuda")
    layer = Int4Linear(packed, scales, 128, activation="silu")
    replayed(lambda: layer.forward(x, residual=res, out=out), [x, res], [out])


def test_grouped_many_captured_with_new_tables():
    """Replays with new offsets and slots, of which the launches know nothing."""
    E, N, K, P = 16, 3000, 256, 1024
    g = generator(53)
    packed, scales = weights((E, N), K, 128, g)
    x = torch.randn(P, K, device="cuda", generator=g).to(torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(P, dtype=torch.int32, device="cuda")
    out = torch.empty(P, N, device="cuda")
    layer = Int4GroupedLinear(packed, scales, 128)

    def tables_of(seed):
        h = generator(seed)
        ids = (torch.rand(P, device="cuda", generator=h) ** 2 * E).long()
        off[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0)
        slots.copy_(torch.sort(ids, stable=True).indices)

    def call():
        layer.forward(x, off, scatter=slots, out=out)

    tables_of(0)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        tables_of(i + 1)
        call()
        want = out.clone()
        torch.cuda.synchronize()
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
