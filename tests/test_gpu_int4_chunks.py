"""The kernel of many rows behind moe_int4_linear and moe_int4_grouped_linear
over many stages of 128 inputs (its buffers of x and codes go round every two or
three) and over chunks of one to six tiles of 32 rows, and calls in flight at
the same time.  Formula and tolerance as in test_gpu_int4_linear."""
import pytest
import torch

from quantized_moe_router_amd import _binding as B
from quantized_moe_router_amd.layer import Int4GroupedLinear, Int4Linear
from test_gpu_int4_linear import check, formula, generator, say, tables, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    B.lib()
    yield


def copies_x(need, rows, k):
    """Whether a call with this workspace takes the kernel of many rows, which holds x there as
    whole stages of fp16 values with a row of zeros behind them; lists of tiles are far smaller."""
    return need >= 2 * (rows + 1) * ((k + 127) // 128 * 128)


# more than 96 rows to an expert on average: chunks of up to 192
OF_192 = [1, 33, 64, 65, 97, 128, 129, 191, 192, 193, 385]
# 32 to 96: chunks of up to 128
OF_128 = [1, 32, 33, 64, 65, 96, 97, 128, 129, 2, 31, 0, 40]


@pytest.mark.parametrize("counts,N", [(OF_192, 1700), (OF_128, 3331)])
@pytest.mark.parametrize("K,G", [(896, 64), (896, 128), (1600, 64), (1664, 128), (2560, 64), (2560, 128)])
def test_many_stages(counts, N, K, G):
    E = len(counts)
    g = generator(K + G + E)
    off, slots, P = tables(counts, seed=K)
    say(f"many stages E={E} places={P} N={N} K={K} G={G}")
    packed, scales = weights((E, N), K, G, g)
    x = torch.randn(P, K, device="cuda", generator=g).to(torch.bfloat16)
    bias = torch.randn(E, N, device="cuda", generator=g)
    rw = torch.randn(P, device="cuda", generator=g)
    layer = Int4GroupedLinear(packed, scales, G, bias=bias)
    groups = B.make_groups(P, P, P, off, scatter=slots, row_weights=rw)
    assert copies_x(B.moe_int4_grouped_linear_workspace_bytes(groups, N, K, G), P, K)
    out = torch.full((P, N), 77.0, device="cuda")
    layer.forward(x, off, scatter=slots, row_weights=rw, out=out)
    ends = off.tolist()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        mine = slots[a:b].long()
        want, tol = formula(x[a:b], packed[e], scales[e], G, "none", bias[e], rw[mine])
        check(out[mine], want, tol, torch.float32, f"expert {e} of {b - a}")
    for _ in range(3):
        again = torch.full((P, N), 77.0, device="cuda")
        layer.forward(x, off, scatter=slots, row_weights=rw, out=again)
        assert torch.equal(again, out)


@pytest.mark.parametrize("T,N,K,G", [(130, 11000, 2560, 128), (400, 5300, 1600, 64), (512, 5200, 10240, 128)])
def test_many_stages_of_one_matrix(T, N, K, G):
    g = generator(T)
    packed, scales = weights((N,), K, G, g)
    x = torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16)
    assert copies_x(B.moe_int4_linear_workspace_bytes(T, N, K, G), T, K)
    want, tol = formula(x, packed, scales, G, "none")
    layer = Int4Linear(packed, scales, G)
    out = layer.forward(x, out_dtype=torch.float32)
    check(out, want, tol, torch.float32, f"T={T} N={N} K={K} G={G}")
    for _ in range(3):
        assert torch.equal(layer.forward(x, out_dtype=torch.float32), out)


def test_many_rows_past_4_gib():
    """Many rows of the last of 40 experts, whose codes lie more than 4 GiB behind the first's."""
    E, N, K, G, rows = 40, 16384, 16384, 128, 1300
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of GPU memory")
    g = generator(44)
    packed = torch.empty(E, N, K // 8, dtype=torch.int32, device="cuda")
    for e in range(E):
        packed[e] = torch.randint(-2**31, 2**31 - 1, (N, K // 8), dtype=torch.int32, device="cuda", generator=g)
    scales = (torch.randn(E, N, K // G, device="cuda", generator=g) * 0.002).to(torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = rows
    groups = B.make_groups(rows, rows, rows, off)
    assert copies_x(B.moe_int4_grouped_linear_workspace_bytes(groups, N, K, G), rows, K)
    x = torch.randn(rows, K, device="cuda", generator=g).to(torch.bfloat16)
    out = Int4GroupedLinear(packed, scales, G).forward(x, off, out_dtype=torch.float32)
    pick = torch.arange(0, N, 97, device="cuda")
    want, tol = formula(x, packed[E - 1][pick], scales[E - 1][pick], G, "none")
    check(out[:, pick], want, tol, torch.float32, f"{rows} rows")


def in_flight(calls):
    """Each of `calls`, five times on a stream of its own, against what it answers alone."""
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, calls[i]()))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)


def test_one_layer_on_two_streams():
    """Calls of one layer in flight at the same time, whose workspaces must not be one: the copy of x differs."""
    T, N, K = 512, 6000, 1280
    g = generator(61)
    layer = Int4Linear(*weights((N,), K, 128, g), 128)
    assert copies_x(B.moe_int4_linear_workspace_bytes(T, N, K, 128), T, K)
    xs = [torch.randn(T, K, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    in_flight([lambda x=x: layer.forward(x, out_dtype=torch.float32) for x in xs])


@pytest.mark.parametrize("P,N", [(300, 1000), (1500, 1700)])
def test_one_set_of_experts_on_two_streams(P, N):
    """The same with experts, by the list of tiles and by the copy of x; the two calls' offsets differ."""
    E, K = 11, 640
    g = generator(67)
    layer = Int4GroupedLinear(*weights((E, N), K, 128, g), 128)
    x = torch.randn(P, K, device="cuda", generator=g).to(torch.bfloat16)
    offs = []
    for seed in range(2):
        ids = (torch.rand(P, device="cuda", generator=generator(seed)) ** 2 * E).long()
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0)
        offs.append(off)
    groups = B.make_groups(P, P, P, offs[0])
    need = B.moe_int4_grouped_linear_workspace_bytes(groups, N, K, 128)
    assert need > 0 and copies_x(need, P, K) == (P == 1500)
    in_flight([lambda o=o: layer.forward(x, o, out_dtype=torch.float32) for o in offs])


def test_few_places_of_the_widest_matrix():
    """128 places of 2^24 - 1 columns, 2^31 - 128 elements of out."""
    E, P, N, K, G = 5, 128, (1 << 24) - 1, 64, 64
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB of GPU memory")
    g = generator(71)
    packed, scales = weights((E, N), K, G, g)
    x = torch.randn(P, K, device="cuda", generator=g).to(torch.bfloat16)
    off = torch.tensor([0, 100, 100, 100, 101, P], dtype=torch.int32, device="cuda")
    out = torch.full((P, N), 77.0, dtype=torch.bfloat16, device="cuda")
    Int4GroupedLinear(packed, scales, G).forward(x, off, out=out)
    pick = torch.cat([torch.arange(200, device="cuda"), torch.arange(1000, N, 100003, device="cuda"),
                      torch.arange(N - 200, N, device="cuda")])
    for e, a, b in ((0, 0, 100), (3, 100, 101), (4, 101, P)):
        want, tol = formula(x[a:b], packed[e][pick], scales[e][pick], G, "none")
        check(out[a:b][:, pick], want, tol, torch.bfloat16, f"expert {e}")
    for a in range(0, P, 16):   # every element has been written: no product is near the fill
        assert (out[a:a + 16] == 77.0).sum() == 0
