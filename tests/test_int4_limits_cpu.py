"""Sizes and queries of the INT4 products at their documented limits: on the
host alone, no GPU needed."""
import ctypes

import pytest

from quantized_moe_router_amd import _binding as B

TABLE = 1 << 24   # never dereferenced


def need(n, k=64, group=64, **u):
    g = B.MoeGroups(**{**dict(offsets=TABLE, gather=None, scatter=None, row_weights=None, gather_div=1), **u})
    b = ctypes.c_size_t(0)
    assert B.lib().moe_int4_grouped_linear_workspace_bytes(ctypes.byref(g), n, k, group, ctypes.byref(b)) == B.OK, \
        B.lib().moe_int4_last_error().decode()
    return b.value


@pytest.mark.parametrize("experts,places", [(5, 128), (32, 128), (1, 128)])
def test_few_places_of_the_widest_matrix(experts, places):
    """A workgroup of 256 for each of 128 places and 128 of 2^24 - 1 columns would be 2^32 threads, which no
    launch takes; with a list of tiles (held in the workspace) there are far fewer."""
    n = (1 << 24) - 1
    bytes_ = need(n, experts=experts, places=places, x_rows=places, out_rows=places)
    tiles = places // 16 + min(experts, places)
    assert bytes_ >= 16 * (tiles + 1)
    assert 256 * tiles * ((n + 127) // 128) < 1 << 32


def test_few_places_of_narrower_matrices_need_none():
    assert need(248320, k=2560, group=128, experts=512, places=128, x_rows=128, out_rows=128) == 0
    assert need(1280, k=2560, group=128, experts=512, places=10, x_rows=10, out_rows=10) == 0


@pytest.mark.parametrize("experts,places,x_rows,n,k", [
    (4, 1000, 1000, 320, 2560),       # the list of tiles
    (512, 640, 64, 1280, 2560),       # fewer rows of x than places: a later gather names them
    (512, 81920, 8192, 1280, 2560),   # the copy of x, a chunk more for each expert
    (4, 1000, 4000, 5120, 2560),      # x with more rows than places
    (8, 40, 40, 320, 640),            # none needed
])
def test_workspace_needs_no_tables(experts, places, x_rows, n, k):
    """A program that allots its workspace before its tables exist gets what the call asks for."""
    sizes = dict(experts=experts, places=places, x_rows=x_rows, out_rows=places)
    want = need(n, k, 128, gather=2 * TABLE, scatter=3 * TABLE, row_weights=4 * TABLE, **sizes)
    assert need(n, k, 128, offsets=None, **sizes) == want
    assert (want > 0) == (places > 128)
    assert need(n, k, 128, offsets=None, **{**sizes, "out_rows": 7}) == want   # rows that a later scatter names


def test_the_call_needs_its_tables():
    """What the query leaves open is checked by the call."""
    def call(**u):
        g = B.MoeGroups(**{**dict(offsets=TABLE, gather=None, scatter=None, row_weights=None, experts=4, places=20,
                                  gather_div=1, x_rows=20, out_rows=20), **u})
        return B.lib().moe_int4_grouped_linear(2 * TABLE, 2560, 3 * TABLE, 4 * TABLE, ctypes.byref(g), 320, 2560, 64,
                                               None, 5 * TABLE, B.TYPE_BF16, 320, None, 0, None)

    for u, msg in ((dict(offsets=None), "offsets is NULL"), (dict(x_rows=2), "x_rows=2"), (dict(out_rows=2), "out_rows=2"),
                   (dict(gather=TABLE, gather_div=0), "gather_div=0")):
        assert call(**u) == B.EINVAL and msg in B.lib().moe_int4_last_error().decode()
