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
