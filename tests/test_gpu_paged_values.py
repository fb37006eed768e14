"""kvd_paged_attn where values are not tame: NaN and infinite queries, one key with nearly all the
weight, value scales of very different size, and neighbours whose rows share a tile."""
import math

import pytest
import torch

import long_context_decode_kv_gb300 as kvd
import paged_ref as R
from test_gpu_paged import DEV, X, _attend, _cache, _q, _starts

pytestmark = pytest.mark.gpu
# new tokens and length of one sequence of 4 heads a KV head: the kernel for few rows, 128 rows and
# row tiles in pairs, each with its item whole and cut between CTAs
SHAPES = [(1, 60), (1, 30000), (8, 300), (8, 20000), (20, 100), (20, 9000), (300, 400), (300, 9000)]


def _x(dtype):
    return X.get(dtype, torch.bfloat16)


# ------------------------------------------------------- NaN and infinities ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("new,L", SHAPES)
def test_a_query_that_is_not_finite_gives_a_nan_row(dtype, new, L):
    """And leaves the others as they are, wherever the item is cut."""
    c = _cache(dtype, [L], 2, 128, 64, L)
    q = _q(new, 8, 128, _x(dtype), new)
    q[0, 1, 5] = math.nan
    q[new // 2, 6, 127] = math.inf
    q[new - 1, 3] = math.nan
    out = _attend(c, q, [new])
    want, tol = R.attn_ref(c, q, [0, new], [L], 128 ** -0.5)
    bad = ~torch.isfinite(q).all(-1)
    assert bool(torch.isnan(out[bad]).all())
    R.assert_within(out[~bad], want[~bad], tol[~bad])
    assert c.device_status() == 0


# --------------------------------------------------------------- neighbours ---

@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("G,new", [(4, [1, 8]), (7, [2, 4]), (4, [9, 30]), (7, [5, 18]), (4, [20, 200]),
                                   (3, [50, 300]), (7, [25, 90])])
def test_a_sequence_does_not_depend_on_its_neighbour(dtype, G, new):
    """The tile's rows behind a sequence's last are the next one's queries, or none's."""
    c = _cache(dtype, [2000, 2300], 2, 128, 64, G)
    q = _q(sum(new), 2 * G, 128, _x(dtype), G)
    n = new[0]
    first = _attend(c, q, new)[:n]
    for other in (300.0, 0.0, math.nan):
        p = q.clone()
        p[n:] *= other
        assert torch.equal(_attend(c, p, new)[:n], first)


@pytest.mark.parametrize("dtype", [kvd.F16, kvd.BF16, kvd.INT8])
@pytest.mark.parametrize("G,new", [(7, 4), (4, 20), (3, 11), (7, 200), (6, 300)])
def test_a_call_does_not_depend_on_the_one_before(dtype, G, new):
    """Rows of a tile that hold no query, after calls whose queries filled them with large values."""
    c = _cache(dtype, [3000], 2, 128, 64, G + new)
    q = _q(new, 2 * G, 128, _x(dtype), new)
    first = _attend(c, q, [new])
    for scale in (1e3, math.nan):
        for g, n in ((G, new), (8, 16), (8, 200), (16, 2)):
            _attend(c, torch.full((n, 2 * g, 128), scale, dtype=q.dtype, device=DEV), [n])
        assert torch.equal(_attend(c, q, [new]), first)
