"""Edges of the 8-bit K/V cache: what lies beside a sequence, blocks that no write has filled, extreme scales and sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _kv8 import attend64, bounds  # noqa: E402
from test_gpu_kv8 import BF16, F32, Both  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code,dtype", [("int8", BF16), ("e4m3", F32)])
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 4), (64, 12), (256, 3)])
@pytest.mark.parametrize("scales", [float("nan"), 0.0, -1.0])
def test_a_sequence_that_no_write_has_filled_leaves_its_neighbours_alone(code, dtype, dim, group, scales):
    """Its scales and codes are what lay in the pool.  The others' tiles end at odd and even places of the warps' shares."""
    b = Both(code, heads=3, dim=dim, page=16, dtype=dtype, n_pages=500, seqs=21, max_pages=200, seed=group)
    for t in (b.cache.k_scale, b.cache.v_scale):
        t.fill_(scales)
    for t in (b.cache.k, b.cache.v):
        t.fill_(-1)
    lens = list(range(1, 580, 31))
    n = len(lens)
    b.append(range(n), lens)
    b.cache.extend(b.ids([20]), each=40)
    q = b.rand(n, 3 * group, dim)
    beside = [x for i in range(n) for x in (i, 20)]
    out, lse = b.cache.attend(0, b.ids(beside), q.repeat_interleave(2, 0).cuda(), lse=True)
    b.cache.check()
    for i in range(n):
        ref = attend64(b.seqs[i], 0, q[i:i + 1].double().numpy(), group, dim ** -0.5, -1, 1, 0, 16)
        tol, tol_lse = bounds(*ref, dim, lens[i], dtype)
        assert (np.abs(out[2 * i:2 * i + 1].double().cpu().numpy() - ref[0]) <= tol).all(), i
        assert (np.abs(lse[2 * i:2 * i + 1].double().cpu().numpy() - ref[1]) <= tol_lse).all(), i
