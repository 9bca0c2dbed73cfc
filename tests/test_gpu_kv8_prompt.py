"""Attention over the 8-bit K/V cache by the kernel for many query rows, against the plain model in 64 bits.  Which kernel
answers a call depends on how it fills the card, so every test here asserts that it was this one."""
import warnings

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _kv8 import attend64, bounds  # noqa: E402
from test_gpu_kv8 import BF16, F32, Both  # noqa: E402

pytestmark = pytest.mark.gpu


class Prompts(Both):
    """A cache whose attention calls have to be answered by kv_prompt_kernel: each is captured first, and the graph's kernels
    are looked at."""

    def __init__(self, tmp_path, *args, **kw):
        super().__init__(*args, **kw)
        attend, path = self.cache.attend, str(tmp_path / "call.dot")

        def checked(*args, **kw):
            graph = torch.cuda.CUDAGraph(keep_graph=True)
            graph.enable_debug_mode()
            with torch.cuda.graph(graph):
                attend(*args, **kw)
            with warnings.catch_warnings():
                warnings.simplefilter("ignore")      # it warns that it writes a file
                graph.debug_dump(path)
            with open(path) as f:
                dot = f.read()
            assert "kv_prompt_kernel" in dot and "kv_attend_kernel" not in dot
            return attend(*args, **kw)

        self.cache.attend = checked


@pytest.mark.parametrize("dim,heads", [(64, 8), (128, 6), (16, 8)])
def test_maxima_that_jump_where_sums_are_flushed(tmp_path, dim, heads):
    """fp32 sums move to their second place every 256 tokens; here the logits of each 256 tokens lie a few powers of two
    above (or below) those before, so that the sums are rescaled just there."""
    b = Prompts(tmp_path, heads=heads, dim=dim, page=64, dtype=F32, n_pages=40, max_pages=20)
    tokens = 1100
    gen = torch.Generator().manual_seed(dim)
    line = torch.randn(dim, generator=gen)
    line /= line.norm()
    level = torch.tensor([0.0, 1.0, 2.0, 1.5, 3.0])[torch.arange(tokens) // 256]
    b.append([0], [tokens], k=b.rand(tokens, heads, dim, gain=0.05) + level[:, None, None] * line)
    step = torch.tensor([4.0, 6.0, 3.0, 10.0, -5.0])[torch.arange(tokens) % 5]      # powers of two a level
    q = (step * 0.6931 * dim ** 0.5)[:, None, None] * line.expand(tokens, heads, dim)
    b.attend([0], [tokens], group=1, q=q.contiguous())


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,page,group", [(64, 48, 4), (128, 32, 3), (80, 16, 5), (16, 64, 8)])
def test_ragged_rows(tmp_path, code, dtype, dim, page, group):
    """As many queries as keys and fewer, odd counts: row tiles whose last warp, or last row tile, is not full."""
    b = Prompts(tmp_path, code, heads=8, dim=dim, page=page, dtype=dtype, n_pages=100, seed=dim)
    lens = [131, 260, 1, 77, 16]
    b.append(range(5), lens)
    b.attend(range(5), lens, group=group)
    b.attend([3, 1, 4, 0], [59, 201, 16, 123], group=group)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-44, -0.3])
def test_scales_of_zero_and_below(tmp_path, dtype, scale):
    b = Prompts(tmp_path, heads=8, dim=64, page=16, dtype=dtype, n_pages=100)
    b.append([0, 1], [150, 60])
    b.attend([0, 1], [150, 60], group=4, scale=scale)
    b.attend([0, 1], [150, 60], group=4, scale=scale, left=20, sinks=3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("keys", [0.0, 1e-38, 1e-6, 1e-3, 1.0])
def test_queries_of_zeros(tmp_path, dtype, keys):
    """Padding: rows of zeros, over keys of zeros and of tiny values, beside rows that are not."""
    b = Prompts(tmp_path, heads=8, dim=64, page=16, dtype=dtype, n_pages=100)
    b.append([0, 1], [170, 75], k=b.rand(245, 8, 64, gain=keys) if keys else torch.zeros(245, 8, 64, dtype=dtype))
    q = b.rand(260, 32, 64)
    q[20:40] = 0
    q[60:260:3] = 0
    b.attend([0, 1], [170, 90], group=4, q=q)                     # the second's first 15 stand before its position 0
    b.attend([0, 1], [170, 90], group=4, q=q, left=33, chunk=4, sinks=20)
    b.attend([0, 1], [170, 90], group=4, q=torch.zeros_like(q))


@pytest.mark.parametrize("dtype,tokens,m,heads,group,dim", [(F32, 70000, 400, 2, 8, 64), (BF16, 2 ** 21 + 2 ** 20, 350, 1, 16, 16)])
def test_lse_over_values_of_zero(tmp_path, dtype, tokens, m, heads, group, dim):
    """V of zeros throughout, scores all alike: lse = log of the count.  Sums over the keys in fp32 as in bounds()."""
    b = Prompts(tmp_path, heads=heads, dim=dim, page=64, dtype=dtype, n_pages=tokens // 64 + 1, seqs=1, max_pages=tokens // 64 + 1)
    zero = torch.zeros(tokens, heads, dim, dtype=dtype, device="cuda")
    b.cache.extend(b.ids([0]), each=tokens)
    b.cache.write(0, b.ids([0]), zero, zero)
    out, lse = b.cache.attend(0, b.ids([0]), b.rand(m, heads * group, dim).cuda(), lse=True)
    b.cache.check()
    want = torch.arange(tokens - m + 1, tokens + 1, dtype=torch.float64).log()
    assert (lse.double().cpu() - want[:, None]).abs().max() <= tokens * 2.0 ** -24 + 2.0 ** -22 * 143
    assert (out == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values_near_the_largest_float(tmp_path, dtype):
    b = Prompts(tmp_path, heads=8, dim=64, page=16, dtype=dtype, n_pages=100)
    b.append([0, 1], [150, 60], v=torch.full((210, 8, 64), 3e38).to(dtype))
    b.attend([0, 1], [150, 60], group=4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("big", [1.0, 1e3, 1e6, 1e10, 1e15, 1e20])
def test_blocks_of_zero_values_beside_large_ones(tmp_path, dtype, big):
    """V blocks of zeros and of tiny values, before and after large ones: their tokens count in the norm with their full weight."""
    b = Prompts(tmp_path, heads=8, dim=64, page=16, dtype=dtype, n_pages=100)
    v = b.rand(400, 8, 64, gain=big)
    v[:16] *= 1e-25
    v[16:48] = 0
    v[96:320] = 0
    v[320:336] *= 1e-18
    b.append([0], [400], v=v)
    codes, scales = b.seqs[0].values(0, "k")
    K = codes.astype(np.float64) * scales[..., None]
    vs = b.seqs[0].values(0, "v")[1].astype(np.float64)
    for m, qgain, left in ((400, 1.0, -1), (160, 4.0, -1), (160, 1.0, 250)):
        q = b.rand(m, 32, 64, gain=qgain)
        out, lse = b.cache.attend(0, b.ids([0]), q.cuda(), att_left=left, lse=True)
        b.cache.check()
        qd = q.double().numpy()
        ref = attend64(b.seqs[0], 0, qd, 4, 0.125, left, 1, 0, 16)
        tol, tol_lse = bounds(*ref, 64, 400, dtype)
        # Weights times V scale are held in fp16 relative to the largest of the row, times 2^7 at least: what lies under fp16's
        # smallest number is off by half of it, 2^-25, which is 2^-32 of the largest for each key and code.  Where the tokens of
        # the largest have a code of 0, that is all of the error that there may be, and bounds() has no term for it.
        p, t = np.arange(400 - m, 400)[:, None], np.arange(400)
        unseen = (t > p) | ((t < p - left) if left >= 0 else False)
        for h in range(32):
            s = np.where(unseen, -np.inf, 0.125 * qd[:, h] @ K[:, h // 4].T)
            w = np.exp(s - ref[1][:, h, None]) * vs[:, h // 4]
            tol[:, h] += 400 * 2.0 ** -32 * 127 * w.max(1)[:, None]
        assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= tol_lse).all()
