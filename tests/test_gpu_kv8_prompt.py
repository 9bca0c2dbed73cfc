"""Attention over the 8-bit K/V cache by the kernel for many query rows, against the plain model in 64 bits.  Which kernel
answers a call depends on how it fills the card (more than 304 tiles of 16 rows on 152 SMs), so every call here is asserted to
be this one's."""
import warnings

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _kv8 import TOP, attend64, bounds  # noqa: E402
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

    def floor(self, i, q, lse, group, scale, left, chunk, sinks):
        """What bounds() has no term for: weights times V scale are held in fp16 under a factor of at least 2^7 (fp32 activations: hi
        and lo, 2^13) that the row's largest has.  One that lies under fp16's smallest number is off by half of that, 2^-25, which
        is 2^-32 (2^-38) of the largest, for each key and unit of its code.  Where the tokens of the largest have a code of 0, that
        is more than bounds() allows."""
        m, n, s = q.shape[0], self.seqs[i].len, self.seqs[i]
        codes, scales = s.values(0, "k")
        K, vs = codes.astype(np.float64) * scales[..., None], s.values(0, "v")[1].astype(np.float64)
        p, t = np.arange(n - m, n)[:, None], np.arange(n)
        begin = p // chunk * chunk
        seen = (t < begin + chunk) & ~np.isin(t // self.cfg.page_tokens, list(s.gone)) & (p >= 0)
        if left >= 0:
            seen &= (t >= begin - left) | (t < sinks)
        out = np.zeros((m, q.shape[1], 1))
        for h in range(q.shape[1] if n else 0):
            x = np.where(seen, scale * q[:, h] @ K[:, h // group].T, -np.inf)
            w = np.exp(x - np.where(np.isfinite(lse[:, h]), lse[:, h], 0)[:, None]) * vs[:, h // group]
            out[:, h, 0] = w.max(1)
        return n * 2.0 ** (-32 if self.dtype == BF16 else -38) * TOP[self.cfg.code] * out

    def attend(self, ids, counts, group=2, left=-1, chunk=1, sinks=0, scale=None, layer=0, q=None, qgain=1.0, uniform=False):
        """As Both.attend(), with floor() in the tolerance."""
        if layer:
            return super().attend(ids, counts, group, left, chunk, sinks, scale, layer, q, qgain, uniform)
        cfg = self.cfg
        q = self.rand(int(np.sum(counts)), group * cfg.kv_heads, cfg.head_dim, gain=qgain) if q is None else q
        rag = {} if uniform else {"starts": self.starts(counts), "max_new": max(counts)}
        out, lse = self.cache.attend(0, self.ids(ids), q.cuda(), att_left=left, att_chunk=chunk, sinks=sinks, scale=scale, lse=True, **rag)
        self.cache.check()
        scale = cfg.head_dim ** -0.5 if scale is None else scale
        at = 0
        for i, m in zip(ids, counts):
            x = q[at:at + m].double().numpy()
            ref = attend64(self.seqs[i], 0, x, group, scale, left, chunk, sinks, cfg.page_tokens)
            tol, tol_lse = bounds(*ref, cfg.head_dim, max(self.seqs[i].len, 1), self.dtype)
            tol = tol + self.floor(i, x, ref[1], group, scale, left, chunk, sinks)
            err = np.abs(out[at:at + m].double().cpu().numpy() - ref[0])
            assert (err <= tol).all(), (i, m, float((err / tol).max()), float(err.max()))
            dead, got = ~np.isfinite(ref[1]), lse[at:at + m].double().cpu().numpy()
            assert (got[dead] == -np.inf).all() and (err[dead] == 0).all()
            assert (np.abs(got[~dead] - ref[1][~dead]) <= tol_lse[~dead]).all(), i
            at += m
        return out, lse


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
    b.attend([0], [400], group=4)
    b.attend([0], [160], group=4, qgain=4.0)
    b.attend([0], [160], group=4, left=250)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("left,chunk,sinks", [(-1, 1, 0), (70, 2, 0), (10, 1, 4), (0, 1, 0), (0, 4, 1), (33, 8, 40), (5, 1000, 2),
                                              (200, 3, 17), (130, 1, 129)])
def test_windows_and_sinks(tmp_path, dtype, left, chunk, sinks):
    b = Prompts(tmp_path, heads=8, dim=64, page=32, dtype=dtype, n_pages=100)
    b.append(range(5), [1, 30, 64, 129, 357])
    b.attend(range(5), [1, 30, 9, 65, 200], group=4, left=left, chunk=chunk, sinks=sinks)
    b.attend(range(5), [0, 3, 0, 129, 1], group=8, left=left, chunk=chunk, sinks=sinks)


def test_extremes_of_the_window(tmp_path):
    big = 2 ** 31 - 1
    b = Prompts(tmp_path, heads=8, dim=64, page=16, n_pages=100)
    b.append([0, 1], [170, 137])
    for left, chunk, sinks in ((big, 1, 0), (0, 1, big), (3, big, 0), (big, big, big), (0, 1, 0)):
        b.attend([0, 1], [140, 137], group=4, left=left, chunk=chunk, sinks=sinks)


@pytest.mark.parametrize("code,dtype", [("int8", BF16), ("e4m3", F32), ("e4m3", BF16)])
def test_released_pages_are_not_seen(tmp_path, code, dtype):
    b = Prompts(tmp_path, code, heads=8, dim=64, page=16, n_pages=100, dtype=dtype)
    b.append([0, 1], [300, 190])
    b.trim([0], 30, 1, 20)
    for t in (b.cache.k_scale, b.cache.v_scale):                  # what lies in pages that nobody names
        t[:, (b.cache.refs == 0).nonzero()[:, 0]] = float("nan")
    b.attend([0, 1], [250, 103], group=2)                         # positions whose own pages are gone
    b.attend([0, 1], [140, 120], group=4, left=50, sinks=3)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_codes_that_no_write_filled_are_never_seen(tmp_path, code, dim):
    """Pages may hold anything before: 0xff is NaN as e4m3, and the scales are NaN too."""
    b = Prompts(tmp_path, code, heads=8, dim=dim, page=48, dtype=BF16, n_pages=60)
    for t in (b.cache.k, b.cache.v):
        t.fill_(-1)
    for t in (b.cache.k_scale, b.cache.v_scale):
        t.fill_(float("nan"))
    b.append([0, 1, 2, 3], [1, 17, 150, 300])
    for kw in ({}, {"left": 20, "sinks": 3}):
        b.attend([0, 1, 2, 3], [1, 17, 150, 300], **kw)
        b.attend([0, 3, 1, 2], [1, 77, 5, 121], group=4, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_queries_than_tokens(tmp_path, dtype):
    """Positions before 0 see nothing; a sequence of no tokens neither."""
    b = Prompts(tmp_path, heads=8, dim=64, page=16, dtype=dtype)
    b.append([0, 1], [3, 120])
    b.attend([0, 1, 2], [160, 140, 2], group=4)
    b.attend([1, 2, 0], [300, 130, 5], group=3, left=40, sinks=2)


@pytest.mark.parametrize("left", [-1, 8])
def test_bad_ids_and_counts_give_zero_rows(tmp_path, left):
    b = Prompts(tmp_path, heads=8, dim=64, page=16)
    b.append([0, 1], [160, 9])
    q = b.rand(360, 32, 64).cuda()
    want, wl = b.attend([0], [160], group=4, q=q[:160].cpu(), left=left)
    for ids, starts, max_new, bad in (([0, 6], [0, 160, 360], 200, slice(160, 360)), ([0, -1], [0, 160, 360], 200, slice(160, 360)),
                                      ([0, 1], [0, 160, 360], 199, slice(160, 360)), ([1, 0], [0, 200, 360], 160, slice(0, 200))):
        out = torch.full_like(q, 5.0)
        x = q if ids[0] == 0 else torch.cat([q[160:], q[:160]])
        _, lse = b.cache.attend(0, b.ids(ids), x, starts=b.ids(starts), max_new=max_new, att_left=left, out=out, lse=True)
        with pytest.raises(b.native.CacError) as e:
            b.cache.check()
        assert e.value.code == -11
        good = slice(0, 160) if ids[0] == 0 else slice(200, 360)
        assert (out[bad] == 0).all() and (lse[bad] == -np.inf).all()
        assert torch.equal(out[good], want) and torch.equal(lse[good], wl)


@pytest.mark.parametrize("left", [-1, 8, 5000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_starts_that_fall_or_pass_the_rows(tmp_path, dtype, left):
    b = Prompts(tmp_path, heads=8, dim=64, page=16, dtype=dtype, n_pages=60)
    good = [0, 160, 192, 232, 252]
    ids = [3, 0, 1, 2]
    b.append(ids, list(np.diff(good)))
    q = b.rand(252, 32, 64)
    want, _ = b.attend(ids, list(np.diff(good)), group=4, q=q, left=left)
    for bad, rows, same in (([0, 160, 192, 20, 40], 252, slice(0, 160)), ([0, 160, 192, 400, 500], 252, slice(0, 192)),
                            ([0, 160, 192, 232, 252], 240, slice(0, 232)), ([-5, 160, 192, 232, 252], 252, slice(160, 252))):
        fence = torch.full((rows + 200, 32, 64), 7.0, device="cuda", dtype=dtype)
        b.cache.attend(0, b.ids(ids), q[:rows].contiguous().cuda(), att_left=left, starts=b.ids(bad), max_new=160, out=fence[100:rows + 100])
        with pytest.raises(b.native.CacError) as e:
            b.cache.check()
        assert e.value.code == -11
        assert (fence[:100] == 7).all() and (fence[rows + 100:] == 7).all()
        if bad[2] < bad[3]:
            assert torch.equal(fence[100:rows + 100][same], want[same])
            if bad[3] != 400 and rows == 252:
                assert (fence[100:260] == 7).all()                # the sequence that begins before row 0
            else:
                assert (fence[100 + same.stop:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_no_sequence_and_row_strides(tmp_path, dtype):
    """Rows in front of the first sequence and behind the last are left alone; q and out are slices of wider rows."""
    b = Prompts(tmp_path, heads=8, dim=64, page=16, dtype=dtype)
    b.append([0, 1], [130, 140])
    wide = b.rand(300, 40, 64).cuda()
    q = wide[:, 3:35]
    out = torch.full((300, 36, 64), 7.0, dtype=dtype, device="cuda")
    b.cache.attend(0, b.ids([0, 1]), q, starts=b.ids([3, 128, 268]), max_new=140, out=out[:, 2:34])
    b.cache.check()
    assert (out[:3] == 7).all() and (out[268:] == 7).all() and (out[:, :2] == 7).all() and (out[:, 34:] == 7).all()
    want, _ = b.attend([0, 1], [125, 140], group=4, q=q[3:268].contiguous().cpu())
    assert torch.equal(out[3:268, 2:34], want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [64, 128])
def test_non_finite_queries_stay_in_their_rows(tmp_path, dtype, dim):
    b = Prompts(tmp_path, heads=8, dim=dim, page=16, dtype=dtype)
    b.append([0], [200])
    q = b.rand(180, 32, dim).cuda()
    want = b.cache.attend(0, b.ids([0]), q)
    q2 = q.clone()
    q2[5, 1, 3], q2[9, 2, 0], q2[9, 3], q2[179, 31, 1] = float("nan"), float("inf"), 0.0, -float("inf")
    got = b.cache.attend(0, b.ids([0]), q2)
    assert got[5, 1].isnan().all() and not torch.isfinite(got[9, 2]).any() and not torch.isfinite(got[179, 31]).any()
    ok = torch.ones(180, 32, dtype=torch.bool, device="cuda")
    ok[5, 1] = ok[9, 2] = ok[9, 3] = ok[179, 31] = False
    assert torch.equal(got[ok], want[ok]) and torch.isfinite(got[9, 3]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_unlike_scales_of_blocks(tmp_path, dtype):
    """Blocks whose V values differ by many powers of two, and logits far apart."""
    b = Prompts(tmp_path, heads=8, dim=64, page=16, dtype=dtype)
    for gain in (1e-4, 1.0, 300.0, 1e-2, 30.0, 1e-6, 5.0, 1e-3, 1.0, 2.0):
        b.append([0], [16], v=b.rand(16, 8, 64, gain=gain))
    b.attend([0], [160], group=4, qgain=1e-3)
    b.attend([0], [160], group=4, qgain=20.0)
    b.attend([0], [100], group=8, scale=-0.3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [64, 128])
def test_maxima_that_rise_and_fall(tmp_path, dtype, dim):
    """Logits that climb by less or more than a few powers of two a block, fall, or stand still, in rows side by side."""
    b = Prompts(tmp_path, heads=8, dim=dim, page=32, dtype=dtype, n_pages=64)
    line = torch.randn(dim, generator=torch.Generator().manual_seed(3))
    line /= line.norm()
    tokens = 430
    k = b.rand(tokens, 8, dim, gain=0.05) + (torch.arange(tokens) / 16.0)[:, None, None].to(dtype) * line.to(dtype)
    b.append([0], [tokens], k=k.to(dtype))
    step = torch.tensor([0.0, 0.3, 0.7, 1.0, 1.5, 4.0, -0.7, -4.0, 12.0, -12.0, 2.0, 1.9])   # powers of two a block
    q = step[torch.arange(200 * 32) % 12, None] * 0.6931 * dim ** 0.5 * line
    b.attend([0], [200], group=4, q=q.view(200, 32, dim).to(dtype))
    b.attend([0], [200], group=4, q=q.view(200, 32, dim).to(dtype), left=100, sinks=20)


@pytest.mark.parametrize("heads,group", [(1, 128), (3, 40), (5, 7)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_query_heads_to_a_kv_head(tmp_path, heads, group, dtype):
    b = Prompts(tmp_path, heads=heads, dim=64, page=32, dtype=dtype)
    b.append([0, 1, 2], [5, 64, 150])
    b.attend([0, 1, 2], [5, 64, 150], group=group)
    b.attend([2, 1], [140, 30], group=group, left=40)


def test_the_same_sequence_twice_two_graphs_and_a_side_stream(tmp_path):
    """Captured and replayed on two streams at once, and called on a third: the same bits each time."""
    b = Prompts(tmp_path, heads=8, dim=128, page=32, dtype=BF16, n_pages=100)
    b.append([0, 1], [400, 150])
    ids, starts = b.ids([0, 1, 0]), b.ids([0, 100, 250, 350])
    q = b.rand(350, 32, 128).cuda()
    q[250:] = q[:100]
    call = lambda **kw: b.cache.attend(0, ids, q, starts=starts, max_new=150, lse=True, **kw)  # noqa: E731
    want = call()
    assert torch.equal(want[0][:100], want[0][250:]) and torch.equal(want[1][:100], want[1][250:])
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    attend = b.cache.attend
    b.cache.attend = type(b.cache).attend.__get__(b.cache)         # plain calls inside a capture
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(call())
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        outs.append(call(stream=streams[2]))
    torch.cuda.synchronize()
    b.cache.check()
    b.cache.attend = attend
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_pools_past_two_gigabytes(tmp_path):
    """Page numbers whose byte offsets pass 2^31 and 2^32."""
    b = Prompts(tmp_path, heads=16, dim=128, page=64, n_pages=18000, seqs=3, max_pages=6, dtype=BF16, layers=2)   # 2.4 GB a layer for K
    b.cache.free.copy_(torch.arange(18000, dtype=torch.int32))
    b.append([0, 1], [70, 230])                              # the pool's last pages
    assert int(b.cache.table[0, 0]) > 17900
    b.attend([0, 1], [40, 130], layer=1)
    b.verify()


def test_more_sequences_than_one_launch_takes(tmp_path):
    """700 sequences, 512 to a launch: ragged and even."""
    b = Prompts(tmp_path, heads=2, dim=80, page=16, n_pages=3500, seqs=700, max_pages=6, dtype=BF16)
    rng = np.random.RandomState(5)
    ids = list(rng.permutation(700))
    b.append(ids, list(rng.randint(1, 60, 700)))
    b.attend(ids, list(rng.randint(0, 20, 700)), group=4)
    b.attend(ids, [9] * 700, group=4, left=12, sinks=3, uniform=True)
