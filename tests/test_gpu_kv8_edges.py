"""Edges of the 8-bit K/V cache: what lies beside a sequence, blocks that no write has filled, extreme scales and sizes."""
import contextlib

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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 12), (256, 2)])
def test_lse_over_values_of_zero(dtype, dim, group):
    """A head whose V is zero throughout, scores all alike: lse = log of the count, whichever warps share the tokens."""
    tokens = 70000
    b = Both(heads=2, dim=dim, page=64, dtype=dtype, n_pages=1200, seqs=2, max_pages=1100)
    zero = torch.zeros(tokens, 2, dim, dtype=dtype, device="cuda")
    for i, m in ((0, tokens), (1, 300)):
        b.cache.extend(b.ids([i]), each=m)
        b.cache.write(0, b.ids([i]), zero[:m], zero[:m])
    for left in (-1, 200):
        out, lse = b.cache.attend(0, b.ids([0, 1]), b.rand(2, 2 * group, dim).cuda(), att_left=left, lse=True)
        b.cache.check()
        want = torch.tensor([tokens, 300] if left < 0 else [left + 1, left + 1], dtype=torch.float64).log()
        # sums over the keys in fp32, and the logarithm's own rounding (see bounds())
        assert (lse.double().cpu() - want[:, None]).abs().max() <= tokens * 2.0 ** -24 + 2.0 ** -22 * 140
        assert (out == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,group", [(1, 1), (5, 4)])
def test_values_near_the_largest_float(dtype, m, group):
    b = Both(heads=2, dim=64, page=16, dtype=dtype)
    b.append([0, 1], [90, 1], v=torch.full((91, 2, 64), 3e38).to(dtype))
    b.attend([0, 1], [m, 1], group=group)
    b.attend([0, 1], [m, 1], group=group, left=20)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("big", [1.0, 1e3, 1e6, 1e10, 1e15, 1e20])
@pytest.mark.parametrize("m,group,dim", [(1, 1, 64), (5, 4, 64), (1, 6, 128), (2, 9, 256)])
def test_blocks_of_zero_values_beside_large_ones(dtype, big, m, group, dim):
    """V blocks of zeros and of tiny values, before and after large ones: their tokens count in the norm with their full weight."""
    b = Both(heads=2, dim=dim, page=16, dtype=dtype, n_pages=100, max_pages=100)
    v = b.rand(400, 2, dim, gain=big)
    v[:16] *= 1e-25
    v[16:48] = 0
    v[96:320] = 0
    v[320:336] *= 1e-18
    b.append([0], [400], v=v)
    for kw in ({}, {"qgain": 4.0}, {"left": 250}, {"left": 350, "sinks": 30}):
        b.attend([0], [m], group=group, **kw)


def test_blocks_of_zero_values_in_parts_that_are_joined():
    """... where warps and blocks each hold a part of the sequence, some of nothing but zeros."""
    b = Both(heads=1, dim=64, page=64, dtype=F32, n_pages=600, seqs=2, max_pages=500)
    v = b.rand(30000, 1, 64, gain=1e12)
    v[1000:29000] = 0
    b.append([0], [30000], v=v)
    b.attend([0], [1], group=2)
    b.attend([0], [3], group=4, qgain=4.0)


class Holes(Both):
    """A cache in which some tokens are never written; what the others hold is compared token by token."""

    def __init__(self, *args, left_over=1e30, **kw):
        super().__init__(*args, **kw)
        for t in (self.cache.k_scale, self.cache.v_scale):
            t.fill_(left_over)
        for t in (self.cache.k, self.cache.v):
            t.fill_(-1)
        self.filled = [np.zeros(0, bool) for _ in self.seqs]

    def hole(self, ids, counts):
        """Room for tokens that no write fills: in the model, codes of 0, and scales of 0 for the blocks that they begin."""
        self.cache.extend(self.ids(ids), starts=self.starts(counts))
        for i, m in zip(ids, counts):
            s = self.seqs[i]
            for key in s.code:
                s.code[key] = np.concatenate([s.code[key][:s.len], np.zeros((m,) + s.code[key].shape[1:], np.float32)])
                old = s.scale[key][:-(-s.len // 16)]
                s.scale[key] = np.concatenate([old, np.zeros((-(-(s.len + m) // 16) - len(old),) + old.shape[1:], np.float32)])
            s.len += m
            self.filled[i] = np.concatenate([self.filled[i], np.zeros(m, bool)])

    def append(self, ids, counts, **kw):
        super().append(ids, counts, **kw)
        for i, m in zip(ids, counts):
            self.filled[i] = np.concatenate([self.filled[i], np.ones(m, bool)])

    def truncate(self, ids, lens):
        super().truncate(ids, lens)
        for i in ids:
            self.filled[i] = self.filled[i][:self.seqs[i].len]

    def fork(self, src, dst):
        super().fork(src, dst)
        for s, d in zip(src, dst):
            self.filled[d] = self.filled[s].copy()

    def verify(self):
        self.cache.check()
        for layer in range(self.cfg.n_layers):
            for i, s in enumerate(self.seqs):
                if s.len == 0:
                    continue
                got = self.cache.read(layer, self.ids([i]), self.ids([0]), s.len)
                for which, x in zip("kv", got):
                    codes, scales = s.values(layer, which)
                    assert np.array_equal(x[0].cpu().numpy()[self.filled[i]], (codes * scales[..., None])[self.filled[i]]), (layer, i)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("left_over", [1e30, float("inf"), float("nan"), 0.0, 1e-30])
def test_tokens_after_unwritten_ones_have_their_own_scale(code, left_over):
    b = Holes(code, dim=32, page=32, layers=2, seqs=6, left_over=left_over)
    b.hole([0, 1, 2], [5, 16, 40])
    b.append([2, 0, 1], [3, 1, 7])
    b.verify()
    b.hole([0, 1], [20, 1])
    b.append([0, 1], [2, 40], gain=0.1)
    b.verify()
    b.append([3], [50], gain=1e4)               # a left-over of the cache's own
    b.truncate([3], [16])
    b.hole([3], [3])
    b.append([3], [2])
    b.verify()


def test_unwritten_blocks_of_shared_pages():
    """Sequences of unlike lengths share a page, are extended at once, and not all of them are written."""
    for parent in (True, False):
        b = Holes("int8", dim=32, page=64, layers=2, seqs=8, n_pages=60)
        b.append([0], [64 + 50], gain=100.0)
        b.fork([0, 0, 0, 0], [1, 2, 3, 4])
        b.truncate([1, 2, 4], [64 + 10, 64 + 33, 64 + 49])
        if not parent:
            b.truncate([0], [0])
        b.hole([1, 3, 2, 4], [30, 5, 2, 10])
        b.append([4, 2, 1, 3], [3, 20, 2, 9])
        b.verify()
        b.cache.compact()
        b.append([4, 2, 1, 3], [1, 1, 1, 1])
        b.verify()


@pytest.mark.parametrize("n,each", [(1, 3000), (300, 2), (40, 70)])
def test_unwritten_blocks_of_even_calls(n, each):
    b = Holes("int8", heads=1, dim=16, page=16, layers=3, seqs=n, n_pages=n * (each // 16 + 4), max_pages=each // 16 + 4)
    b.hole(range(n), [each - 1] * n)
    b.append(range(n), [3] * n)
    b.cache.extend(b.ids(range(n)), each=each % 29 + 1)
    b.cache.check()
    assert b.cache.lens.tolist() == [each + 2 + each % 29 + 1] * n
    t = each + 2                                 # the first of the new blocks of every sequence has scale 0 in every layer
    t += -t % 16
    if t < each + 2 + each % 29 + 1:
        page = b.cache.table[:, t // 16].long()
        assert (b.cache.k_scale[:, page] == 0).all() and (b.cache.v_scale[:, page] == 0).all()
    b.truncate(range(n), [each + 2] * n)
    b.verify()


def test_unwritten_tokens_are_not_seen_from_other_sequences_of_a_prompt_call():
    b = Holes("e4m3", heads=8, dim=64, page=16, n_pages=200, seqs=3, dtype=BF16, left_over=float("nan"))
    b.append([0, 1], [200, 90])
    b.hole([2], [150])
    q = b.rand(440, 32, 64)
    out = b.cache.attend(0, b.ids([0, 2, 1]), q.cuda(), starts=b.ids([0, 200, 350, 440]), max_new=200)
    b.cache.check()
    for i, rows in ((0, slice(0, 200)), (1, slice(350, 440))):
        ref = attend64(b.seqs[i], 0, q[rows].double().numpy(), 4, 0.125, -1, 1, 0, 16)
        tol, _ = bounds(*ref, 64, 200, BF16)
        assert (np.abs(out[rows].double().cpu().numpy() - ref[0]) <= tol).all()


def test_workspace_is_asked_for_with_any_max_new():
    """The C call without starts ignores max_new, and so does the size that it is told."""
    import ctypes
    b = Both(heads=1, dim=64, page=16, max_pages=100, n_pages=100)
    b.append([0], [700])
    lib, ref = b.native.lib(), ctypes.addressof(b.cache._c)
    q = b.rand(8, 1, 64).cuda()
    want = b.cache.attend(0, b.ids([0]), q, att_left=280)
    for max_new in (0, 1, 8, 100):
        need = lib.cac_kv8_attend_workspace(ref, 1, 8, max_new, 1, 280, 1, 0)
        space = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        ids = b.ids([0])
        r = lib.cac_kv8_attend(ref, 0, 1, ids.data_ptr(), None, 8, max_new, 1, 0.125, 280, 1, 0, q.data_ptr(), 64, out.data_ptr(), 64,
                               None, 0, space.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert r == 0, max_new
        b.cache.check()
        assert torch.equal(out, want)


def test_a_read_of_as_many_tokens_as_an_int_counts():
    """2^31 - 1 tokens, all but the last few before the sequence's first: 69 GB of zeros."""
    import ctypes
    count, tokens = 2 ** 31 - 1, 20
    b = Both(heads=1, dim=16, page=16, dtype=BF16)
    b.append([0], [tokens])
    k = torch.full((count, 16), 3.0, dtype=BF16, device="cuda")
    ids, first = b.ids([0]), b.ids([tokens - count])
    r = b.native.lib().cac_kv8_read(ctypes.addressof(b.cache._c), 0, 1, ids.data_ptr(), first.data_ptr(), count, k.data_ptr(), None, 1,
                                    torch.cuda.current_stream().cuda_stream)
    assert r == 0
    want, _ = b.cache.read(0, ids, torch.zeros_like(ids), tokens, dtype=BF16)
    b.cache.check()
    assert torch.equal(k[-tokens:], want[0, :, 0])
    assert not any(bool(x.any()) for x in k[:-tokens].split(2 ** 27))
    del k
    torch.cuda.empty_cache()


@pytest.mark.parametrize("how", ["argument", "current"])
def test_a_cache_dropped_behind_its_calls_on_a_side_stream(how):
    """Its memory is not given out again before they have run."""
    b = Both(heads=2, dim=64, page=16, n_pages=700, max_pages=64)
    side = torch.cuda.Stream()
    ids, x = b.ids([0, 1]), torch.randn(2000, 2, 64, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10 ** 9)                                   # about half a second in front of the calls
    kw = {"stream": side} if how == "argument" else {}
    with contextlib.nullcontext() if kw else torch.cuda.stream(side):
        b.cache.extend(ids, each=1000, **kw)
        b.cache.write(0, ids, x, x, **kw)
        b.cache.compact(**kw)
    own = {t.data_ptr() for t in b.cache._own}
    sizes = [(t.shape, t.dtype) for t in b.cache._own]
    b.cache = None
    assert not side.query()                                          # the calls are still to come
    taken = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes]
    assert not own & {t.data_ptr() for t in taken}
    torch.cuda.synchronize()
