"""Attention of sequences that share a prefix on the GPU: against the plain model in 64
bits, sequence by sequence, and against what may and may not be shared.  A call that has
less than 70 MB to read even if it shares nothing is cac_kv8_attend's, so the caches here have
tables for far longer sequences than they hold, and calls are asserted to be the shared
kernels' by the kernels of a captured graph."""
import warnings

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _kv8 import attend64, bounds  # noqa: E402
from test_gpu_kv8 import Both  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BOUNDS = -11


class Shared(Both):
    def __init__(self, code="int8", layers=1, heads=2, dim=64, page=32, n_pages=64, seqs=6, dtype=F32, seed=0, least=2):
        """least: the tables have room for 100 MB of so many sequences."""
        room = 100_000_000 // (least * heads * 2 * dim * page) + 1
        super().__init__(code, layers, heads, dim, page, n_pages, seqs, room, dtype, seed)

    def kernels(self, call):
        """Names in the graph of a captured call."""
        import tempfile
        graph = torch.cuda.CUDAGraph(keep_graph=True)
        graph.enable_debug_mode()
        with torch.cuda.graph(graph):
            call()
        with tempfile.NamedTemporaryFile(suffix=".dot") as f:
            with warnings.catch_warnings():
                warnings.simplefilter("ignore")      # it warns that it writes a file
                graph.debug_dump(f.name)
            return open(f.name).read()

    def family(self, groups, first=0, gain=1.0):
        """groups: (prefix, [own tokens of each member]).  A member is a fork of its group's prefix, extended.  Returns the
        groups' starts; members are sequences first, first + 1, ..."""
        at, starts = first, [0]
        for prefix, own in groups:
            members = list(range(at, at + len(own)))
            if prefix:
                self.append(members[:1], [prefix], gain=gain)
                if members[1:]:
                    self.fork(members[:1] * (len(members) - 1), members[1:])
            for m, t in zip(members, own):
                if t:
                    self.append([m], [t], gain=gain)
            at += len(own)
            starts.append(at - first)
        return starts

    def check_shared(self, ids, counts, groups, group=2, left=-1, chunk=1, sinks=0, scale=None, layer=0, q=None, qgain=1.0,
                     uniform=False, shares=True, prefix=None, **kw):
        """shares: whether the call is the shared kernels' (None: either).  prefix: whether the shared tokens are read by the kernel for
        many rows (None: either)."""
        cfg = self.cfg
        T, heads = int(np.sum(counts)), group * cfg.kv_heads
        q = self.rand(T, heads, cfg.head_dim, gain=qgain) if q is None else q
        rag = {} if uniform else {"starts": self.starts(counts), "max_new": max(counts, default=0)}
        dev, dq, dg = self.ids(ids), q.cuda(), None if groups is None else self.ids(groups)
        call = lambda: self.cache.attend_shared(layer, dev, dq, groups=dg, att_left=left, att_chunk=chunk, sinks=sinks, scale=scale,  # noqa: E731
                                                lse=True, **rag, **kw)
        if shares is not None or prefix is not None:
            names = self.kernels(call)
            assert shares is None or ("kv_plan_shared_kernel" in names) == shares
            assert prefix is None or ("kv_prefix_kernel" in names) == prefix
        out, lse = call()
        self.cache.check()
        assert out.dtype == q.dtype and out.shape == q.shape and lse.shape == (T, heads)
        sc = scale if scale is not None else cfg.head_dim ** -0.5
        at = 0
        for i, m in zip(ids, counts):
            if m == 0:
                continue
            ref = attend64(self.seqs[i], layer, q[at:at + m].double().numpy(), group, sc, left, chunk, sinks, cfg.page_tokens)
            tol, tol_lse = bounds(*ref, cfg.head_dim, max(self.seqs[i].len, 1), self.dtype)
            # the join of the parts: an exponential (2^-21) and four roundings for each, in the sum and in its norm
            tol, tol_lse = tol + 2 * (2.0 ** -21 + 2.0 ** -22) * ref[2], tol_lse + 2.0 ** -20
            # A weight times its V scale enters the product as fp16 in steps of 2^-24 where the largest is held as 2^13 or more
            # (bf16: 2^7), so each token is off by half a step of that, 2^-38 (2^-32) of the largest, times its code.  That is nothing
            # beside the weights' own roundings unless the token that outweighs all others has a value near 0.
            top = max(float(self.seqs[i].values(layer, "v")[1].max(initial=0)) * (127 if cfg.code == "int8" else 448), 0)
            tol = tol + self.seqs[i].len * top * (2.0 ** -32 if self.dtype is BF16 else 2.0 ** -38)
            o, s = out[at:at + m].double().cpu().numpy(), lse[at:at + m].double().cpu().numpy()
            err = np.abs(o - ref[0])
            assert (err <= tol).all(), (i, m, float((err / tol).max()), float(err.max()))
            dead = ~np.isfinite(ref[1])
            assert (s[dead] == -np.inf).all() and (o[dead] == 0).all()
            err = np.abs(s[~dead] - ref[1][~dead])
            assert (err <= tol_lse[~dead]).all(), (i, float(err.max()))
            at += m
        return out, lse


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,page,group", [(64, 16, 1), (128, 32, 4), (80, 48, 3), (16, 16, 8), (256, 64, 2), (64, 64, 17), (144, 16, 5)])
def test_one_group(code, dtype, dim, page, group):
    b = Shared(code, heads=2, dim=dim, page=page, n_pages=200, seqs=8, dtype=dtype, seed=dim)
    b.family([(5 * page + 7, [1, 3, 17, 2 * page + 1, 5, 40, 1, 9])])
    b.check_shared(range(8), [1] * 8, None, group=group, uniform=True)
    b.check_shared(range(8), [1, 3, 2, 5, 1, 0, 1, 9], [0, 8], group=group)
    b.check_shared(range(2), [1, 1], [0, 2], group=group)


@pytest.mark.parametrize("code,dtype", [("int8", BF16), ("e4m3", F32), ("int8", F32), ("e4m3", BF16)])
@pytest.mark.parametrize("n,group,dim", [(24, 1, 64), (9, 8, 128), (40, 4, 64), (40, 8, 128), (70, 1, 128), (33, 5, 80), (20, 3, 256), (60, 1, 64),
                                         (12, 4, 128), (17, 8, 128), (33, 8, 64), (300, 1, 32)])
def test_many_rows(code, dtype, n, group, dim):
    """Groups of more rows than a tile has, of 8 to 350 rows."""
    rng = np.random.default_rng(n)
    own = rng.integers(1, 90, n).tolist()
    b = Shared(code, heads=2, dim=dim, page=32, n_pages=600 + 4 * n, seqs=n, dtype=dtype, seed=n)
    b.family([(1100, own)])
    rows = n * group
    b.check_shared(range(n), [1] * n, None, group=group, uniform=True, prefix=rows > 32 and dim <= 128)
    b.check_shared(range(n), rng.integers(0, 3, n).tolist(), [0, n], group=group, qgain=4.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [1, 4])
def test_several_groups_and_sequences_of_none(dtype, group):
    b = Shared("int8", heads=2, dim=64, page=16, n_pages=500, seqs=20, dtype=dtype, seed=3)
    st = b.family([(300, [5, 6, 7]), (20, [1]), (900, [30, 1, 1, 80, 2, 4]), (16, [2, 3]), (0, [4, 5, 6]), (333, [1, 2, 3, 4, 5])])
    assert st[-1] == 20
    b.check_shared(range(20), [1] * 20, st, group=group)
    b.check_shared(range(20), [2, 1, 3, 1, 1, 1, 0, 2, 5, 1, 2, 1, 4, 5, 6, 1, 0, 0, 0, 2], st, group=group)
    b.check_shared(range(20), [1] * 20, st[1:5], group=group)            # the first and last stand alone
    b.check_shared(range(20), [1] * 20, [0, 20], group=group)            # one group of unlike tables shares nothing
    b.check_shared(range(20), [1] * 20, list(range(21)), group=group)    # groups of one
    b.check_shared(range(20), [1] * 20, [0, 0, 3, 3, 10, 10], group=group)
    b.check_shared([4, 5, 6, 4, 9, 5], [1] * 6, None, group=group)       # a sequence more than once


@pytest.mark.parametrize("left,chunk,sinks", [(-1, 1, 0), (-1, 4, 0), (70, 2, 0), (10, 1, 4), (0, 1, 0), (5, 1000, 2), (100000, 1, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_windows_and_sinks(dtype, left, chunk, sinks):
    """Small windows are attend's, chunks and windows that the sequence never fills the shared kernels'."""
    b = Shared("int8", heads=1, dim=64, page=16, n_pages=300, seqs=6, dtype=dtype, seed=left + chunk)
    b.family([(389, [1, 20, 60, 130, 2, 7])])
    args = {"left": left, "chunk": chunk, "sinks": sinks, "shares": None if left >= 0 else True}
    b.check_shared(range(6), [1] * 6, None, uniform=True, **args)
    b.check_shared(range(6), [1, 4, 2, 1, 2, 3], [0, 6], **args)
    b.check_shared([4, 0], [2, 1], [0, 2], group=9, **args)


@pytest.mark.parametrize("dtype,code", [(F32, "e4m3"), (BF16, "int8")])
@pytest.mark.parametrize("left,chunk,sinks,counts", [(800, 1, 4, "one"), (800, 8, 40, "some"), (790, 1, 0, "some"), (1010, 2, 0, "one"), (870, 1, 900, "some")])
def test_windows_that_end_within_the_prefix(dtype, code, left, chunk, sinks, counts):
    """Enough sequences for the shared kernels: windows that begin before the prefix, within it, and for some of a group only."""
    n = 70
    rng = np.random.default_rng(left)
    own = rng.integers(1, 140, n)
    own[3], own[40] = 700, 1
    b = Shared(code, heads=8, dim=128, page=32, n_pages=1200, seqs=n, dtype=dtype, seed=left, least=20)
    st = b.family([(901, own[:30].tolist()), (640, own[30:].tolist())])
    many = [1] * n if counts == "one" else rng.integers(0, 4, n).tolist()
    b.check_shared(range(n), many, st, group=2, left=left, chunk=chunk, sinks=sinks, uniform=counts == "one")


def test_queries_inside_the_prefix_and_nothing_of_ones_own():
    """Sequences that are copies of one another: the last query sees to the end, the first ones do not."""
    b = Shared("int8", heads=2, dim=64, page=16, n_pages=100, seqs=5)
    b.family([(160, [0, 0, 0, 0, 0])])
    for counts in ([1] * 5, [1, 160, 3, 30, 2], [170, 1, 1, 1, 1]):
        b.check_shared(range(5), counts, None)
    b.check_shared(range(5), [1] * 5, None, chunk=16)
    b.check_shared(range(5), [1] * 5, None, chunk=7, left=20, shares=False)


def test_released_pages_and_truncated_members():
    b = Shared("e4m3", heads=2, dim=64, page=16, n_pages=200, seqs=6, dtype=BF16)
    b.family([(400, [3, 4, 5, 6, 7, 8])])
    b.trim(range(6), 100, 1, 20)                     # the same pages of all: still one group
    b.check_shared(range(6), [1] * 6, None, left=100, sinks=20, shares=False)
    b.check_shared(range(6), [1] * 6, None)          # released pages are not seen
    b.truncate([2, 4], [330, 0])                     # into a page that the window has not passed
    b.check_shared([0, 1, 2, 3, 5], [1] * 5, None, left=100, sinks=20, shares=False)
    b.append([2, 4], [90, 30])                       # other pages from there on
    b.check_shared(range(6), [1] * 6, None)
    b.check_shared(range(6), [1, 2, 1, 1, 30, 1], None)
    b.check_shared(range(6), [1] * 6, None, group=9)  # released pages in front of the kernel for many rows


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [1, 12])
def test_a_token_that_outweighs_the_rest_on_either_side(dtype, group):
    """Maxima far apart between the parts, and V blocks of unlike sizes."""
    b = Shared("int8", heads=1, dim=64, page=16, n_pages=200, seqs=4, dtype=dtype)
    b.family([(200, [20, 30, 40, 50])])
    q = b.rand(4, group, 64)
    big = q[1:2, :1].float() * 40
    b.append([1], [1], k=big.to(dtype), v=b.rand(1, 1, 64, gain=100.0))
    b.check_shared(range(4), [1] * 4, None, group=group, q=q, uniform=True)
    c = Shared("int8", heads=1, dim=64, page=16, n_pages=200, seqs=4, dtype=dtype)
    c.append([0], [100])
    c.append([0], [1], k=big.to(dtype), v=c.rand(1, 1, 64, gain=1e-4))
    c.append([0], [16], k=c.rand(16, 1, 64), v=torch.zeros(16, 1, 64, dtype=dtype))
    c.append([0], [30])
    c.fork([0, 0, 0], [1, 2, 3])
    for i in range(4):
        c.append([i], [5 + i], gain=1e3 if i == 2 else 1.0)
    c.check_shared(range(4), [1] * 4, None, group=group, q=q, uniform=True)


def test_non_finite_queries_stay_in_their_rows():
    b = Shared("int8", heads=1, dim=64, page=16, n_pages=200, seqs=30, dtype=BF16)
    b.family([(600, [2] * 30)])
    q = b.rand(30, 6, 64)
    want, _ = b.check_shared(range(30), [1] * 30, None, group=6, q=q, uniform=True)
    bad = q.clone()
    bad[3, 2, 5], bad[17, 0, 0] = float("nan"), float("inf")
    got = b.cache.attend_shared(0, b.ids(range(30)), bad.cuda())
    keep = torch.ones(30, 6, dtype=torch.bool)
    keep[3, 2] = keep[17, 0] = False
    assert torch.equal(got.cpu()[keep], want.cpu()[keep])
    assert torch.isnan(got[3, 2]).all() and torch.isnan(got[17, 0]).all()


def test_long_prefix_split_over_the_card():
    b = Shared("int8", heads=2, dim=64, page=64, n_pages=700, seqs=8, dtype=BF16)
    b.family([(30011, [5, 900, 33, 1, 2, 64, 8, 12])])
    b.check_shared(range(8), [1] * 8, None, group=4, uniform=True)


@pytest.mark.parametrize("bad", [[0, 3, 2, 6], [-1, 6], [0, 7], [5, 3]])
def test_bad_groups_are_refused_and_share_nothing(bad):
    b = Shared("int8", heads=1, dim=64, page=16, n_pages=200, seqs=6)
    b.family([(200, [1, 2, 3, 4, 5, 6])])
    q = b.rand(6, 2, 64).cuda()
    want = b.cache.attend(0, b.ids(range(6)), q)
    got = b.cache.attend_shared(0, b.ids(range(6)), q, groups=b.ids(bad))
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == BOUNDS
    assert (got - want).abs().max() <= 2e-6 * want.abs().max()


def test_bad_ids_and_counts_as_in_attend():
    """Rows of such sequences are zero, or left where their rows pass the end; the others of the group are right."""
    b = Shared("int8", heads=1, dim=64, page=16, n_pages=200, seqs=6)
    b.family([(200, [1, 2, 3, 4, 5, 6])])
    for ids, counts, max_new in (([0, 1, 9, 3], [1, 1, 2, 1], 2), ([0, -1, 2, 3], [1, 1, 1, 1], 1), ([0, 1, 2, 3], [1, 12, 1, 1], 3)):
        q = b.rand(int(np.sum(counts)), 2, 64).cuda()
        args = {"starts": b.starts(counts), "max_new": max_new, "lse": True}
        want, s = b.cache.attend(0, b.ids(ids), q, **args)
        with pytest.raises(b.native.CacError):
            b.cache.check()
        got, t = b.cache.attend_shared(0, b.ids(ids), q, **args)
        with pytest.raises(b.native.CacError) as e:
            b.cache.check()
        assert e.value.code == BOUNDS
        zero = (want == 0).all(-1)
        assert torch.equal((got == 0).all(-1), zero) and zero.any() and torch.equal(torch.isinf(t), torch.isinf(s))
        assert (got - want).abs().max() <= 2e-6 * want.abs().max()


def test_rows_of_no_sequence_are_left_alone():
    b = Shared("int8", heads=1, dim=64, page=16, n_pages=200, seqs=6)
    b.family([(200, [1, 2, 3, 4, 5, 6])])
    q = b.rand(12, 2, 64).cuda()
    out = torch.full_like(q, 7.0)
    b.cache.attend_shared(0, b.ids([0, 1, 2]), q, starts=b.ids([3, 4, 6, 7]), max_new=2, out=out)
    b.cache.check()
    assert (out[:3] == 7).all() and (out[7:] == 7).all() and (out[3:7] != 7).all()
    want = b.cache.attend(0, b.ids([0, 1, 2]), q, starts=b.ids([3, 4, 6, 7]), max_new=2)
    assert (out[3:7] - want[3:7]).abs().max() <= 2e-6 * want[3:7].abs().max()
    out.fill_(7.0)
    b.cache.attend_shared(0, b.ids([0, 1]), q, starts=b.ids([0, 2, 13]), max_new=20, out=out)   # rows past the end
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == BOUNDS and (out[2:] == 7).all() and (out[:2] != 7).all()


def test_strided_queries_and_outputs():
    b = Shared("int8", heads=2, dim=64, page=16, n_pages=200, seqs=5, dtype=BF16)
    b.family([(200, [1, 2, 3, 4, 5])])
    wide = b.rand(5, 9, 64).cuda()
    out = torch.full((5, 7, 64), 3.0, dtype=BF16, device="cuda")
    got = b.cache.attend_shared(0, b.ids(range(5)), wide[:, 2:6], out=out[:, 1:5])
    assert torch.equal(got, b.cache.attend_shared(0, b.ids(range(5)), wide[:, 2:6].contiguous()))
    assert (out[:, :1] == 3).all() and (out[:, 5:] == 3).all()


def test_the_same_result_each_time():
    b = Shared("int8", heads=2, dim=128, page=32, n_pages=400, seqs=40, dtype=F32)
    b.family([(3000, list(range(1, 41)))])
    q = b.rand(40, 8, 128).cuda()
    first = b.cache.attend_shared(0, b.ids(range(40)), q, lse=True)
    for _ in range(5):
        again = b.cache.attend_shared(0, b.ids(range(40)), q, lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_more_sequences_and_groups_than_one_launch_takes():
    n = 1100
    b = Shared("int8", heads=1, dim=64, page=16, n_pages=2400, seqs=n, dtype=BF16)
    st = b.family([(64, [1] * 4), (150, [2] * 700), (40, [1] * 396)])
    ids = list(range(n))
    q = b.rand(n, 2, 64)
    got = b.cache.attend_shared(0, b.ids(ids), q.cuda(), groups=b.ids(st))
    want = b.cache.attend(0, b.ids(ids), q.cuda())
    b.cache.check()
    # both are rounded to bf16 and hold weights to 11 bits
    assert (got.float() - want.float()).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -10) * want.float().abs().max()
    some = [0, 3, 4, 5, 600, 703, 704, 1099]
    b.check_shared(some, [1] * 8, [0, 2, 6, 8], q=q[some])
    pairs = list(range(0, n + 1, 2))                 # 550 groups
    got = b.cache.attend_shared(0, b.ids(ids), q.cuda(), groups=b.ids(pairs))
    assert (got.float() - want.float()).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -10) * want.float().abs().max()
    b.cache.check()


@pytest.mark.parametrize("group,counts", [(4, [1] * 10), (4, [1, 2, 0, 3, 1, 1, 1, 1, 1, 7])])
def test_two_captured_graphs_replayed_at_once(group, counts):
    """Each has its workspace; the tables and lengths may change in between."""
    b = Shared("int8", heads=2, dim=64, page=16, n_pages=400, seqs=10, dtype=BF16)
    b.family([(500, list(range(1, 11)))])
    T = int(np.sum(counts))
    qs = [b.rand(T, 2 * group, 64) for _ in range(2)]
    dev, outs, graphs, streams = [q.cuda() for q in qs], [], [], [torch.cuda.Stream() for _ in range(2)]
    ids, st = b.ids(range(10)), b.starts(counts)
    torch.cuda.synchronize()
    for q in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.cache.attend_shared(0, ids, q, starts=st, max_new=max(counts)))
        graphs.append(g)
    b.append([2, 5], [3, 20])
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    b.cache.check()
    for q, out in zip(qs, outs):
        want, _ = b.check_shared(range(10), counts, None, group=group, q=q)
        assert torch.equal(out, want)


def test_on_another_stream():
    b = Shared("int8", heads=2, dim=64, page=16, n_pages=400, seqs=10, dtype=BF16)
    b.family([(500, list(range(1, 11)))])
    q, ids, groups = b.rand(10, 8, 64).cuda(), b.ids(range(10)), b.ids([0, 10])
    want = b.cache.attend_shared(0, ids, q, groups=groups)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    one = b.cache.attend_shared(0, ids, q, groups=groups, stream=s)
    with torch.cuda.stream(s):
        two = b.cache.attend_shared(0, ids, q, groups=groups)
    torch.cuda.synchronize()
    assert torch.equal(one, want) and torch.equal(two, want)


def test_prompts_behind_a_prefix_go_to_the_prompts_kernel():
    """Sequences of many query rows: attend itself, bit for bit."""
    b = Shared("int8", heads=2, dim=64, page=32, n_pages=400, seqs=80, dtype=BF16)
    b.family([(300, [100] * 80)])
    q, st = b.rand(8000, 4, 64).cuda(), b.starts([100] * 80)
    got = b.cache.attend_shared(0, b.ids(range(80)), q, starts=st, max_new=100)
    assert torch.equal(got, b.cache.attend(0, b.ids(range(80)), q, starts=st, max_new=100))


def test_empty_calls():
    b = Shared("int8", heads=2, dim=64, page=16, n_pages=40, seqs=4)
    b.family([(20, [1, 2])])
    none = torch.empty(0, 2, 64, device="cuda")
    assert b.cache.attend_shared(0, b.ids([]), none).shape == (0, 2, 64)
    assert b.cache.attend_shared(0, b.ids([0, 1]), none, starts=b.ids([0, 0, 0]), max_new=1).shape == (0, 2, 64)
    b.check_shared([3, 2], [1, 1], None)             # sequences without tokens
    b.check_shared([0, 3, 1], [1, 1, 1], None)       # one of them without
    b.cache.check()


# ---------------------------------------------------------------------------
# a run of the operators, as a step uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("graph", [False, True])
def test_a_decoding_step(dtype, graph):
    """Two layers: product into q, k and v, rotation, write, attention behind a shared prefix, product out.  Every
    operator's output is compared with the 64-bit form of its inputs, step by step."""
    from cache_aware_conformer_gb300 import native, w4
    from cache_aware_conformer_gb300.config import RotaryConfig
    from test_gpu_rotate import close, exact
    from test_gpu_w4 import exact as exact_w4
    H, G, D, n, L = 2, 4, 64, 6, 2
    width = H * G * D
    b = Shared("int8", layers=L, heads=H, dim=D, page=16, n_pages=200, seqs=n, dtype=dtype, seed=31)
    b.family([(150, [3, 4, 5, 6, 7, 8])])
    g = torch.Generator().manual_seed(7)
    weights = [[w4.quantize(torch.randn(o, i, generator=g) * i ** -0.5, 64, z) for o, i, z in ((width + 2 * H * D, width, True), (width, width, False))]
               for _ in range(L)]
    dev = [[[None if t is None else t.cuda() for t in w] for w in layer] for layer in weights]
    gains = [1 + 0.1 * torch.randn(D, generator=g) for _ in range(2)]
    cfg = RotaryConfig(head_dim=D, rot_dim=32)
    rotary = native.Rotary(cfg, *[x.cuda() for x in gains])
    ids, groups = b.ids(range(n)), b.ids([0, n])
    x0 = b.rand(n, width).cuda()

    def step():
        x, seen = x0, []
        b.cache.extend(ids)
        for layer in range(L):
            qkv = native.gemm_w4(x, *dev[layer][0]).view(n, -1, D)
            q, k = b.cache.rotate(ids, rotary, qkv[:, :H * G], qkv[:, H * G:H * G + H])
            b.cache.write(layer, ids, k, qkv[:, H * G + H:])
            o = b.cache.attend_shared(layer, ids, q, groups=groups)
            y = native.gemm_w4(o.view(n, width), *dev[layer][1])
            seen.append((x, qkv, q, k, o, y))
            x = y
        return seen

    if graph:
        run = torch.cuda.CUDAGraph()
        with torch.cuda.graph(run):
            seen = step()
    for t in range(3):
        if graph:
            run.replay()
        else:
            seen = step()
        torch.cuda.synchronize()
        b.cache.check()
        for layer, (x, qkv, q, k, o, y) in enumerate(seen):
            want, tol = exact_w4(x.cpu(), *weights[layer][0], None)
            assert ((qkv.reshape(n, -1).double().cpu() - want).abs() <= tol).all()
            pos = torch.tensor([s.len for s in b.seqs])
            close(q, *exact(cfg, qkv[:, :H * G].cpu(), gains[0], pos), dtype)
            close(k, *exact(cfg, qkv[:, H * G:H * G + H].cpu(), gains[1], pos), dtype)
            for i in range(n):
                b.seqs[i].append(layer, "k", k[i:i + 1].float().cpu().numpy(), "int8")
                b.seqs[i].append(layer, "v", qkv[i:i + 1, H * G + H:].float().cpu().numpy(), "int8")
                b.seqs[i].len += 1
                ref = attend64(b.seqs[i], layer, q[i:i + 1].double().cpu().numpy(), G, D ** -0.5, -1, 1, 0, 16)
                b.seqs[i].len -= 1
                tol, _ = bounds(*ref, D, b.seqs[i].len, dtype)
                assert (np.abs(o[i:i + 1].double().cpu().numpy() - ref[0]) <= tol + 2.0 ** -19 * ref[2]).all()
            want, tol = exact_w4(o.reshape(n, width).cpu(), *weights[layer][1], None)
            assert ((y.double().cpu() - want).abs() <= tol).all()
        for s in b.seqs:
            s.len += 1
        b.verify()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group,prefix", [(2, True), (1, False)])
def test_nothing_of_ones_own_at_all(dtype, group, prefix):
    """Everything is shared: there are no pieces of the sequences' own tokens, and what joins the parts still waits for the shared ones'."""
    n = 40 if prefix else 9
    b = Shared("int8", heads=2, dim=64, page=32, n_pages=300, seqs=n, dtype=dtype, seed=n)
    b.family([(1024, [0] * n)])
    for _ in range(3):
        b.check_shared(range(n), [1] * n, None, group=group, uniform=True, prefix=prefix)


def test_calls_of_unlike_sizes_one_behind_the_other():
    """Launches start before those before them have ended: calls that follow each other in a graph, in one workspace, keep apart."""
    n = 64
    b = Shared("e4m3", heads=2, dim=128, page=32, n_pages=900, seqs=n, dtype=BF16, seed=5)
    rng = np.random.default_rng(5)
    b.family([(1500, rng.integers(0, 90, n // 2).tolist()), (700, rng.integers(0, 300, n // 2).tolist())])
    cases = []
    for ids, groups, group in [(range(n), [0, n // 2, n], 4), (range(3), None, 2), (range(20, 50), [0, 12, 30], 8), (range(n), None, 1)]:
        q = b.rand(len(ids), group * 2, 128).cuda()
        cases.append((b.ids(ids), q, None if groups is None else b.ids(groups)))
    attend = lambda: [b.cache.attend_shared(0, ids, q, groups=groups) for ids, q, groups in cases]  # noqa: E731
    want = []
    for ids, q, groups in cases:
        want.append(b.cache.attend_shared(0, ids, q, groups=groups).clone())
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [y for _ in range(3) for y in attend()]
    for _ in range(10):
        for y in got:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, y in enumerate(got):
            assert torch.equal(y, want[k % len(want)]), k
    b.cache.check()
