"""The paged 8-bit K/V cache on the GPU against a plain model of it: codes and scales
bit for bit, attention within bounds derived from the kernels' arithmetic."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from cache_aware_conformer_gb300.config import Kv8Config  # noqa: E402

from _kv8 import Seq, attend64, bounds  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INVAL, STATE, NOMEM, NONFINITE, LIMIT, BOUNDS = -1, -3, -4, -7, -10, -11


class Both:
    """A cache on the GPU and its plain model, driven together."""

    def __init__(self, code="int8", layers=1, heads=2, dim=64, page=32, n_pages=64, seqs=6, max_pages=40, dtype=F32, seed=0):
        from cache_aware_conformer_gb300 import native
        self.native = native
        self.cfg = Kv8Config(layers, heads, dim, page, n_pages, seqs, max_pages, code)
        self.cache = native.Kv8Cache(self.cfg)
        self.seqs = [Seq(layers, heads, dim) for _ in range(seqs)]
        self.dtype = dtype
        self.gen = torch.Generator().manual_seed(seed)

    def rand(self, *shape, gain=1.0):
        return (torch.randn(*shape, generator=self.gen) * gain).to(self.dtype)

    def ids(self, x):
        return torch.tensor(list(x), dtype=torch.int32, device="cuda")

    def starts(self, counts):
        return self.ids(np.concatenate([[0], np.cumsum(counts)]))

    def append(self, ids, counts, gain=1.0, k=None, v=None):
        T = int(np.sum(counts))
        st = self.starts(counts)
        self.cache.extend(self.ids(ids), starts=st)
        c = self.cfg
        for layer in range(c.n_layers):
            kk = self.rand(T, c.kv_heads, c.head_dim, gain=gain) if k is None else k
            vv = self.rand(T, c.kv_heads, c.head_dim, gain=gain) if v is None else v
            self.cache.write(layer, self.ids(ids), kk.cuda(), vv.cuda(), starts=st)
            at = 0
            for i, m in zip(ids, counts):
                self.seqs[i].append(layer, "k", kk[at:at + m].float().numpy(), c.code)
                self.seqs[i].append(layer, "v", vv[at:at + m].float().numpy(), c.code)
                at += m
        for i, m in zip(ids, counts):
            self.seqs[i].len += int(m)

    def fork(self, src, dst):
        self.cache.fork(self.ids(src), self.ids(dst))
        new = [self.seqs[s].copy() for s in src]
        for d, s in zip(dst, new):
            self.seqs[d] = s

    def truncate(self, ids, lens):
        self.cache.truncate(self.ids(ids), self.ids(lens))
        for i, n in zip(ids, lens):
            self.seqs[i].cut(n, self.cfg.page_tokens)

    def trim(self, ids, left, chunk, sinks):
        self.cache.trim(self.ids(ids), left, chunk, sinks)
        for i in ids:
            self.seqs[i].trim(left, chunk, sinks, self.cfg.page_tokens)

    def verify(self):
        """Everything that the cache holds, and its books."""
        c, cfg = self.cache, self.cfg
        c.check()
        lens = [s.len for s in self.seqs]
        assert c.lens.tolist() == lens
        table, refs = c.table.cpu().numpy(), c.refs.cpu().numpy()
        PT = cfg.page_tokens
        named = np.zeros(cfg.n_pages, int)
        for s, seq in enumerate(self.seqs):
            have = -(-seq.len // PT)
            assert (table[s, have:] == -1).all()
            assert [j for j in range(have) if table[s, j] < 0] == sorted(seq.gone)
            for p in table[s, :have]:
                if p >= 0:
                    named[p] += 1
        assert (named == refs).all()
        nf = int(c.n_free)
        free = c.free.cpu().numpy()[:nf]
        assert sorted(free) == [p for p in range(cfg.n_pages) if refs[p] == 0]
        w = c.work.cpu().numpy()
        assert not w[:2 * cfg.n_pages].any()        # extend's counters are back to zero
        longest = max(lens)
        if longest == 0:
            return
        ids = self.ids(range(cfg.max_seqs))
        for layer in range(cfg.n_layers):
            got = c.read(layer, ids, torch.zeros_like(ids), longest)
            for which, x in zip("kv", got):
                x = x.cpu().numpy()
                for s, seq in enumerate(self.seqs):
                    codes, scales = seq.values(layer, which)
                    want = np.zeros((longest, cfg.kv_heads, cfg.head_dim), np.float32)
                    want[:seq.len] = (codes * scales[..., None])[:seq.len]
                    for j in seq.gone:
                        want[j * PT:(j + 1) * PT] = 0
                    assert np.array_equal(x[s], want), (layer, which, s, np.abs(x[s] - want).max())

    def attend(self, ids, counts, group=2, left=-1, chunk=1, sinks=0, scale=None, layer=0, q=None, qgain=1.0, uniform=False,
               **kw):
        cfg = self.cfg
        T, heads = int(np.sum(counts)), group * cfg.kv_heads
        q = self.rand(T, heads, cfg.head_dim, gain=qgain) if q is None else q
        rag = {} if uniform else {"starts": self.starts(counts), "max_new": max(counts, default=0)}
        out, lse = self.cache.attend(layer, self.ids(ids), q.cuda(), att_left=left, att_chunk=chunk, sinks=sinks, scale=scale,
                                     lse=True, **rag, **kw)
        self.cache.check()
        assert out.dtype == q.dtype and out.shape == q.shape and lse.shape == (T, heads)
        sc = scale if scale is not None else cfg.head_dim ** -0.5
        at = 0
        for i, m in zip(ids, counts):
            if m == 0:
                continue
            ref = attend64(self.seqs[i], layer, q[at:at + m].double().numpy(), group, sc, left, chunk, sinks, cfg.page_tokens)
            tol, tol_lse = bounds(*ref, cfg.head_dim, max(self.seqs[i].len, 1), self.dtype)
            o, s = out[at:at + m].double().cpu().numpy(), lse[at:at + m].double().cpu().numpy()
            err = np.abs(o - ref[0])
            assert (err <= tol).all(), (i, m, float((err / tol).max()), float(err.max()))
            dead = ~np.isfinite(ref[1])
            assert (s[dead] == -np.inf).all() and (o[dead] == 0).all()
            err = np.abs(s[~dead] - ref[1][~dead])
            assert (err <= tol_lse[~dead]).all(), (i, float(err.max()))
            at += m
        return out, lse


# ---------------------------------------------------------------------------
# writing and reading
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,page,heads", [(16, 16, 1), (64, 32, 3), (80, 48, 2), (128, 64, 2), (256, 16, 1), (144, 16, 5)])
def test_written_values_bit_for_bit(code, dtype, dim, page, heads):
    b = Both(code, heads=heads, dim=dim, page=page, dtype=dtype, layers=2, seed=dim)
    b.append([0, 1, 2, 3, 4], [1, 15, 16, 17, 3 * page + 5])
    b.verify()
    for gain in (0.5, 4.0, 1e-3):      # smaller, larger (the blocks' scales grow) and much smaller values
        b.append([0, 2, 1, 4], [1, 0, 18, 1], gain=gain)
        b.verify()
    for _ in range(17):                # token by token over a block's border
        b.append([3, 5], [1, 1])
    b.verify()


def test_zeros_tiny_huge_and_non_finite_values():
    b = Both(heads=1, dim=32, page=16)
    x = torch.zeros(16, 1, 32)
    b.append([0], [16], k=x, v=x)                                 # a block of zeros
    b.append([0], [16], k=x + 1e-38, v=x + 3e38)                  # under the smallest scale; near the largest float
    b.verify()
    y = torch.randn(5, 1, 32, generator=b.gen)
    y[1, 0, 3], y[2, 0, 4], y[4, 0, 0] = float("nan"), float("inf"), -float("inf")
    z = torch.full((5, 1, 32), float("nan"))
    b.cache.extend(b.ids([1]), each=5)
    b.cache.write(0, b.ids([1]), y.cuda(), z.cuda())
    b.seqs[1].append(0, "k", y.numpy(), "int8")
    b.seqs[1].append(0, "v", z.numpy(), "int8")
    b.seqs[1].len = 5
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == NONFINITE
    b.verify()


def test_row_strides_and_slices_of_one_projection():
    b = Both(heads=2, dim=64, page=32, dtype=BF16)
    T, H, D = 21, 2, 64
    qkv = b.rand(T, 4 * H + 2, D).cuda()                           # a wider row than K and V together
    k, v = qkv[:, 1:1 + H], qkv[:, 4:4 + H]
    b.cache.extend(b.ids([2]), each=T)
    b.cache.write(0, b.ids([2]), k, v)
    for which, x in (("k", k), ("v", v)):
        b.seqs[2].append(0, which, x.float().cpu().numpy(), "int8")
    b.seqs[2].len = T
    b.verify()
    q = qkv[:, 6:10]
    out = torch.full((T, 7, D), 3.0, dtype=BF16, device="cuda")
    got = b.cache.attend(0, b.ids([2]), q, out=out[:, 2:6])
    want = b.cache.attend(0, b.ids([2]), q.contiguous())
    assert torch.equal(got, want)
    assert (out[:, :2] == 3).all() and (out[:, 6:] == 3).all()     # nothing beside it


def test_read_outside_a_sequence_is_zero():
    b = Both(dim=32, page=16)
    b.append([0, 1], [20, 3])
    k, v = b.cache.read(0, b.ids([0, 1, 2, 0]), b.ids([-4, 1, 0, 2 ** 31 - 3]), 30, dtype=BF16)
    b.cache.check()
    assert k.dtype == BF16 and k.shape == (4, 30, 2, 32)
    assert (k[0, :4] == 0).all() and (k[0, 24:] == 0).all() and (k[0, 4:24] != 0).any()
    assert (k[1, 2:] == 0).all() and (v[1, :2] != 0).any() and (k[2] == 0).all() and (v[3] == 0).all()
    b.cache.read(0, b.ids([-1, 7]), b.ids([0, 0]), 2)
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == BOUNDS


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("code,page", [("int8", 16), ("e4m3", 32), ("int8", 64)])
def test_a_life_of_forks_and_releases(code, page):
    """Random calls; after each, values, tables, counts and free pages are those of the model."""
    rng = np.random.RandomState(page)
    b = Both(code, layers=2, heads=2, dim=32, page=page, n_pages=90, seqs=8, max_pages=24, seed=page)
    for step in range(60):
        what = rng.randint(6)
        pick = list(rng.permutation(8)[:rng.randint(1, 5)])
        used = 90 - int(b.cache.n_free)
        if what <= 1 and used < 60:
            b.append(pick, list(rng.randint(0, 2 * page + 3, len(pick)) if rng.rand() < 0.5 else [1] * len(pick)))
        elif what == 2:
            src = list(rng.permutation(8)[:2])
            dst = [x for x in rng.permutation(8) if x not in src][:4]
            b.fork([src[j % 2] for j in range(len(dst))], dst)
        elif what == 3:
            b.truncate(pick, [int(rng.randint(0, b.seqs[i].len + 3)) // page * page for i in pick])
        elif what == 4:
            # a window that keeps the last page, so that the sequence can go on
            b.trim(pick, int(rng.randint(0, 2 * page)), int(rng.randint(1, 4)), int(rng.randint(0, page)))
        else:
            b.cache.compact()
            assert (b.cache.refs[:90 - int(b.cache.n_free)] > 0).all()
        if max(s.len for s in b.seqs) > 20 * page:
            long = [i for i, s in enumerate(b.seqs) if s.len > 20 * page]
            b.truncate(long, [0] * len(long))
        b.verify()


def test_a_shared_page_is_copied_once_too_few_times():
    """Three hypotheses share a half-full page: extended together, one keeps it and two take copies; with the parent
    still there, all three take copies."""
    for keep_parent in (True, False):
        b = Both(dim=32, page=32, layers=2)
        b.append([0], [40])
        b.fork([0, 0, 0], [1, 2, 3])
        if not keep_parent:
            b.truncate([0], [0])
        before = int(b.cache.n_free)
        b.append([1, 2, 3], [1, 2, 3])
        assert before - int(b.cache.n_free) == (3 if keep_parent else 2)
        b.verify()
        b.append([3, 2], [1, 1])          # their own pages by now
        assert before - int(b.cache.n_free) == (3 if keep_parent else 2)
        b.verify()


def test_compact_frees_one_piece_of_the_pool():
    b = Both(layers=3, dim=64, page=16, n_pages=200, seqs=10, max_pages=30)
    for _ in range(6):
        b.append(range(10), [37] * 10)
    b.fork([3], [9])
    b.truncate([0, 2, 4, 6], [0, 5, 100, 33])
    used = 200 - int(b.cache.n_free)
    b.cache.compact()
    refs = b.cache.refs.cpu().numpy()
    assert (refs[:used] > 0).all() and (refs[used:] == 0).all()
    b.verify()
    b.cache.compact()                     # nothing to move
    b.verify()
    b.truncate(range(10), [0] * 10)
    b.cache.compact()                     # empty
    b.verify()
    assert int(b.cache.n_free) == 200


def test_refused_calls_change_nothing():
    b = Both(dim=32, page=16, n_pages=10, seqs=6, max_pages=8)
    b.append([0, 1], [40, 20])
    err = b.native.CacError

    def latched(code, call):
        call()
        with pytest.raises(err) as e:
            b.cache.check()
        assert e.value.code == code
        b.verify()

    latched(NOMEM, lambda: b.cache.extend(b.ids([2, 3]), each=60))          # 8 pages, 5 free
    latched(LIMIT, lambda: b.cache.extend(b.ids([2, 0]), each=100))         # 140 tokens > 128
    latched(BOUNDS, lambda: b.cache.extend(b.ids([2, 6]), each=1))
    latched(BOUNDS, lambda: b.cache.extend(b.ids([-1, 2]), each=1))
    latched(BOUNDS, lambda: b.cache.extend(b.ids([2, 3]), starts=b.ids([0, 4, 2])))
    latched(INVAL, lambda: b.cache.extend(b.ids([2, 3, 2]), each=1))
    latched(INVAL, lambda: b.cache.truncate(b.ids([0, 1, 0, 1]), 3))
    latched(BOUNDS, lambda: b.cache.truncate(b.ids([6]), 3))
    latched(BOUNDS, lambda: b.cache.truncate(b.ids([0]), b.ids([-1])))
    latched(INVAL, lambda: b.cache.trim(b.ids([0, 0]), 4))
    latched(BOUNDS, lambda: b.cache.trim(b.ids([99]), 4))
    latched(INVAL, lambda: b.cache.fork(b.ids([0, 1]), b.ids([3, 3])))
    latched(INVAL, lambda: b.cache.fork(b.ids([0, 1]), b.ids([1, 1])))
    latched(INVAL, lambda: b.cache.fork(b.ids([0]), b.ids([0])))
    latched(BOUNDS, lambda: b.cache.fork(b.ids([0]), b.ids([6])))
    x = torch.randn(8, 2, 32, device="cuda")
    latched(STATE, lambda: b.cache.write(0, b.ids([2]), x, x))              # nothing was extended
    b.cache.extend(b.ids([0, 1]), each=4)
    b.seqs[0].len, b.seqs[1].len = 44, 24
    call = lambda ids, **kw: b.cache.write(0, b.ids(ids), x, x, **kw)       # noqa: E731

    def refused(code, ids, **kw):
        before = b.cache.k.clone()
        call(ids, **kw)
        with pytest.raises(err) as e:
            b.cache.check()
        same = torch.equal(before, b.cache.k)
        assert e.value.code == code and same

    refused(STATE, [1, 0])                                                  # another order
    refused(STATE, [2, 3])
    call([0, 1], starts=b.ids([0, 4, 9]))                                   # rows past the tensor: the first is written
    with pytest.raises(err) as e:
        b.cache.check()
    assert e.value.code == BOUNDS


def test_one_bad_sequence_leaves_the_others_written():
    b = Both(dim=32, page=16)
    b.cache.extend(b.ids([0, 1]), each=4)
    x = b.rand(8, 2, 32)
    b.cache.write(0, b.ids([0, 3]), x.cuda(), x.cuda())
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == STATE
    for w in "kv":
        b.seqs[0].append(0, w, x[:4].numpy(), "int8")
    got = b.cache.read(0, b.ids([0]), b.ids([0]), 4)[0][0].cpu().numpy()
    c, s = b.seqs[0].values(0, "k")
    assert np.array_equal(got, c * s[..., None])


def test_a_fork_ends_the_right_to_write():
    b = Both(dim=32, page=16)
    b.append([0], [20])
    b.cache.extend(b.ids([0]), each=3)
    b.cache.fork(b.ids([0]), b.ids([1]))
    x = torch.randn(3, 2, 32, device="cuda")
    before = b.cache.k.clone()
    b.cache.write(0, b.ids([0]), x, x)
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == STATE and torch.equal(before, b.cache.k)


def test_extend_after_the_window_passed_the_last_page():
    """A truncate into pages that trim released: the tokens there are lost, and the sequence cannot go on from them."""
    b = Both(dim=32, page=16)
    b.append([0], [100])
    b.trim([0], 10, 1, 0)
    b.truncate([0], [40])
    b.cache.extend(b.ids([0]), each=1)
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == STATE
    b.verify()
    b.truncate([0], [32])                  # a page's border is fine
    b.append([0], [5])
    b.verify()
    b.attend([0], [2])


def test_tokens_trimmed_before_they_are_written():
    b = Both(dim=32, page=16)
    b.cache.extend(b.ids([0]), each=70)
    b.trim([0], 4, 1, 0)                   # length 0 in the model: nothing to release there
    b.seqs[0].len = 70
    b.seqs[0].trim(4, 1, 0, 16)
    x = b.rand(70, 2, 32)
    b.cache.write(0, b.ids([0]), x.cuda(), x.cuda())
    b.seqs[0].len = 0
    for w in "kv":
        b.seqs[0].append(0, w, x.numpy(), "int8")
    b.seqs[0].len = 70
    b.verify()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,page,group", [(64, 16, 1), (128, 32, 4), (80, 48, 3), (16, 16, 8), (256, 64, 2), (64, 64, 17)])
def test_single_tokens(code, dtype, dim, page, group):
    b = Both(code, dim=dim, page=page, dtype=dtype, seqs=7, n_pages=100, seed=group)
    b.append(range(6), [1, 2, 16, 33, 2 * page + 7, 300])
    b.attend([5, 0, 3, 1, 4, 2], [1] * 6, group=group, uniform=True)
    b.attend([5, 6, 1], [1, 1, 1], group=group)                      # one is empty: its row sees nothing


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("left,chunk,sinks", [(-1, 1, 0), (70, 2, 0), (10, 1, 4), (0, 1, 0), (0, 4, 1), (33, 8, 40), (5, 1000, 2),
                                              (200, 3, 17)])
def test_windows_and_sinks(dtype, left, chunk, sinks):
    b = Both(dim=64, page=32, dtype=dtype, n_pages=100)
    b.append(range(5), [1, 30, 64, 129, 257])
    for counts in ([1] * 5, [1, 2, 5, 3, 7], [1, 30, 9, 65, 100], [0, 3, 0, 129, 1]):
        b.attend(range(5), counts, left=left, chunk=chunk, sinks=sinks)


@pytest.mark.parametrize("code,dtype", [("int8", BF16), ("e4m3", F32)])
@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (5, 80), (8, 64)])
def test_prompts(code, dtype, group, dim):
    """As many queries as keys, ragged, odd; tiles that end inside pages."""
    b = Both(code, heads=1, dim=dim, page=48, dtype=dtype, n_pages=100, seed=dim)
    lens = [131, 260, 1, 77, 16]
    b.append(range(5), lens)
    b.attend(range(5), lens, group=group)
    b.attend([1, 0], [129, 128], group=group, left=64, sinks=5)


def test_long_sequences_split_over_the_card():
    b = Both("int8", heads=1, dim=64, page=64, dtype=BF16, n_pages=400, seqs=3, max_pages=320)
    b.append([0, 1], [20000, 3000])
    b.attend([0], [1], group=4)
    b.attend([1, 0], [1, 3], group=2)
    b.attend([0, 1], [2, 2], group=1, left=9000, sinks=100)
    b.attend([0], [1], group=1, left=5, sinks=12000)


def test_released_pages_are_not_seen():
    b = Both(dim=64, page=16, n_pages=100)
    b.append([0, 1], [200, 90])
    b.trim([0], 30, 1, 20)
    b.attend([0, 1], [1, 1])                    # no window here: what is left of 0 is seen
    b.attend([0, 1], [40, 3], left=50, sinks=3)
    b.attend([0], [150])                        # positions whose own pages are gone


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 80])
def test_codes_that_no_write_filled_are_never_seen(code, dim):
    """Pages may hold anything before: 0xff is NaN as e4m3, and the scales are NaN too."""
    b = Both(code, dim=dim, page=48, dtype=BF16, n_pages=60)
    for t in (b.cache.k, b.cache.v):
        t.fill_(-1)
    for t in (b.cache.k_scale, b.cache.v_scale):
        t.fill_(float("nan"))
    b.append([0, 1, 2, 3], [1, 17, 150, 300])
    b.verify()
    for counts in ([1] * 4, [1, 2, 3, 4], [1, 17, 150, 300]):
        b.attend([0, 1, 2, 3], counts)
        b.attend([0, 1, 2, 3], counts, left=20, sinks=3)


def test_more_queries_than_tokens():
    """Positions before 0 see nothing."""
    b = Both(dim=64, page=16)
    b.append([0, 1], [3, 20])
    b.attend([0, 1, 2], [6, 2, 2])


def test_rows_of_no_sequence_are_left_alone():
    b = Both(dim=64, page=16)
    b.append([0, 1], [30, 40])
    q = torch.randn(20, 4, 64, device="cuda")
    out = torch.full_like(q, 7.0)
    b.cache.attend(0, b.ids([0, 1]), q, starts=b.ids([3, 8, 12]), max_new=5, out=out)
    b.cache.check()
    assert (out[:3] == 7).all() and (out[12:] == 7).all()
    want = b.cache.attend(0, b.ids([0]), q[3:8].contiguous())
    assert torch.equal(out[3:8], want)


def test_bad_ids_and_counts_give_zero_rows():
    b = Both(dim=64, page=16)
    b.append([0], [30])
    q = torch.randn(4, 4, 64, device="cuda")
    for ids, kw in (([0, 6], {}), ([-1, 0], {}), ([0, 1], {"starts": [0, 1, 4], "max_new": 2})):
        kw = {k: b.ids(v) if k == "starts" else v for k, v in kw.items()}
        out, lse = b.cache.attend(0, b.ids(ids), q, lse=True, **kw)
        with pytest.raises(b.native.CacError) as e:
            b.cache.check()
        assert e.value.code == BOUNDS
        bad = {0: slice(2, 4), 1: slice(0, 2), 2: slice(1, 4)}[[([0, 6]), ([-1, 0]), ([0, 1])].index(ids)]
        assert (out[bad] == 0).all() and (lse[bad] == -np.inf).all()


@pytest.mark.parametrize("left", [-1, 8])
@pytest.mark.parametrize("max_new,rows", [(1, 9), (2, 40), (40, 300)])
def test_counts_above_max_new_give_zero_rows(left, max_new, rows):
    """Every row of such a sequence, however many tiles of rows it has."""
    b = Both(dim=64, page=16)
    b.append([0, 1], [30, 9])
    q = torch.randn(rows + 1, 4, 64, device="cuda")
    out = torch.full_like(q, 5.0)
    _, lse = b.cache.attend(0, b.ids([0, 1]), q, starts=b.ids([0, 1, rows + 1]), max_new=max_new, att_left=left, out=out,
                            lse=True)
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == BOUNDS
    assert (out[1:] == 0).all() and (lse[1:] == -np.inf).all() and (out[0] != 5).any()


def test_unlike_scales_of_blocks():
    """Blocks whose V values differ by many powers of two, and logits far apart."""
    b = Both(dim=64, page=16, dtype=F32)
    for gain in (1e-4, 1.0, 300.0, 1e-2, 30.0, 1e-6):
        b.append([0], [16], k=b.rand(16, 2, 64), v=b.rand(16, 2, 64, gain=gain))
    b.attend([0], [1])
    b.attend([0], [5], qgain=20.0)
    b.attend([0], [96], qgain=1e-3)
    b.attend([0], [3], scale=0.0)
    b.attend([0], [3], scale=-0.3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,group", [(64, 8), (128, 4), (256, 7), (64, 12)])
def test_maxima_that_rise_and_fall(dtype, dim, group):
    """Logits that climb by less or more than a few powers of two a block, fall, or stand still, in rows side by side."""
    b = Both(dim=dim, page=32, dtype=dtype, n_pages=64)
    line = torch.randn(dim, generator=torch.Generator().manual_seed(3))
    line /= line.norm()
    tokens = 430
    k = b.rand(tokens, 2, dim, gain=0.05) + (torch.arange(tokens) / 16.0)[:, None, None].to(dtype) * line.to(dtype)
    b.append([0], [tokens], k=k.to(dtype))
    step = torch.tensor([0.0, 0.3, 0.7, 1.0, 1.5, 4.0, -0.7, -4.0, 12.0, -12.0, 2.0, 1.9])   # powers of two a block
    q = step[torch.arange(2 * group) % 12, None] * 0.6931 * dim ** 0.5 * line
    b.attend([0], [1], group=group, q=q[None].to(dtype))
    b.attend([0], [1], group=group, q=q[None].to(dtype), left=100, sinks=20)


def test_non_finite_queries_stay_in_their_rows():
    b = Both(dim=64, page=16, dtype=F32)
    b.append([0], [40])
    q = torch.randn(20, 4, 64, device="cuda")
    want = b.cache.attend(0, b.ids([0]), q)
    q2 = q.clone()
    q2[5, 1, 3], q2[9, 2, 0], q2[9, 3] = float("nan"), float("inf"), 0.0
    got = b.cache.attend(0, b.ids([0]), q2)
    assert got[5, 1].isnan().all() and not torch.isfinite(got[9, 2]).any()
    ok = torch.ones(20, 4, dtype=torch.bool, device="cuda")
    ok[5, 1] = ok[9, 2] = ok[9, 3] = False
    assert torch.equal(got[ok], want[ok])
    assert torch.isfinite(got[9, 3]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_queries_of_few_rows(dtype, bad):
    b = Both(dim=128, page=16, dtype=dtype, n_pages=100)
    b.append([0, 1], [600, 33])
    b.cache.check()
    q = torch.randn(4, 4, 128, device="cuda").to(dtype)              # two tokens each, two heads to a K/V head: four rows
    want = b.cache.attend(0, b.ids([0, 1]), q)
    q2 = q.clone()
    q2[1, 2, 5] = bad
    got = b.cache.attend(0, b.ids([0, 1]), q2)
    ok = torch.ones(4, 4, dtype=torch.bool, device="cuda")
    ok[1, 2] = False
    assert not torch.isfinite(got[1, 2]).any() and torch.equal(got[ok], want[ok])


@pytest.mark.parametrize("n,longest,left,group,dim", [(160, 900, 950, 4, 64), (20, 480, 500, 12, 64), (21, 470, 490, 1, 128),
                                                      (40, 450, 470, 7, 128), (13, 400, 420, 16, 64)])
def test_units_cut_anywhere_and_whole_units_agree(n, longest, left, group, dim):
    """A window that shows everything makes a warp take whole units; without one the tiles are dealt out over the card and
    joined.  Both are within bounds() of the exact result: with sums of |q k| of at most 8 that is 1.4e-4 of sum p |v| <= 4 for each
    weight, twice for each side."""
    cfg = Kv8Config(1, 8, dim, 16, n * (longest // 16 + 1), n, 4096)
    from cache_aware_conformer_gb300 import native
    cache = native.Kv8Cache(cfg)
    gen = torch.Generator().manual_seed(n)
    ids = torch.randperm(n, generator=gen).to(torch.int32).cuda()
    counts = torch.randint(1, longest + 1, (n,), generator=gen, dtype=torch.int32)
    starts = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).to(torch.int32)]).cuda()
    k = torch.randn(int(counts.sum()), 8, dim, generator=gen).clamp(-4, 4).cuda() / 2
    v = torch.randn(int(counts.sum()), 8, dim, generator=gen).clamp(-4, 4).cuda()
    cache.extend(ids, starts=starts)
    cache.write(0, ids, k, v, starts=starts)
    q = torch.randn(n, 8 * group, dim, generator=gen).clamp(-4, 4).cuda() / 2
    whole, wl = cache.attend(0, ids, q, att_left=left, lse=True)
    dealt, dl = cache.attend(0, ids, q, lse=True)
    cache.check()
    assert torch.isfinite(whole).all() and torch.isfinite(wl).all()
    assert (whole - dealt).abs().max() <= 4 * 1.4e-4 * 4 and (wl - dl).abs().max() <= 4e-4
    assert not torch.equal(whole, dealt)     # the two ways are two ways


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code,dim,group,left,chunk,sinks", [("int8", 64, 2, -1, 1, 0), ("e4m3", 128, 3, 500, 4, 5), ("int8", 80, 1, 1700, 1, 33),
                                                             ("e4m3", 64, 8, 1001, 16, 0)])
def test_queries_of_a_prompt_and_alone_agree(dtype, code, dim, group, left, chunk, sinks):
    """The last queries of long pieces against the same queries asked for alone, which other kernels answer.  Tolerances as in
    bounds(): sums of |q k| of at most 8, sum p |v| <= 4.1, 3,600 keys."""
    n, heads = 5, 4
    counts = torch.tensor([3600, 1201, 2222, 1500, 2999], dtype=torch.int32)
    from cache_aware_conformer_gb300 import native
    cache = native.Kv8Cache(Kv8Config(1, heads, dim, 16, 760, n, 240, code))
    gen = torch.Generator().manual_seed(dim + group)
    ids = torch.tensor([3, 0, 4, 1, 2], dtype=torch.int32, device="cuda")
    starts = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).to(torch.int32)]).cuda()
    k = (torch.randn(int(counts.sum()), heads, dim, generator=gen).clamp(-4, 4) / 2).cuda().to(dtype)
    v = torch.randn(int(counts.sum()), heads, dim, generator=gen).clamp(-4, 4).cuda().to(dtype)
    cache.extend(ids, starts=starts)
    cache.write(0, ids, k, v, starts=starts)
    q = (torch.randn(n, 1200, heads * group, dim, generator=gen).clamp(-4, 4) / 2).cuda().to(dtype)
    args = dict(att_left=left, att_chunk=chunk, sinks=sinks, lse=True)
    out, lse = cache.attend(0, ids, q.reshape(n * 1200, -1, dim), **args)
    out, lse = out.reshape(n, 1200, -1, dim).float(), lse.reshape(n, 1200, -1)
    w = (dim + 8) * 2.0 ** -24 * 8 + 2.0 ** -23 * 136 + 2.0 ** -21 + 3600 * 2.0 ** -24
    e = w + (2.0 ** -11 if dtype == BF16 else 2.0 ** -20)
    for m in (1, 2, 5, 40):
        o, s = cache.attend(0, ids, q[:, -m:].reshape(n * m, -1, dim), **args)
        o, s = o.reshape(n, m, -1, dim).float(), s.reshape(n, m, -1)
        cache.check()
        assert torch.isfinite(s).all()
        assert ((o - out[:, -m:]).abs() <= 4 * e * 4.1 + torch.finfo(dtype).eps * o.abs()).all(), m
        assert (s - lse[:, -m:]).abs().max() <= 2 * (w + 2.0 ** -22 * 140), m


def test_the_same_sequence_twice_and_deterministic():
    b = Both(dim=128, page=32, dtype=BF16, n_pages=300, max_pages=200)
    b.append([0, 1], [4000, 50])
    q = b.rand(3, 4, 128).cuda()
    q[2] = q[0]
    a1 = b.cache.attend(0, b.ids([0, 1, 0]), q)
    a2 = b.cache.attend(0, b.ids([0, 1, 0]), q)
    assert torch.equal(a1, a2)
    tol = 2.0 ** -7 * a1[0].float().abs().max()      # another split of the keys: roundings of the sums, and one of the output
    assert (a1[0].float() - a1[2].float()).abs().max() <= tol


@pytest.mark.parametrize("counts", ["ones", "ragged", "prompts"])
def test_more_sequences_than_one_launch_takes(counts):
    """1,300 sequences in one call: extend plans 1,024 at a time, attention launches 512 at a time."""
    n = 1300
    b = Both(heads=1, dim=16, page=16, n_pages=8000, seqs=n + 20, max_pages=6, dtype=F32)
    rng = np.random.RandomState(3)
    ids = rng.permutation(n)
    first = rng.randint(1, 40, n)
    b.append(ids, list(first))
    b.fork(list(ids[:20]), list(range(n, n + 20)))          # shared pages in the next extend, some in each chunk
    new = {"ones": np.ones(n, int), "ragged": rng.randint(0, 4, n), "prompts": rng.randint(0, 40, n)}[counts]
    all_ids = list(ids) + list(range(n, n + 20))
    all_new = list(new) + [int(x) for x in new[:20]]
    b.append(all_ids, all_new)
    b.verify()
    b.attend(all_ids, all_new, uniform=counts == "ones")
    b.attend(all_ids, all_new, left=7, sinks=2, uniform=counts == "ones")


def test_pools_past_two_gigabytes():
    """Page numbers whose byte offsets pass 2^31 and 2^32."""
    from cache_aware_conformer_gb300 import native
    b = Both(heads=1, dim=16, page=16, n_pages=4, seqs=3, max_pages=4, dtype=BF16)
    cfg = Kv8Config(2, 16, 256, 64, 9000, 3, 6, "int8")     # 2.4 GB a layer for K and as much for V
    pages = torch.arange(9000, dtype=torch.int32, device="cuda")
    b.cfg, b.seqs = cfg, [Seq(2, 16, 256) for _ in range(3)]
    b.cache = native.Kv8Cache(cfg, tensors={
        "table": torch.full((3, 6), -1, dtype=torch.int32, device="cuda"), "lens": torch.zeros(3, dtype=torch.int32, device="cuda"),
        "refs": torch.zeros(9000, dtype=torch.int32, device="cuda"), "free": pages, "n_free": pages[:1] + 9000})
    b.append([0, 1], [70, 130])                              # the pool's last pages
    assert int(b.cache.table[0, 0]) > 8900
    b.verify()
    b.attend([0, 1], [1, 1], layer=1)
    b.attend([0, 1], [2, 40], layer=1)
    b.fork([1], [2])
    b.append([1, 2], [3, 5])
    b.cache.compact()
    assert int(b.cache.table.max()) < 10
    b.verify()


@pytest.mark.parametrize("heads,group", [(1, 128), (2, 40), (5, 7)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_query_heads_to_a_kv_head(heads, group, dtype):
    b = Both(heads=heads, dim=64, page=32, dtype=dtype)
    b.append([0, 1, 2], [5, 64, 150])
    b.attend([0, 1, 2], [1, 1, 1], group=group, uniform=True)
    b.attend([2, 1], [7, 3], group=group, left=40)


def test_extremes_of_the_window():
    big = 2 ** 31 - 1
    b = Both(dim=64, page=16)
    b.append([0, 1], [100, 37])
    for left, chunk, sinks in ((big, 1, 0), (0, 1, big), (3, big, 0), (big, big, big), (0, 1, 0)):
        b.attend([0, 1], [1, 1], left=left, chunk=chunk, sinks=sinks)
        b.attend([0, 1], [40, 37], left=left, chunk=chunk, sinks=sinks)
    b.trim([0], big, big, 0)
    b.trim([1], 0, 1, big)
    b.verify()


def test_empty_calls():
    b = Both(dim=64, page=16)
    b.append([0], [5])
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 4, 64, device="cuda")
    assert b.cache.attend(0, none, q).shape == (0, 4, 64)
    assert b.cache.attend(0, b.ids([0, 1]), q, starts=b.ids([0, 0, 0])).shape == (0, 4, 64)
    out, lse = b.cache.attend(0, b.ids([0]), torch.randn(3, 4, 64, device="cuda"), starts=b.ids([1, 1]), max_new=0, lse=True,
                              out=torch.full((3, 4, 64), 2.0, device="cuda"))
    assert (out == 2).all()
    x = torch.empty(0, 2, 64, device="cuda")
    b.cache.extend(none), b.cache.write(0, none, x, x), b.cache.fork(none, none), b.cache.truncate(none), b.cache.trim(none, 3)
    b.cache.extend(b.ids([0]), each=0), b.cache.write(0, b.ids([0]), x, x)
    assert b.cache.read(0, none, none, 4)[0].shape == (0, 4, 2, 64) and b.cache.read(0, b.ids([0]), b.ids([0]), 0)[1].shape[1] == 0
    b.verify()


def test_starts_past_the_rows_touch_nothing():
    b = Both(dim=64, page=16)
    b.append([0, 1], [30, 40])
    for rows, starts in ((8, [0, 5, 9]), (30, [0, 25, 60]), (8, [0, 5, -3])):
        q = torch.randn(rows, 4, 64, device="cuda")
        out = torch.full_like(q, 9.0)
        b.cache.attend(0, b.ids([0, 1]), q, starts=b.ids(starts), max_new=40, out=out)
        with pytest.raises(b.native.CacError) as e:
            b.cache.check()
        assert e.value.code == BOUNDS
        assert (out[starts[1]:] == 9).all() and (out[:starts[1]] != 9).any()


# ---------------------------------------------------------------------------
# streams, graphs, a step
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("left", [-1, 8, 5000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_starts_that_fall_are_refused(dtype, left):
    """Between starts that fall, a tile or block number may stand before its sequence's first: nothing there is touched."""
    b = Both(dim=64, page=16, dtype=dtype, n_pages=60)
    good, bad = b.ids([0, 160, 192, 232, 252]), b.ids([0, 160, 192, 20, 40])
    ids = b.ids([3, 0, 1, 2])
    b.cache.extend(ids, starts=good)
    x = torch.randn(252, 2, 64, device="cuda").to(dtype)
    tables, k_scale = b.cache.table.clone(), b.cache.k_scale.clone()
    b.cache.write(0, ids, x, x, starts=bad)
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code in (BOUNDS, STATE) and torch.equal(tables, b.cache.table)
    b.cache.write(0, ids, x, x, starts=good)
    b.cache.check()
    q = torch.randn(252, 4, 64, device="cuda").to(dtype)
    fence = torch.full((252 + 200, 4, 64), 7.0, device="cuda", dtype=dtype)
    out = fence[100:352]
    b.cache.attend(0, ids, q, att_left=left, starts=bad, max_new=160, out=out)
    with pytest.raises(b.native.CacError) as e:
        b.cache.check()
    assert e.value.code == BOUNDS
    assert (fence[:100] == 7).all() and (fence[352:] == 7).all()
    out2, lse = b.cache.attend(0, ids, q, att_left=left, starts=good, max_new=160, lse=True)
    b.cache.check()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("m", [1, 60])
def test_a_first_call_inside_a_capture(m):
    """Nothing has to be set up outside: kernels of a head size that no other test of this process uses."""
    b = Both("e4m3", heads=1, dim=112 if m > 1 else 48, page=16, dtype=BF16, n_pages=60)
    b.append([0, 1], [70, 300])
    q = b.rand(2 * m, 3, b.cfg.head_dim).cuda()
    ids = b.ids([0, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.cache.attend(0, ids, q)
    graph.replay()
    first = out.clone()
    graph.replay()
    b.cache.check()
    assert torch.equal(out, first) and torch.equal(b.cache.attend(0, ids, q), first)


def test_two_captured_graphs_replayed_at_once():
    """Attention captured twice, replayed on two streams at the same time: each has a workspace of its own."""
    b = Both(dim=128, page=32, dtype=BF16, n_pages=700, max_pages=660, seqs=3)
    b.append([0, 1], [20000, 900])
    ids, graphs, outs, want = b.ids([0, 1]), [], [], []
    for _ in range(2):
        q = b.rand(2, 8, 128).cuda()
        want.append(b.cache.attend(0, ids, q))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.cache.attend(0, ids, q))
        graphs.append((g, q))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    b.cache.check()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_a_captured_step_replays():
    """Extend, write and attend captured once; each replay goes one token further."""
    b = Both(dim=64, page=16, dtype=BF16, n_pages=200, layers=2)
    b.append([0, 1, 2], [5, 40, 100])
    ids = b.ids([0, 1, 2])
    k, v, q = (torch.zeros(3, h, 64, dtype=BF16, device="cuda") for h in (2, 2, 4))
    outs = [torch.zeros_like(q) for _ in range(2)]

    def step():
        b.cache.extend(ids)
        for layer in range(2):
            b.cache.write(layer, ids, k, v)
            b.cache.attend(layer, ids, q, out=outs[layer], att_left=70, att_chunk=2, sinks=1)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.cache.read(0, ids, ids, 1)                 # whatever is set up on first use
        b.cache.attend(0, ids, q, att_left=70, att_chunk=2, sinks=1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(20):
        kk, vv, qq = b.rand(3, 2, 64), b.rand(3, 2, 64), b.rand(3, 4, 64)
        k.copy_(kk), v.copy_(vv), q.copy_(qq)
        graph.replay()
        torch.cuda.synchronize()
        for i in range(3):
            for layer in range(2):
                b.seqs[i].append(layer, "k", kk[i:i + 1].float().numpy(), "int8")
                b.seqs[i].append(layer, "v", vv[i:i + 1].float().numpy(), "int8")
            b.seqs[i].len += 1
            for layer in range(2):
                ref = attend64(b.seqs[i], layer, qq[i:i + 1].double().numpy(), 2, 0.125, 70, 2, 1, 16)
                tol, _ = bounds(*ref, 64, 200, BF16)
                assert (np.abs(outs[layer][i:i + 1].double().cpu().numpy() - ref[0]) <= tol).all(), (t, i, layer)
    b.verify()


def test_attention_on_several_streams_at_once():
    b = Both(dim=128, page=32, dtype=BF16, n_pages=900, max_pages=800, seqs=3)
    b.append([0, 1], [20000, 300])
    q = [b.rand(2, 8, 128).cuda() for _ in range(6)]
    ids = b.ids([0, 1])
    want = [b.cache.attend(0, ids, x) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(5):
        got = [b.cache.attend(0, ids, x, stream=s) for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert torch.equal(a, w)


def test_calls_on_another_stream_than_the_tensors_own():
    """Everything on a side stream, its inputs dropped at once: their memory is not given out again before it has been read."""
    b = Both(dim=128, page=32, dtype=BF16, n_pages=300, max_pages=200)
    side = torch.cuda.Stream()
    outs, qs = [], []
    for step in range(6):
        kk, vv, qq = b.rand(400, 2, 128), b.rand(400, 2, 128), b.rand(2, 8, 128)
        k, v, q, ids = kk.cuda(), vv.cuda(), qq.cuda(), b.ids([1, 3])
        side.wait_stream(torch.cuda.current_stream())
        b.cache.extend(ids, each=200, stream=side)
        b.cache.write(0, ids, k, v, stream=side)
        outs.append(b.cache.attend(0, ids, q, stream=side))
        del k, v, q, ids
        torch.full((2, 400, 2, 128), float("nan"), device="cuda", dtype=BF16)      # takes what is free
        for n, i in enumerate((1, 3)):
            b.seqs[i].append(0, "k", kk[200 * n:200 * n + 200].float().numpy(), "int8")
            b.seqs[i].append(0, "v", vv[200 * n:200 * n + 200].float().numpy(), "int8")
            b.seqs[i].len += 200
        qs.append(qq)
    torch.cuda.synchronize()
    b.verify()
    for n, i in enumerate((1, 3)):
        ref = attend64(b.seqs[i], 0, qs[-1][n:n + 1].double().numpy(), 4, 128 ** -0.5, -1, 1, 0, 32)
        tol, _ = bounds(*ref, 128, 1200, BF16)
        assert (np.abs(outs[-1][n:n + 1].double().cpu().numpy() - ref[0]) <= tol).all()


def test_binding_refuses_bad_tensors():
    b = Both(dim=64, page=16)
    b.append([0], [5])
    ids, q = b.ids([0]), torch.randn(1, 4, 64, device="cuda")
    bad = [lambda: b.cache.attend(0, ids.long(), q), lambda: b.cache.attend(0, ids.cpu(), q),
           lambda: b.cache.attend(0, ids, q.double()), lambda: b.cache.attend(0, ids, q.half()),
           lambda: b.cache.attend(0, ids, q[..., :32]), lambda: b.cache.attend(0, ids, q.cpu()),
           lambda: b.cache.attend(0, ids, q.transpose(0, 1).expand(4, 4, 64)[:1]),
           lambda: b.cache.attend(0, ids, q, out=torch.empty(2, 4, 64, device="cuda")),
           lambda: b.cache.attend(0, ids, q, out=torch.empty(1, 4, 64, device="cuda", dtype=BF16)),
           lambda: b.cache.attend(0, ids, q, starts=b.ids([0])),
           lambda: b.cache.write(0, ids, q, q), lambda: b.cache.write(0, ids, q[:, :2], q[:, :2].bfloat16()),
           lambda: b.cache.read(0, ids, b.ids([0, 1]), 1), lambda: b.cache.read(0, ids, ids, 1, dtype=torch.half),
           lambda: b.cache.fork(ids, b.ids([1, 2])), lambda: b.cache.truncate(ids, ids.cpu())]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(b.native.CacError):
        b.cache.attend(0, ids, torch.randn(1, 3, 64, device="cuda"))          # heads not a multiple
    with pytest.raises(ValueError):
        b.native.Kv8Cache(b.cfg, tensors={"k": b.cache.k})
    b.cache.check()
