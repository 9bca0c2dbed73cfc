"""Attention behind a shared prefix, in a workspace that the test holds: what a call reads of it, and what it finds to be shared."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from _kv8 import attend64, bounds  # noqa: E402
from test_gpu_kv8 import Both  # noqa: E402
from test_gpu_kv8_shared import Shared  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


class Sized(Shared):
    """With tables for so many tokens."""

    def __init__(self, tokens, code="int8", layers=1, heads=2, dim=64, page=32, n_pages=64, seqs=6, dtype=F32, seed=0):
        Both.__init__(self, code, layers, heads, dim, page, n_pages, seqs, -(-tokens // page), dtype, seed)


class Call:
    """A call of cac_kv8_attend_shared with a row for each sequence, into an output and a workspace of its own."""

    def __init__(self, b, ids, q, groups=None, left=-1, chunk=1, sinks=0):
        self.b, self.n, self.q = b, len(ids), q.cuda()
        self.ids, self.groups = b.ids(ids), None if groups is None else b.ids(groups)
        self.n_groups = 0 if groups is None else len(groups) - 1
        self.out = torch.empty_like(self.q)
        self.window = (left, chunk, sinks)
        self.lib, self.ref = b.native.lib(), b.cache._ref
        need = self.lib.cac_kv8_attend_shared_workspace(self.ref, self.n, self.n, 1, self.n_groups, q.shape[1], *self.window)
        self.space = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(self):
        q, out = self.q, self.out
        r = self.lib.cac_kv8_attend_shared(
            self.ref, 0, self.n, self.ids.data_ptr(), None, self.n, 1, self.n_groups, None if self.groups is None else self.groups.data_ptr(),
            q.shape[1], q.shape[2] ** -0.5, *self.window, q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0), None,
            1 if q.dtype is BF16 else 0, self.space.data_ptr(), self.space.numel(), torch.cuda.current_stream().cuda_stream)
        assert r == 0
        return out


@pytest.mark.parametrize("n,heads,dim", [(64, 8, 128), (9, 2, 64), (20, 6, 144)])
def test_nothing_of_a_workspace_is_read_before_the_call_has_written_it(n, heads, dim):
    """Calls behind one another over a workspace that is filled with other bytes before each: whatever a launch reads of it, it has
    waited for."""
    b = Shared("int8", heads=2, dim=dim, page=32, n_pages=700, seqs=n, dtype=BF16, seed=n)
    rng = np.random.default_rng(n)
    st = b.family([(1500, rng.integers(0, 200, n // 2).tolist()), (700, rng.integers(0, 90, n - n // 2).tolist())])
    call = Call(b, range(n), b.rand(n, heads, dim), st)
    want = call.run().clone()
    b.check_shared(range(n), [1] * n, st, group=heads // 2, uniform=True, q=call.q.cpu())
    graph, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for fill in (0, 255, 1, 127):
            call.space.fill_(fill)
            outs.append(call.run().clone())
            outs.append(call.run().clone())
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    b.cache.check()
    assert all(torch.equal(x, want) for x in outs)


@pytest.mark.parametrize("dtype,n,group,heads,dim,tokens,shares", [
    (F32, 24, 16, 4, 64, 5600, False), (F32, 24, 16, 4, 64, 5800, True), (BF16, 32, 4, 8, 128, 1040, False), (BF16, 32, 4, 8, 128, 1100, True),
    (F32, 8, 1, 8, 64, 6000, False), (F32, 8, 1, 8, 64, 6400, True), (BF16, 8, 1, 8, 64, 8400, False), (BF16, 8, 1, 8, 64, 8800, True)])
def test_calls_that_attend_answers_sooner_go_to_it(dtype, n, group, heads, dim, tokens, shares):
    """By what the tables have room for: 70 MB, or 50 where fp32 queries are few."""
    b = Sized(tokens, heads=heads, dim=dim, page=16, n_pages=3 * n + 20, seqs=n, dtype=dtype)
    b.family([(100, [1] * n)])
    q, ids = b.rand(n, heads * group, dim).cuda(), b.ids(range(n))
    names = b.kernels(lambda: b.cache.attend_shared(0, ids, q))
    assert ("kv_plan_shared_kernel" in names) == shares
    want = b.cache.attend(0, ids, q)
    got = b.cache.attend_shared(0, ids, q)
    b.cache.check()
    assert torch.equal(got, want) or shares


def at64(b, i, out, q, group):
    """The result of sequence i's one query against 64 bits, with the bounds of Shared.check_shared."""
    c = b.cfg
    ref = attend64(b.seqs[i], 0, q.double().cpu().numpy(), group, c.head_dim ** -0.5, -1, 1, 0, c.page_tokens)
    tol, _ = bounds(*ref, c.head_dim, b.seqs[i].len, b.dtype)
    top = float(b.seqs[i].values(0, "v")[1].max()) * (127 if c.code == "int8" else 448)
    tol = tol + 2 * (2.0 ** -21 + 2.0 ** -22) * ref[2] + b.seqs[i].len * top * (2.0 ** -32 if b.dtype is BF16 else 2.0 ** -38)
    err = np.abs(out.double().cpu().numpy() - ref[0])
    assert (err <= tol).all(), (i, float((err / tol).max()), float(err.max()))


def shared_blocks(call):
    """The blocks of 16 tokens of each sequence that its group shares, with which the workspace begins."""
    return call.space[:8 * call.n].view(torch.int32).view(-1, 2).cpu().numpy()


@pytest.mark.parametrize("dtype,code", [(F32, "e4m3"), (BF16, "int8")])
@pytest.mark.parametrize("left,sinks", [(800, 0), (800, 40)])
def test_members_that_have_released_different_pages_share_the_others(dtype, code, left, sinks):
    """A sliding window with trim: longer members have released pages that shorter ones still hold, in front of what all see."""
    n, page = 70, 32
    rng = np.random.default_rng(7)
    own = rng.integers(1, 190, n)
    b = Shared(code, heads=8, dim=128, page=page, n_pages=1200, seqs=n, dtype=dtype, seed=9, least=20)
    prefixes = [901, 1000]
    st = b.family([(prefixes[0], own[:30].tolist()), (prefixes[1], own[30:].tolist())])
    b.trim(range(n), left, 1, sinks)
    table = b.cache.table.cpu().numpy()
    assert all(len({tuple(t) for t in table[x:y, :8] < 0}) > 1 for x, y in zip(st, st[1:]))
    call = Call(b, range(n), b.rand(n, 16, 128), st, left, 1, sinks)
    call.run()
    blocks = shared_blocks(call)
    for (x, y), prefix in zip(zip(st, st[1:]), prefixes):
        low = prefix + own[x:y].max() - 1 - left
        assert (blocks[x:y] == [-(-low // 16), prefix // page * page // 16]).all()
    b.check_shared(range(n), [1] * n, st, left=left, sinks=sinks, uniform=True, q=call.q.cpu())


def pieces_of_units(call):
    """Into how many pieces the kernel for many rows cuts each unit of a group's shared tokens: the workspace has 8 bytes and 4 for each
    sequence, 16 and 4 for each group and 4 more, then (first piece, pieces, first slot, 0) of each group."""
    up, g = lambda x: -(-x // 16) * 16, max(call.n_groups, 1)  # noqa: E731
    at = up(8 * call.n) + up(4 * call.n) + up(16 * g) + up(4 * (g + 1))
    return call.space[at:at + 16 * g].view(torch.int32).view(-1, 4)[:, 1].cpu().numpy()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("code,heads,dim,group,each", [("int8", 8, 64, 4, 9), ("e4m3", 7, 128, 16, 20), ("int8", 8, 32, 32, 10)])
def test_a_long_prefix_among_short_ones_is_cut(dtype, code, heads, dim, group, each):
    """More units than SMs, of groups of which one is far longer: no block gets all of its tokens."""
    groups, long = 24, 5
    n = groups * each
    rng = np.random.default_rng(groups)
    b = Shared(code, heads=heads, dim=dim, page=64, n_pages=700 + 3 * n, seqs=n, dtype=dtype, seed=dim)
    st = b.family([(12000 if g == long else int(rng.integers(64, 500)), rng.integers(1, 60, each).tolist()) for g in range(groups)])
    call = Call(b, range(n), b.rand(n, heads * group, dim), st)
    got = call.run()
    cuts = pieces_of_units(call)
    assert cuts[long] > 4 and (np.delete(cuts, long) == 1).all()
    b.cache.check()
    for x, y in ((st[long], st[long + 1]), (0, st[2])):
        for i in range(x, y, 7):
            at64(b, i, got[i:i + 1], call.q[i:i + 1], group)


@pytest.mark.parametrize("long", [3, 540])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_groups_than_a_launch_takes_with_a_long_one(dtype, long):
    """550 groups over two launches, one of them far longer than the others: in the first launch, or the last."""
    groups, group = 550, 20
    b = Shared("int8", heads=1, dim=32, page=16, n_pages=9000, seqs=2 * groups, dtype=dtype, seed=long)
    st = b.family([(30000 if g == long else 16 + g % 50, [1 + g % 3, 2]) for g in range(groups)])
    call = Call(b, range(2 * groups), b.rand(2 * groups, group, 32), st)
    got = call.run()
    b.cache.check()
    cuts = pieces_of_units(call)
    assert cuts[long] > 20 and (np.delete(cuts, long) == 1).all()
    for i in (0, 1, 2 * long - 1, 2 * long, 2 * long + 1, 2 * long + 2, 1023, 1024, 1025, 1099):
        at64(b, i, got[i:i + 1], call.q[i:i + 1], group)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompts_need_no_workspace_of_their_own_kind(dtype):
    """Calls that attend's kernel for prompts takes ask for attend's workspace, not for sums of all of their rows."""
    b = Shared("int8", heads=2, dim=64, page=32, n_pages=400, seqs=80, dtype=dtype)
    b.family([(300, [100] * 80)])
    lib, ref = b.native.lib(), b.cache._ref
    for rows, heads in ((8000, 4), (80000, 64)):
        need = lib.cac_kv8_attend_shared_workspace(ref, 80, rows, rows // 80, 0, heads, -1, 1, 0)
        assert need == lib.cac_kv8_attend_workspace(ref, 80, rows, rows // 80, heads, -1, 1, 0) > 0
    q = b.rand(8000, 4, 64).cuda()
    got = b.cache.attend_shared(0, b.ids(range(80)), q)
    assert torch.equal(got, b.cache.attend(0, b.ids(range(80)), q))
    b.cache.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,group,dim", [(30, 6, 64), (9, 1, 64), (12, 8, 128), (12, 4, 144)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_queries_of_both_types_and_kernels(dtype, n, group, dim, bad):
    """Their own row and head become NaN, and no other changes."""
    b = Shared("int8", heads=1, dim=dim, page=16, n_pages=60 + 2 * n, seqs=n, dtype=dtype)
    b.family([(600, [2] * n)])
    q, ids = b.rand(n, group, dim), b.ids(range(n))
    want, lse = b.cache.attend_shared(0, ids, q.cuda(), lse=True)
    x = q.clone()
    x[3, group - 1, 5] = bad
    got, s = b.cache.attend_shared(0, ids, x.cuda(), lse=True)
    b.cache.check()
    keep = torch.ones(n, group, dtype=torch.bool)
    keep[3, group - 1] = False
    assert torch.equal(got.cpu()[keep], want.cpu()[keep]) and torch.equal(s.cpu()[keep], lse.cpu()[keep])
    assert torch.isnan(got[3, group - 1]).all() and torch.isnan(s[3, group - 1])
    alone = b.cache.attend(0, ids, x.cuda())
    assert torch.equal(torch.isnan(alone), torch.isnan(got))
