"""Norm and rotation of queries and keys on the GPU against the formula in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from cache_aware_conformer_gb300.config import Kv8Config, RotaryConfig  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BOUNDS = -11


@pytest.fixture(scope="module")
def native():
    from cache_aware_conformer_gb300 import native as nat
    return nat


def exact(cfg, x, gain, pos):
    """(result, bound) in 64 bits of x [rows, heads, D] at positions pos.

    The norm: the sum of D squares is off by D 2^-24 of itself at most, half of which reaches its root; the root, the
    division and two products add 4 roundings of 2^-24.  The angle is off by 2^-33 of a turn and by 2^-25 of what is
    left of it after whole quarters (pi / 4 at most), sine and cosine by 2 units in the last place: 2^-22 in all.  Each
    turned value is two products and a sum of them, and the product with the amplitude."""
    D, R = cfg.head_dim, cfg.head_dim if cfg.rot_dim < 0 else cfg.rot_dim
    x = x.double()
    rel = 0.0
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + cfg.eps) * gain.double()
        rel = (D / 2 + 8) * 2.0 ** -24
    i = torch.arange(R // 2, dtype=torch.float64)
    base = cfg.base * cfg.factor ** (R / (R - 2)) if cfg.scaling == "base" else cfg.base
    f = base ** (-2 * i / max(R, 1))
    if cfg.scaling == "linear":
        f = f / cfg.factor
    if cfg.scaling == "ramp":
        keep = ((cfg.original * f / (2 * math.pi) - cfg.low) / (cfg.high - cfg.low)).clamp(0, 1)
        f = f * (keep + (1 - keep) / cfg.factor)
    angle = pos.double()[:, None, None] * f
    c, s = cfg.amplitude * torch.cos(angle), cfg.amplitude * torch.sin(angle)
    first = torch.arange(R // 2) * (1 if cfg.layout == "half" else 2)
    second = first + (R // 2 if cfg.layout == "half" else 1)
    a, b = x[..., first], x[..., second]
    out, tol = x.clone(), x.abs() * rel
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    # the reference's own angles: a double's rounding of a far position
    turned = abs(cfg.amplitude) * (a.abs() + b.abs()) * (rel + 2.0 ** -22 + 4 * 2.0 ** -24 + 2.0 ** -50 * pos.double().abs()[:, None, None])
    tol[..., first], tol[..., second] = turned, turned
    return out, tol


def close(got, want, tol, dtype):
    err = (got.double().cpu() - want).abs()
    tol = tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + 1e-37
    assert (err <= tol).all(), (float((err / tol).max()), (err > tol).nonzero()[:4].tolist())


def rows(g, T, H, D, dtype, gain=1.0):
    return (torch.randn(T, H, D, generator=g) * torch.exp(torch.randn(H, D, generator=g)) * gain).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,R", [(64, -1), (128, -1), (16, -1), (80, -1), (256, -1), (128, 64), (144, 48), (64, 2), (64, 0), (80, 34), (256, 250),
                                 (48, 14), (128, 126)])
def test_layouts_and_parts_of_heads(native, dtype, layout, norm, D, R):
    g = torch.Generator().manual_seed(D + R)
    cfg = RotaryConfig(head_dim=D, rot_dim=R, layout=layout, amplitude=1.0 if D != 80 else 1.25)
    gains = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)] if norm else [None, None]
    r = native.Rotary(cfg, *[None if x is None else x.cuda() for x in gains])
    for T, H, KH in ((1, 1, 1), (5, 6, 2), (70, 3, 3), (700, 5, 1)):
        q, k = rows(g, T, H, D, dtype), rows(g, T, KH, D, dtype)
        pos = torch.randint(0, 40000, (T,), generator=g, dtype=torch.int32)
        got = r.rotate(pos.cuda(), q.cuda(), k.cuda())
        for x, y, gain in zip((q, k), got, gains):
            close(y, *exact(cfg, x, gain, pos), dtype)


@pytest.mark.parametrize("kw", [{"scaling": "linear", "factor": 4.0}, {"scaling": "base", "factor": 8.0},
                                {"scaling": "ramp", "factor": 16.0, "original": 8192, "base": 500000.0, "amplitude": 1.277},
                                {"scaling": "ramp", "factor": 2.0, "original": 300, "low": 0.5, "high": 3.0}, {}])
def test_far_positions(native, kw):
    """At any position: the product with it is taken modulo a turn, in whole numbers."""
    g = torch.Generator().manual_seed(5)
    cfg = RotaryConfig(head_dim=128, **kw)
    r = native.Rotary(cfg)
    pos = torch.tensor([0, 1, -1, 2, 4095, 65537, 999983, 16777217, -123456789, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    q = rows(g, len(pos), 2, 128, F32)
    out, none = r.rotate(pos.cuda(), q.cuda())
    assert none is None
    close(out, *exact(cfg, q, None, pos), F32)


def test_one_side_only_and_norm_of_one(native):
    g = torch.Generator().manual_seed(9)
    cfg = RotaryConfig(head_dim=64, rot_dim=32)
    gain = 1 + torch.randn(64, generator=g)
    q, k, pos = rows(g, 9, 4, 64, BF16), rows(g, 9, 2, 64, BF16), torch.arange(9, dtype=torch.int32)
    r = native.Rotary(cfg, k_gain=gain.cuda())
    a, b = r.rotate(pos.cuda(), q.cuda(), k.cuda())
    close(a, *exact(cfg, q, None, pos), BF16)
    close(b, *exact(cfg, k, gain, pos), BF16)
    x, y = r.rotate(pos.cuda(), None, k.cuda())
    assert x is None and torch.equal(y, b)
    x, y = r.rotate(pos.cuda(), q.cuda(), None)
    assert y is None and torch.equal(x, a)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout,R", [("half", 64), ("half", 36), ("pairs", 64)])
def test_in_place_within_one_projection(native, dtype, layout, R):
    """Queries and keys turned where they lie in a wider row; what is beside them stays."""
    g = torch.Generator().manual_seed(11)
    T, D = 33, 64
    cfg = RotaryConfig(head_dim=D, rot_dim=R, layout=layout)
    gains = [1 + 0.1 * torch.randn(D, generator=g) for _ in range(2)]
    r = native.Rotary(cfg, *[x.cuda() for x in gains])
    qkv = rows(g, T, 10, D, dtype)
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    dev = qkv.cuda()
    q, k = dev[:, 1:5], dev[:, 6:8]
    a, b = r.rotate(pos.cuda(), q, k, out=(q, k))
    assert a.data_ptr() == q.data_ptr() and b.data_ptr() == k.data_ptr()
    close(q, *exact(cfg, qkv[:, 1:5], gains[0], pos), dtype)
    close(k, *exact(cfg, qkv[:, 6:8], gains[1], pos), dtype)
    for at in (slice(0, 1), slice(5, 6), slice(8, 10)):
        assert torch.equal(dev[:, at].cpu(), qkv[:, at])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norms_of_zero_tiny_huge_and_non_finite_heads(native, dtype):
    g = torch.Generator().manual_seed(13)
    D = 64
    cfg = RotaryConfig(head_dim=D)
    gain = 1 + 0.2 * torch.randn(D, generator=g)
    r = native.Rotary(cfg, gain.cuda(), gain.cuda())
    q = rows(g, 8, 2, D, F32)
    q[0, 0] = 0
    q[1] *= 1e-30
    q[2] *= 1e25
    q[3, 0] = q[3, 0] * 1e3 + 3e38 * torch.sign(q[3, 0])
    q[4, 1] *= 1e17
    q = q.clamp(-3.3e38, 3.3e38).to(dtype)
    pos = torch.arange(8, dtype=torch.int32) * 1000
    out, _ = r.rotate(pos.cuda(), q.cuda())
    close(out, *exact(cfg, q, gain, pos), dtype)
    bad = q.clone()
    bad[5, 0, 3], bad[6, 1, 60] = float("nan"), float("inf")
    got, _ = r.rotate(pos.cuda(), bad.cuda())
    keep = torch.ones(8, 2, dtype=torch.bool)
    keep[5, 0] = keep[6, 1] = False
    assert torch.equal(got.cpu()[keep], out.cpu()[keep])
    assert torch.isnan(got[5, 0]).all()
    plain = native.Rotary(cfg)
    got, _ = plain.rotate(pos.cuda(), bad.cuda())
    want, _ = plain.rotate(pos.cuda(), q.cuda())
    hit = torch.zeros(8, 2, D, dtype=torch.bool)
    hit[5, 0, [3, 35]] = hit[6, 1, [28, 60]] = True
    assert torch.equal(got.cpu()[~hit], want.cpu()[~hit]) and not torch.isfinite(got.cpu()[hit]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout,R", [("half", 64), ("half", 34), ("pairs", 64), ("pairs", 20), ("half", 0)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_norm_of_a_head_with_an_infinity(native, dtype, layout, R, bad):
    """x / infinity: 0 where x is finite, NaN for the infinity, which reaches the other element of its pair."""
    g = torch.Generator().manual_seed(14)
    D = 64
    r = native.Rotary(RotaryConfig(head_dim=D, rot_dim=R, layout=layout), (1 + 0.2 * torch.randn(D, generator=g)).cuda())
    q = rows(g, 6, 3, D, dtype)
    pos = torch.arange(6, dtype=torch.int32).cuda() * 77
    want, _ = r.rotate(pos, q.cuda())
    for e in (0, 3, 16, 17, 33, 63):
        x = q.clone()
        x[2, 1, e] = bad
        got, _ = r.rotate(pos, x.cuda())
        half = R // 2
        pair = {e} if e >= R else {e, e ^ 1} if layout == "pairs" else {e, e + half if e < half else e - half}
        hit = torch.zeros(D, dtype=torch.bool)
        hit[sorted(pair)] = True
        head = got[2, 1].float().cpu()
        assert torch.isnan(head[hit]).all() and (head[~hit] == 0).all(), e
        keep = torch.ones(6, 3, dtype=torch.bool)
        keep[2, 1] = False
        assert torch.equal(got.cpu()[keep], want.cpu()[keep])


def make_cache(native, lens, heads=2, dim=64, page=16):
    cfg = Kv8Config(1, heads, dim, page, 1, len(lens), max(max(lens) // page + 1, 1))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return native.Kv8Cache(cfg, tensors={"table": torch.full((len(lens), cfg.max_pages), -1, dtype=torch.int32, device="cuda"),
                                         "lens": i32(lens), "refs": i32([0]), "free": i32([0]), "n_free": i32([1])}), i32


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_positions_from_the_cache(native, dtype):
    g = torch.Generator().manual_seed(17)
    lens = [5, 900, 33, 70000, 4, 12, 1]
    cache, i32 = make_cache(native, lens)
    cfg = RotaryConfig(head_dim=64)
    r = native.Rotary(cfg)
    ids, counts = [3, 0, 6, 2, 5], [4, 5, 1, 0, 12]
    T = sum(counts)
    q, k = rows(g, T, 6, 64, dtype), rows(g, T, 2, 64, dtype)
    pos = torch.cat([torch.arange(lens[i] - m, lens[i]) for i, m in zip(ids, counts)])
    a, b = cache.rotate(i32(ids), r, q.cuda(), k.cuda(), starts=i32(np.concatenate([[0], np.cumsum(counts)]).tolist()))
    cache.check()
    close(a, *exact(cfg, q, None, pos), dtype)
    close(b, *exact(cfg, k, None, pos), dtype)
    q, k = rows(g, 6, 6, 64, dtype), rows(g, 6, 2, 64, dtype)
    pos = torch.cat([torch.arange(lens[i] - 2, lens[i]) for i in (1, 3, 1)])     # a sequence twice
    a, b = cache.rotate(i32([1, 3, 1]), r, q.cuda(), k.cuda())
    close(a, *exact(cfg, q, None, pos), dtype)
    close(b, *exact(cfg, k, None, pos), dtype)
    # the same as with the positions given
    c, d = r.rotate(pos.int().cuda(), q.cuda(), k.cuda())
    assert torch.equal(a, c) and torch.equal(b, d)


def test_rows_that_no_sequence_has_and_bad_ids_are_left(native):
    g = torch.Generator().manual_seed(19)
    cache, i32 = make_cache(native, [10, 20, 30])
    r = native.Rotary(RotaryConfig(head_dim=64))
    q, k = rows(g, 12, 2, 64, F32).cuda(), rows(g, 12, 2, 64, F32).cuda()
    full = lambda: (torch.full_like(q, 7.0), torch.full_like(k, 7.0))  # noqa: E731
    out = full()
    cache.rotate(i32([0, 2]), r, q, k, starts=i32([2, 4, 7]), out=out)
    cache.check()
    for x in out:
        assert (x[:2] == 7).all() and (x[7:] == 7).all() and (x[2:7] != 7).any()
    for ids, starts, alone in (([0, 3], [0, 4, 8], slice(4, 12)), ([0, -1], [0, 4, 8], slice(4, 12)), ([0, 1], [0, 4, 13], slice(4, 12)),
                               ([1, 0], [-2, 4, 8], slice(0, 4))):
        out = full()
        cache.rotate(i32(ids), r, q, k, starts=i32(starts), out=out)
        with pytest.raises(native.CacError) as e:
            cache.check()
        assert e.value.code == BOUNDS
        for x in out:
            assert (x[alone] == 7).all() and (x != 7).any()


def test_captured_steps_follow_the_lengths(native):
    g = torch.Generator().manual_seed(23)
    lens = [100, 7]
    cache, i32 = make_cache(native, [200, 200])
    cache.lens.copy_(i32(lens))
    cfg = RotaryConfig(head_dim=64)
    r = native.Rotary(cfg)
    q, k = rows(g, 2, 4, 64, F32), rows(g, 2, 2, 64, F32)
    dq, dk, ids = q.cuda(), k.cuda(), i32([1, 0])
    out = (torch.empty_like(dq), torch.empty_like(dk))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.rotate(ids, r, dq, dk, out=out)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        pos = torch.tensor([lens[1] + step - 1, lens[0] + step - 1])
        close(out[0], *exact(cfg, q, None, pos), F32)
        close(out[1], *exact(cfg, k, None, pos), F32)
        cache.lens += 1


def test_on_another_stream(native):
    g = torch.Generator().manual_seed(29)
    r = native.Rotary(RotaryConfig(head_dim=64))
    q, k, pos = rows(g, 50, 4, 64, BF16).cuda(), rows(g, 50, 2, 64, BF16).cuda(), torch.arange(50, dtype=torch.int32, device="cuda")
    want = r.rotate(pos, q, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    one = r.rotate(pos, q, k, stream=s)
    with torch.cuda.stream(s):
        two = r.rotate(pos, q, k)
    torch.cuda.synchronize()
    for got in (one, two):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refuses_bad_tensors(native):
    r = native.Rotary(RotaryConfig(head_dim=64))
    q, k, pos = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, 1, 64, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")
    cache, i32 = make_cache(native, [10, 20])
    for bad in (lambda: r.rotate(pos), lambda: r.rotate(pos, q.half()), lambda: r.rotate(pos, q, k.bfloat16()), lambda: r.rotate(pos, q, k[:3]),
                lambda: r.rotate(pos[:3], q), lambda: r.rotate(pos.long(), q), lambda: r.rotate(pos, q.cpu()),
                lambda: r.rotate(pos, q[..., :32]), lambda: r.rotate(pos, q.transpose(0, 1)), lambda: r.rotate(pos, q, out=(k, None)),
                lambda: r.rotate(pos, q, None, out=(None, k)), lambda: cache.rotate(i32([0, 1]), r, q, q[:, :1]),
                lambda: native.Rotary(RotaryConfig(head_dim=64), q_gain=torch.ones(32))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(native.CacError):
        cache.rotate(i32([0, 1, 0]), r, q)                       # rows that do not divide
    with pytest.raises(native.CacError):
        cache.rotate(i32([0, 1]), native.Rotary(RotaryConfig(head_dim=128)), torch.zeros(2, 1, 128, device="cuda"))
    assert r.rotate(pos[:0], q[:0], k[:0])[0].shape == (0, 2, 64)
