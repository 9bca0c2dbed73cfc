"""Products with weights at 4 bits on the GPU against the weights that the codes stand for, in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from cache_aware_conformer_gb300 import w4  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def native():
    from cache_aware_conformer_gb300 import native as nat
    return nat


def make(M, N, K, group, zeros, bias, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * M + N + K)
    gain = torch.exp(torch.randn(K, generator=g))
    a = (torch.randn(M, K, generator=g) * gain).to(dtype)
    code = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    scale = (torch.exp(torch.randn(N, K // group, generator=g)) * K ** -0.5).to(BF16)
    scale = torch.where(torch.rand(N, K // group, generator=g) < 0.1, -scale, scale)
    zero = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    b = torch.randn(N, generator=g) if bias else None
    return a, w4.pack(code), scale, zero, b


def exact(a, packed, scale, zero, bias):
    """(result, bound of the kernel's arithmetic) in 64 bits.

    Codes less zero points are exact.  Activations enter as fp16 after a power of two that brings the largest of 256 of a row
    to 2^14 or more: bf16 ones (8 bits) exactly and fp32 ones as two parts that hold 22 bits, but for those so small that
    fp16's last step, 2^-24, counts: off by half of it, 2^-39 of the largest.  Sums of a group's products (128 at most) on the
    tensor cores lose 2^-23 of the partial sum a step at most (they cut off), the groups' sums are scaled and added in fp32, at
    most K / 32 + 32 of them with the parts of a split, the bias once more."""
    w = w4.dequantize(packed, scale, zero)
    x = a.double()
    out, mass = x @ w.T, x.abs() @ w.abs().T
    tol = (2.0 ** -22 + (128 + a.size(1) / 32 + 32) * 2.0 ** -23) * mass
    tol = tol + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * w.abs().sum(1)
    if bias is not None:
        out = out + bias.double()
        tol = tol + 2.0 ** -24 * (out.abs() + bias.double().abs())
    return out, tol + torch.finfo(a.dtype).eps / 2 * out.abs() * (1 + 2.0 ** -7)


def check(native, a, packed, scale, zero, bias, **kw):
    put = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = native.gemm_w4(put(a) if not a.is_cuda else a, put(packed), put(scale), zero=put(zero), bias=put(bias), **kw)
    want, tol = exact(a.cpu(), packed, scale, zero, bias)
    err = (got.double().cpu() - want).abs()
    assert got.dtype == a.dtype and got.shape == want.shape
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()), (err > tol).nonzero()[:4].tolist())
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,k", [(1, 16, 1), (1, 1, 3), (3, 33, 5), (8, 100, 9), (9, 257, 2), (17, 48, 4), (37, 130, 7), (64, 64, 6),
                                   (65, 31, 3), (130, 17, 2)])
def test_small_and_odd_sizes(native, dtype, group, zeros, M, N, k):
    check(native, *make(M, N, k * group, group, zeros, M % 2 == 1, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N,K,group,zeros", [(1, 2048, 512, 64, False), (1, 4096, 8192, 128, False), (2, 5000, 4096, 32, True),
                                               (16, 1026, 4096, 64, True), (24, 2000, 8192, 32, False), (37, 1026, 2080, 32, True),
                                               (64, 640, 8192, 128, True), (1, 20000, 640, 128, True), (5, 48, 32768, 64, False),
                                               (40, 4100, 1024, 64, True)])
def test_larger_sizes(native, dtype, M, N, K, group, zeros):
    check(native, *make(M, N, K, group, zeros, False, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_rows_and_outputs(native, dtype):
    M, N, K = 7, 77, 256
    a, packed, scale, zero, bias = make(M, N, K, 64, True, True, dtype)
    wide = torch.full((M, K + 64), float("nan"), dtype=dtype, device="cuda")
    wide[:, 32:32 + K] = a.cuda()
    out = torch.full((M, N + 5), 3.0, dtype=dtype, device="cuda")
    got = check(native, wide[:, 32:32 + K], packed, scale, zero, bias, out=out[:, 3:3 + N])
    assert got.data_ptr() == out[:, 3:].data_ptr()
    assert (out[:, :3] == 3).all() and (out[:, 3 + N:] == 3).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values_of_any_size(native, dtype):
    """Rows of tiny, huge and zero values, and of both, keep their own precision."""
    M, N, K = 9, 40, 512
    a, packed, scale, zero, _ = make(M, N, K, 32, True, False, F32)
    a[0] *= 1e-30
    a[1] *= 1e30
    a[2] = 0
    a[3, ::2] *= 1e-20
    a[4] = a[4].abs() * 2.0 ** -100
    a[5, 7] = 1e32
    scale = scale.float().clamp(-1, 1).to(BF16)
    check(native, a.to(dtype), packed, scale, zero, None)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("M", [3, 20])
def test_non_finite_rows_stay_by_themselves(native, dtype, bad, M):
    a, packed, scale, zero, bias = make(M, 50, 256, 64, False, True, dtype)
    want = native.gemm_w4(a.cuda(), packed.cuda(), scale.cuda(), bias=bias.cuda())
    b = a.clone()
    b[1, 100] = bad
    got = native.gemm_w4(b.cuda(), packed.cuda(), scale.cuda(), bias=bias.cuda())
    keep = torch.arange(M) != 1
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])
    w = w4.dequantize(packed, scale)[:, 100]
    assert not torch.isfinite(got[1].cpu()[w != 0]).any()


def test_many_rows(native):
    check(native, *make(700, 96, 128, 32, True, True, BF16))


def test_the_same_result_each_time(native):
    a, packed, scale, zero, bias = (None if t is None else t.cuda() for t in make(6, 3000, 4096, 64, True, True, BF16))
    first = native.gemm_w4(a, packed, scale, zero, bias)
    for _ in range(5):
        assert torch.equal(native.gemm_w4(a, packed, scale, zero, bias), first)
    assert torch.equal(native.gemm_w4(a[:1], packed, scale, zero, bias), native.gemm_w4(a[:1].clone(), packed, scale, zero, bias))


def test_captured_and_replayed_with_new_rows(native):
    a, packed, scale, zero, bias = (None if t is None else t.cuda() for t in make(4, 700, 1024, 64, True, True, BF16))
    out = torch.empty(4, 700, dtype=BF16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        native.gemm_w4(a, packed, scale, zero, bias, out=out)
    a.copy_(torch.randn_like(a))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, native.gemm_w4(a, packed, scale, zero, bias))


def test_on_another_stream(native):
    a, packed, scale, zero, bias = (None if t is None else t.cuda() for t in make(4, 700, 1024, 64, True, True, F32))
    want = native.gemm_w4(a, packed, scale, zero, bias)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    one = native.gemm_w4(a, packed, scale, zero, bias, stream=s)
    with torch.cuda.stream(s):
        two = native.gemm_w4(a, packed, scale, zero, bias)
    torch.cuda.synchronize()
    assert torch.equal(one, want) and torch.equal(two, want)


def test_binding_refuses_bad_tensors(native):
    a, packed, scale, zero, bias = (t.cuda() for t in make(2, 8, 128, 64, True, True, F32))
    run = native.gemm_w4
    for bad in (lambda: run(a.half(), packed, scale), lambda: run(a[:, :64], packed, scale), lambda: run(a, packed.int(), scale),
                lambda: run(a, packed, scale.float()), lambda: run(a, packed, scale, zero=zero[:, :1]),
                lambda: run(a, packed, scale, bias=bias[:4]), lambda: run(a, packed, scale, bias=bias.double()),
                lambda: run(a, packed.cpu(), scale), lambda: run(a, packed, scale, out=torch.empty(2, 8, dtype=BF16, device="cuda")),
                lambda: run(a.t().contiguous().t(), packed, scale), lambda: run(a, packed, scale[:4])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(native.CacError):
        run(a, packed, scale[:, :1].contiguous().expand(8, 1).contiguous().repeat(1, 8))    # groups of 16
    assert run(a[:0], packed, scale).shape == (0, 8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,K", [(1, 131072), (3, 131072), (9, 65536), (31, 40960)])
def test_deep_rows(native, dtype, M, K):
    """Depths that a cluster of blocks shares, with fewer rows at a time where they do not fit."""
    check(native, *make(M, 40, K, 128, True, False, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group,K", [(32, 64), (32, 192), (64, 128), (64, 1152), (128, 768)])
def test_slices_of_larger_weights(native, dtype, group, K):
    """Rows 2 and on of weights: scales and zero points that begin anywhere on 4 bytes, and whose neighbours are not this call's."""
    N = 50
    a, packed, scale, zero, _ = make(5, N + 6, K, group, True, False, dtype)
    scale[:2], scale[N + 2:] = float("nan"), float("inf")
    put = [t.cuda() for t in (packed, scale, zero)]
    cut = [t[2:N + 2] for t in put]
    got = native.gemm_w4(a.cuda(), cut[0], cut[1], zero=cut[2])
    want, tol = exact(a, packed[2:N + 2], scale[2:N + 2], zero[2:N + 2], None)
    assert ((got.double().cpu() - want).abs() <= tol).all()


def test_two_streams_at_once(native):
    """Nothing is shared between calls: two graphs replayed side by side give what each gives alone."""
    cases = []
    for M, N, K, group, dtype in [(3, 3000, 4096, 64, F32), (16, 2048, 8192, 32, BF16)]:
        args = [None if t is None else t.cuda() for t in make(M, N, K, group, True, True, dtype)]
        want = native.gemm_w4(args[0], args[1], args[2], zero=args[3], bias=args[4])
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = [native.gemm_w4(args[0], args[1], args[2], zero=args[3], bias=args[4]) for _ in range(8)]
        cases.append((args, want, got, graph, stream))
    for _ in range(5):
        for *_, graph, stream in cases:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, want, got, *_ in cases:
        assert all(torch.equal(g, want) for g in got)


def spread(a, packed, scale, zero):
    """(result in 64 bits, root of the sum of squares of its products) of fp32 rows."""
    w = w4.dequantize(packed, scale, zero)
    x = a.double()
    return x @ w.T, torch.sqrt((x * x) @ (w * w).T)


def rms_bound(K):
    """Largest root mean square of a deep fp32 result's error, over the root of the sum of squares S of its products, whose signs are
    random.

    An element of A as two fp16 parts is off by 2^-22 of itself at most: 2^-22 S together, since signs are random.  A sum of 32
    products takes four tensor-core steps (two of each part) that cut off 2^-23 of the partial sum at most; the sums of 32 are of random
    signs too, and their squares add up to S^2: 2^-21 S.  K / 32 + 32 sums are added in fp32, each rounded by 2^-24 of the running
    sum at most, which grows with the root of its length: 2^-24 S sqrt(sum of j / n) = 2^-24 S sqrt(n / 2).  The scale's product and the last
    sums: 2^-22 S.  A mean over 40 or more results is within twice its expectation."""
    n = K / 32 + 32
    return 2 * (2.0 ** -22 + 2.0 ** -21 + 2.0 ** -24 * (n / 2) ** 0.5 + 2.0 ** -22)


def fp16_part(a):
    """What the first of the two fp16 parts holds of fp32 rows: 11 bits under the largest of 256."""
    x = a.view(a.size(0), -1, 256)
    up = torch.exp2(14 - torch.floor(torch.log2(x.abs().amax(-1, keepdim=True))))
    return ((x * up).half().float() / up).view_as(a)


@pytest.mark.parametrize("M,N,K,group", [(24, 500, 8192, 32), (5, 48, 32768, 64), (9, 40, 65536, 128), (31, 40, 40960, 128), (3, 40, 131072, 128),
                                         (1, 64, 131072, 128), (2, 600, 16384, 64)])
def test_deep_fp32_rows_keep_both_parts(native, M, N, K, group):
    """The bound of test_deep_rows, a worst case that grows with the depth, would not see the low parts left out; the mean error does."""
    a, packed, scale, zero, _ = make(M, N, K, group, True, False, F32)
    want, S = spread(a, packed, scale, zero)
    off = lambda y: float(((y.double() - want) / S).square().mean().sqrt())  # noqa: E731
    # the oracle without the low parts, and without one group: both are far outside
    w = w4.dequantize(packed, scale, zero)
    assert off(fp16_part(a).double() @ w.T) > 20 * rms_bound(K)
    assert off(a[:, group:].double() @ w[:, group:].T) > 20 * rms_bound(K)
    got = native.gemm_w4(a.cuda(), packed.cuda(), scale.cuda(), zero=zero.cuda())
    assert off(got.cpu()) <= rms_bound(K), (off(got.cpu()), rms_bound(K))
