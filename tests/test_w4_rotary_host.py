"""Weights at 4 bits and the rotation of queries and keys without a GPU: the packing,
the frequencies, and the refusals that are decided before anything is queued."""
import ctypes
import math
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from cache_aware_conformer_gb300 import w4  # noqa: E402
from cache_aware_conformer_gb300.config import RotaryConfig  # noqa: E402

INVAL, ALIGN, LIMIT = -1, -2, -10
OK = 0x10000


@pytest.fixture(scope="module")
def native():
    from cache_aware_conformer_gb300 import native as nat
    if not os.path.exists(nat.LIB_PATH):
        from cache_aware_conformer_gb300 import build
        build.build()
    return nat


def test_structs_match_the_header(native):
    assert ctypes.sizeof(native.CacW4) == 4 * 4 + 3 * 8 and native.CacW4.packed.offset == 16
    assert ctypes.sizeof(native.CacRotary) == 8 * 4 + 3 * 8 and native.CacRotary.steps.offset == 32
    assert native.CacRotary.amplitude.offset == 20 and native.CacRotary.eps.offset == 24


# ---------------------------------------------------------------------------
# packing
# ---------------------------------------------------------------------------
def test_pack_puts_the_even_code_low():
    code = torch.tensor([[1, 2, 15, 0], [0, 15, 7, 8]], dtype=torch.uint8)
    packed = w4.pack(code)
    assert packed.tolist() == [[0x21, 0x0F], [0xF0, 0x87]]
    assert torch.equal(w4.unpack(packed), code)


@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("zeros", [False, True])
def test_codes_are_the_nearest(group, zeros):
    """A weight is off by half a step at most, but where its code was cut off at the range's end: the scale is rounded to
    bf16, which moves the end by 2^-9 of the range, 7 or 15 steps, and the zero point is rounded by half a step."""
    g = torch.Generator().manual_seed(group)
    w = torch.randn(9, 3 * group, generator=g)
    w[2, :group] = 0
    w[3, :group] = w[3, :group].abs() + 1   # 0 at the range's end
    packed, scale, zero = w4.quantize(w, group, zeros)
    assert scale.dtype == torch.bfloat16 and scale.shape == (9, 3) and packed.shape == (9, 3 * group // 2)
    off = (w4.dequantize(packed, scale, zero) - w.double()).abs().view(9, 3, group)
    most = (0.5 + (0.5 + 15 * 2.0 ** -8 if zeros else 7 * 2.0 ** -8)) * scale.double()[..., None] + 1e-12
    assert (off <= most).all()
    assert (w4.dequantize(packed, scale, zero)[2, :group] == 0).all()


def test_bad_weights_are_refused():
    with pytest.raises(ValueError):
        w4.quantize(torch.zeros(2, 64), 48)
    with pytest.raises(ValueError):
        w4.quantize(torch.zeros(2, 96), 64)
    with pytest.raises(ValueError):
        w4.quantize(torch.full((2, 64), float("nan")), 64)


@pytest.mark.parametrize("kw,code", [
    ({"n": 0}, INVAL), ({"k": 0}, INVAL), ({"k": 96}, INVAL), ({"group": 16}, INVAL), ({"group": 0}, INVAL), ({"device": -1}, INVAL),
    ({"packed": None}, INVAL), ({"scale": None}, INVAL), ({"M": 0}, INVAL), ({"A": None}, INVAL), ({"C": None}, INVAL),
    ({"C": OK}, INVAL), ({"a_stride": 127}, INVAL), ({"c_stride": 9}, INVAL), ({"dtype": 2}, INVAL), ({"packed": OK + 8}, ALIGN),
    ({"scale": OK + 2}, ALIGN), ({"zero": OK + 1}, ALIGN), ({"A": OK + 8}, ALIGN), ({"a_stride": 132}, ALIGN), ({"C": 2 * OK + 1}, ALIGN),
    ({"bias": OK + 2}, ALIGN), ({"dtype": 0, "C": 2 * OK + 2}, ALIGN), ({"k": 131072 + 64, "a_stride": 200000}, LIMIT), ({"M": 65536}, LIMIT)])
def test_bad_products_are_refused(native, kw, code):
    a = {"n": 10, "k": 128, "group": 64, "device": 0, "packed": OK, "scale": OK, "zero": None, "M": 1, "A": OK, "a_stride": 128,
         "bias": None, "C": 2 * OK, "c_stride": 10, "dtype": 1, **kw}
    w = native.CacW4(a["n"], a["k"], a["group"], a["device"], a["packed"], a["scale"], a["zero"])
    assert native.lib().cac_op_gemm_w4(ctypes.addressof(w), a["M"], a["A"], a["a_stride"], a["bias"], a["C"], a["c_stride"],
                                       a["dtype"], None) == code
    assert native.lib().cac_op_gemm_w4(None, 1, OK, 128, None, 2 * OK, 10, 1, None) == INVAL


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def steps(native, rot, base=10000.0, scaling=0, factor=1.0, original=0.0, low=1.0, high=32.0):
    out = (ctypes.c_uint64 * max(rot // 2, 1))()
    r = native.lib().cac_op_rotary_steps(rot, base, scaling, factor, original, low, high, ctypes.addressof(out))
    return r, [int(x) for x in out][:rot // 2]


@pytest.mark.parametrize("rot,base,scaling,factor,original,low,high", [
    (64, 10000.0, 0, 1.0, 0, 1, 32), (128, 10000.0, 1, 4.0, 0, 1, 32), (80, 10000.0, 2, 8.0, 0, 1, 32),
    (128, 500000.0, 3, 16.0, 8192, 1, 32), (2, 10.0, 3, 2.0, 100, 0, 1), (2, 10.0, 1, 3.0, 0, 0, 1)])
def test_steps_are_the_frequencies(native, rot, base, scaling, factor, original, low, high):
    """To the double's own rounding: a few 2^-53 of the frequency."""
    r, got = steps(native, rot, base, scaling, factor, original, low, high)
    assert r == 0
    for i, s in enumerate(got):
        f = (base * factor ** (rot / (rot - 2)) if scaling == 2 else base) ** (-2 * i / rot)
        if scaling == 1:
            f /= factor
        if scaling == 3:
            keep = min(max((original * f / (2 * math.pi) - low) / (high - low), 0), 1)
            f = f * keep + f * (1 - keep) / factor
        assert abs(s / 2.0 ** 64 * 2 * math.pi - f) <= 64 * 2.0 ** -53 * f + 2.0 ** -60


def test_the_ramp_keeps_fast_pairs_and_divides_slow_ones(native):
    _, plain = steps(native, 128, 10000.0)
    _, ramp = steps(native, 128, 10000.0, 3, 8.0, 4096, 1.0, 32.0)
    assert ramp[0] == plain[0] and abs(ramp[-1] * 8 - plain[-1]) <= 8
    ratio = np.array(ramp, float) / np.array(plain, float)
    assert (np.diff(ratio) <= 1e-12).all()


@pytest.mark.parametrize("kw", [{"rot": 3}, {"rot": -2}, {"rot": 258}, {"base": 1.0}, {"base": float("nan")}, {"factor": 0.5},
                                {"scaling": 4}, {"scaling": -1}, {"rot": 2, "scaling": 2}, {"scaling": 3, "original": 0.0},
                                {"scaling": 3, "original": 10.0, "low": 2.0, "high": 2.0}])
def test_bad_frequencies_are_refused(native, kw):
    assert steps(native, **{"rot": 64, **kw})[0] == INVAL
    assert native.lib().cac_op_rotary_steps(64, 10.0, 0, 1.0, 0.0, 0.0, 1.0, None) == INVAL


def test_a_ramp_without_an_upper_end_divides_all(native):
    assert steps(native, 64, scaling=3, factor=4.0, original=1000.0, high=math.inf) == steps(native, 64, scaling=1, factor=4.0)


@pytest.mark.parametrize("low,high", [(-math.inf, 32.0), (-math.inf, math.inf), (math.nan, 32.0), (1.0, math.nan), (-1e308, 1e308)])
def test_a_ramp_between_turns_that_are_no_numbers_is_refused(native, low, high):
    """Its share of a frequency would be a NaN, and the step any number."""
    assert steps(native, 64, scaling=3, factor=4.0, original=1000.0, low=low, high=high)[0] == INVAL


def test_no_rotation_has_no_steps(native):
    assert steps(native, 0)[0] == 0


# ---------------------------------------------------------------------------
# the rotation's refusals
# ---------------------------------------------------------------------------
def rotary(native, **kw):
    a = {"head_dim": 64, "rot_dim": 32, "layout": 0, "dtype": 1, "device": 0, "amplitude": 1.0, "eps": 1e-6, "steps": OK,
         "q_gain": None, "k_gain": None, **kw}
    return native.CacRotary(a["head_dim"], a["rot_dim"], a["layout"], a["dtype"], a["device"], a["amplitude"], a["eps"], 0, a["steps"],
                            a["q_gain"], a["k_gain"])


def call(native, r, **kw):
    a = {"rows": 2, "positions": OK, "heads": 4, "q": OK, "q_stride": 256, "q_out": 2 * OK, "q_out_stride": 256, "kv_heads": 2,
         "k": 3 * OK, "k_stride": 128, "k_out": 4 * OK, "k_out_stride": 128, **kw}
    return native.lib().cac_op_rotate(r and ctypes.addressof(r), a["rows"], a["positions"], a["heads"], a["q"], a["q_stride"],
                                      a["q_out"], a["q_out_stride"], a["kv_heads"], a["k"], a["k_stride"], a["k_out"],
                                      a["k_out_stride"], None)


@pytest.mark.parametrize("kw,code", [
    ({"head_dim": 8}, INVAL), ({"head_dim": 72}, INVAL), ({"head_dim": 272}, INVAL), ({"rot_dim": 33}, INVAL), ({"rot_dim": 66}, INVAL),
    ({"rot_dim": -2}, INVAL), ({"layout": 2}, INVAL), ({"dtype": 2}, INVAL), ({"device": -1}, INVAL), ({"amplitude": float("inf")}, INVAL),
    ({"eps": 0.0}, INVAL), ({"eps": float("nan")}, INVAL), ({"steps": None}, INVAL), ({"steps": OK + 4}, ALIGN),
    ({"q_gain": OK + 8}, ALIGN), ({"k_gain": OK + 4}, ALIGN)])
def test_bad_rotations_are_refused(native, kw, code):
    r = rotary(native, **kw)
    assert call(native, r) == code
    c = native.CacKv8(2, 2, 64, 32, 100, 8, 20, 0, 0, 0)
    for name in ("k", "v", "k_scale", "v_scale", "table", "lens", "refs", "free_list", "n_free", "pending", "work", "status"):
        setattr(c, name, OK)
    assert native.lib().cac_kv8_rotate(ctypes.addressof(c), ctypes.addressof(r), 1, OK, None, 2, 4, OK, 256, 2 * OK, 256, 3 * OK, 128,
                                       4 * OK, 128, None) == code
    assert call(native, None) == INVAL


@pytest.mark.parametrize("kw,code", [
    ({"rows": -1}, INVAL), ({"heads": -1}, INVAL), ({"kv_heads": -1}, INVAL), ({"heads": 65536}, INVAL), ({"rows": 1 << 30}, LIMIT), ({"positions": None}, INVAL),
    ({"positions": OK + 2}, ALIGN), ({"q": None}, INVAL), ({"q_out": None}, INVAL), ({"k": None}, INVAL), ({"k_out": None}, INVAL),
    ({"q_stride": 255}, INVAL), ({"k_out_stride": 64}, INVAL), ({"q_out": OK, "q_out_stride": 512}, INVAL), ({"q": OK + 8}, ALIGN),
    ({"k_out": 4 * OK + 2}, ALIGN), ({"q_stride": 260}, ALIGN), ({"rows": 0}, 0), ({"heads": 0, "kv_heads": 0}, 0)])
def test_bad_rotate_calls_are_refused(native, kw, code):
    assert call(native, rotary(native), **kw) == code


@pytest.mark.parametrize("kw,code", [
    ({"n": -1}, INVAL), ({"ids": None}, INVAL), ({"rows": -1}, INVAL), ({"rows": 3, "n": 2}, INVAL), ({"heads": -1}, INVAL),
    ({"ids": OK + 2}, ALIGN), ({"starts": OK + 1}, ALIGN), ({"k": None}, INVAL), ({"k_out": None}, INVAL), ({"q": None}, INVAL),
    ({"n": 0}, 0), ({"rows": 0}, 0)])
def test_bad_rotate_calls_on_a_cache_are_refused(native, kw, code):
    a = {"n": 1, "ids": OK, "starts": None, "rows": 2, "heads": 4, "q": OK, "k": 3 * OK, "k_out": 4 * OK, **kw}
    c = native.CacKv8(2, 2, 64, 32, 100, 8, 20, 0, 0, 0)
    for name in ("k", "v", "k_scale", "v_scale", "table", "lens", "refs", "free_list", "n_free", "pending", "work", "status"):
        setattr(c, name, OK)
    r = rotary(native)
    run = lambda r: native.lib().cac_kv8_rotate(ctypes.addressof(c), ctypes.addressof(r), a["n"], a["ids"], a["starts"], a["rows"],  # noqa: E731
                                                a["heads"], a["q"], 256, 2 * OK, 256, a["k"], 128, a["k_out"], 128, None)
    assert run(r) == code
    if code == 0:
        assert run(rotary(native, head_dim=80)) == INVAL     # not the cache's
        assert run(rotary(native, device=1)) == INVAL
    c.n_pages = 0
    assert run(r) == INVAL


def test_binding_refuses_bad_rotations(native):
    for kw in ({"layout": "other"}, {"scaling": "other"}, {"rot_dim": 33}, {"rot_dim": 66}, {"head_dim": 24}, {"base": 0.5},
               {"scaling": "ramp"}):
        with pytest.raises(ValueError):
            native.Rotary(RotaryConfig(**{"head_dim": 64, **kw}), device="cuda:0")
    with pytest.raises(ValueError):
        native.Rotary(RotaryConfig(head_dim=64), device="cpu")


def test_binding_refuses_bad_products(native):
    a, p, s = torch.zeros(2, 64), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        native.gemm_w4(a, p, s)                # not on a GPU
