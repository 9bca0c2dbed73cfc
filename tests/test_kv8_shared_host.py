"""Attention behind a shared prefix without a GPU: refusals that are decided before
anything is queued, and the workspace."""
import ctypes
import os

import pytest

from test_kv8_host import make

INVAL, ALIGN = -1, -2
OK = 0x10000


@pytest.fixture(scope="module")
def native():
    from cache_aware_conformer_gb300 import native as nat
    if not os.path.exists(nat.LIB_PATH):
        from cache_aware_conformer_gb300 import build
        build.build()
    return nat


def call(native, c, **kw):
    a = {"layer": 0, "n": 1, "ids": OK, "starts": None, "rows": 1, "max_new": 1, "n_groups": 0, "groups": None, "heads": 8, "scale": 1.0,
         "left": -1, "chunk": 1, "sinks": 0, "q": OK, "q_stride": 512, "out": 2 * OK, "out_stride": 512, "lse": None, "dtype": 1, **kw}
    return native.lib().cac_kv8_attend_shared(
        ctypes.addressof(c), a["layer"], a["n"], a["ids"], a["starts"], a["rows"], a["max_new"], a["n_groups"], a["groups"], a["heads"],
        a["scale"], a["left"], a["chunk"], a["sinks"], a["q"], a["q_stride"], a["out"], a["out_stride"], a["lse"], a["dtype"], None, 0,
        None)


@pytest.mark.parametrize("kw,code", [
    ({"layer": 2}, INVAL), ({"heads": 6}, INVAL), ({"heads": 0}, INVAL), ({"rows": -2}, INVAL), ({"chunk": 0}, INVAL),
    ({"sinks": -1}, INVAL), ({"scale": float("nan")}, INVAL), ({"q": None}, INVAL), ({"out": None}, INVAL), ({"out": OK}, INVAL),
    ({"q_stride": 511}, INVAL), ({"out_stride": 100}, INVAL), ({"dtype": 5}, INVAL), ({"q": OK + 2}, ALIGN), ({"q_stride": 514}, ALIGN),
    ({"lse": 3 * OK + 1}, ALIGN), ({"n": 2, "rows": 3}, INVAL), ({"starts": OK, "max_new": -1}, INVAL), ({"n_groups": -1}, INVAL),
    ({"n_groups": 1}, INVAL), ({"groups": OK}, INVAL), ({"n_groups": 1, "groups": OK + 2}, ALIGN), ({"n": 0, "rows": 0}, 0),
    ({"n": 0, "rows": 0, "n_groups": 1}, INVAL)])
def test_bad_calls_are_refused(native, kw, code):
    assert call(native, make(native), **kw) == code


@pytest.mark.parametrize("field,value,code", [("head_dim", 72, -9), ("table", None, INVAL), ("k", OK + 8, ALIGN)])
def test_bad_caches_are_refused(native, field, value, code):
    assert call(native, make(native, **{field: value})) == code


def test_workspace_covers_that_of_attend(native):
    c = make(native, kv_heads=4, max_pages=4000, max_seqs=600)
    L, p = native.lib(), ctypes.addressof(c)
    for n, rows in ((1, 1), (3, 150), (40, 40), (300, 900)):
        for heads in (4, 32):
            for left in (-1, 70, 5000):
                need = L.cac_kv8_attend_shared_workspace(p, n, rows, rows, 0, heads, left, 1, 0)
                assert need >= rows * heads * (c.head_dim + 1) * 4
                assert need >= L.cac_kv8_attend_workspace(p, n, rows, rows, heads, left, 1, 0)
                assert L.cac_kv8_attend_shared_workspace(p, n, rows, rows, n, heads, left, 1, 0) >= need
    assert L.cac_kv8_attend_shared_workspace(p, 0, 1, 1, 0, 4, -1, 1, 0) == 0
    assert L.cac_kv8_attend_shared_workspace(p, 1, 1, 1, -1, 4, -1, 1, 0) == 0
    assert L.cac_kv8_attend_shared_workspace(None, 1, 1, 1, 0, 4, -1, 1, 0) == 0
