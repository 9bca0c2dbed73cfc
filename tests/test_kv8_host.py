"""The paged 8-bit K/V cache without a GPU: exported symbols and the refusals that
are decided before anything is queued."""
import ctypes
import os
import re
import subprocess
from dataclasses import replace

import pytest

from cache_aware_conformer_gb300.config import Kv8Config

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVAL, ALIGN, UNSUPPORTED, LIMIT = -1, -2, -9, -10


@pytest.fixture(scope="module")
def native():
    from cache_aware_conformer_gb300 import native as nat
    if not os.path.exists(nat.LIB_PATH):
        from cache_aware_conformer_gb300 import build
        build.build()
    return nat


def make(native, fake=0x10000, **kw):
    """A cache struct whose pointers are never followed."""
    c = native.CacKv8(2, 4, 64, 32, 100, 8, 20, 0, 0, 0)
    for name in ("k", "v", "k_scale", "v_scale", "table", "lens", "refs", "free_list", "n_free", "pending", "work", "status"):
        setattr(c, name, fake)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_header_and_library_agree(native):
    text = open(os.path.join(ROOT, "include", "cac_kv8.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(cac_kv8_\w+)\s*\(", text))
    assert declared == set(native.KV8_SYMBOLS)
    out = subprocess.run(["nm", "-D", "--defined-only", native.LIB_PATH], capture_output=True, text=True).stdout
    assert declared <= set(re.findall(r"\bT (cac_\w+)", out))


def test_struct_matches_the_header(native):
    """Ten 32-bit fields, then twelve pointers."""
    assert ctypes.sizeof(native.CacKv8) == 10 * 4 + 12 * 8
    assert native.CacKv8.k.offset == 40 and native.CacKv8.status.offset == 40 + 11 * 8


def test_work_size(native):
    c = make(native)
    assert native.lib().cac_kv8_work_ints(ctypes.addressof(c)) == 4 * 100 + 2 + 2 * 8 + 16


@pytest.mark.parametrize("field,value,code", [
    ("n_layers", 0, INVAL), ("kv_heads", 0, INVAL), ("kv_heads", 65536, INVAL), ("head_dim", 8, INVAL),
    ("head_dim", 72, UNSUPPORTED), ("head_dim", 272, UNSUPPORTED), ("page_tokens", 24, UNSUPPORTED),
    ("page_tokens", 2048, UNSUPPORTED), ("n_pages", 0, INVAL), ("max_seqs", 0, INVAL), ("max_pages", 0, INVAL),
    ("max_pages", 1 << 26, UNSUPPORTED), ("code", 2, UNSUPPORTED), ("table", None, INVAL), ("status", None, INVAL),
    ("k", 0x10008, ALIGN), ("lens", 0x10002, ALIGN)])
def test_bad_caches_are_refused(native, field, value, code):
    c = make(native, **{field: value})
    L, p = native.lib(), ctypes.addressof(c)
    if code != ALIGN and value is not None:
        assert L.cac_kv8_work_ints(p) == 0
    assert L.cac_kv8_init(p, None) == code
    assert L.cac_kv8_extend(p, 1, 0x10000, None, 1, None) == code
    assert L.cac_kv8_write(p, 0, 1, 0x10000, None, 1, 0x10000, 0x10000, 256, 256, 1, None) == code
    assert L.cac_kv8_read(p, 0, 1, 0x10000, 0x10000, 1, 0x10000, 0x10000, 1, None) == code
    assert L.cac_kv8_attend(p, 0, 1, 0x10000, None, 1, 1, 4, 1.0, -1, 1, 0, 0x10000, 256, 0x20000, 256, None, 1, None, 0,
                            None) == code
    assert L.cac_kv8_fork(p, 1, 0x10000, 0x10000, None) == code
    assert L.cac_kv8_truncate(p, 1, 0x10000, None, 0, None) == code
    assert L.cac_kv8_trim(p, 1, 0x10000, 1, 1, 0, None) == code
    assert L.cac_kv8_compact(p, None) == code
    assert L.cac_kv8_check(p) == code


def test_null_cache_is_refused(native):
    L = native.lib()
    assert L.cac_kv8_init(None, None) == INVAL and L.cac_kv8_work_ints(None) == 0
    assert L.cac_kv8_compact(None, None) == INVAL and L.cac_kv8_check(None) == INVAL


def test_bad_lists_are_refused(native):
    c = make(native)
    L, p, ok = native.lib(), ctypes.addressof(c), 0x10000
    assert L.cac_kv8_extend(p, -1, ok, None, 1, None) == INVAL
    assert L.cac_kv8_extend(p, 1, None, None, 1, None) == INVAL
    assert L.cac_kv8_extend(p, 1, ok, None, -1, None) == INVAL
    assert L.cac_kv8_extend(p, 9, ok, None, 1, None) == INVAL           # more than max_seqs
    assert L.cac_kv8_extend(p, 1, ok, None, 20 * 32 + 1, None) == LIMIT
    assert L.cac_kv8_extend(p, 1, ok + 2, None, 1, None) == ALIGN
    assert L.cac_kv8_fork(p, 1, ok, None, None) == INVAL
    assert L.cac_kv8_truncate(p, 1, ok, None, -1, None) == INVAL
    assert L.cac_kv8_trim(p, 1, ok, 5, 0, 0, None) == INVAL
    assert L.cac_kv8_trim(p, 1, ok, 5, 1, -1, None) == INVAL
    assert L.cac_kv8_read(p, 2, 1, ok, ok, 1, ok, ok, 1, None) == INVAL  # layer
    assert L.cac_kv8_read(p, 0, 1, ok, None, 1, ok, ok, 1, None) == INVAL
    assert L.cac_kv8_read(p, 0, 1, ok, ok, -1, ok, ok, 1, None) == INVAL
    assert L.cac_kv8_read(p, 0, 1, ok, ok, 1, ok, ok, 2, None) == INVAL
    assert L.cac_kv8_read(p, 0, 1, ok, ok, 1, ok + 4, ok, 1, None) == ALIGN
    # nothing to do
    assert L.cac_kv8_extend(p, 0, None, None, 1, None) == 0
    assert L.cac_kv8_read(p, 0, 1, ok, ok, 0, ok, ok, 1, None) == 0
    assert L.cac_kv8_trim(p, 1, ok, -1, 1, 0, None) == 0


@pytest.mark.parametrize("kw,code", [
    ({"layer": -1}, INVAL), ({"layer": 2}, INVAL), ({"rows": -1}, INVAL), ({"rows": 3, "n": 2}, INVAL), ({"k": None}, INVAL),
    ({"k_stride": 255}, INVAL), ({"v_stride": 8}, INVAL), ({"dtype": 7}, INVAL), ({"k": 0x10008}, ALIGN),
    ({"k_stride": 260}, ALIGN), ({"n": 9}, INVAL), ({"rows": 0}, 0)])
def test_bad_writes_are_refused(native, kw, code):
    c = make(native)
    a = {"layer": 0, "n": 1, "rows": 1, "k": 0x10000, "v": 0x10000, "k_stride": 256, "v_stride": 256, "dtype": 1, **kw}
    assert native.lib().cac_kv8_write(ctypes.addressof(c), a["layer"], a["n"], 0x10000, None, a["rows"], a["k"], a["v"],
                                      a["k_stride"], a["v_stride"], a["dtype"], None) == code


@pytest.mark.parametrize("kw,code", [
    ({"layer": 2}, INVAL), ({"heads": 6}, INVAL), ({"heads": 0}, INVAL), ({"rows": -2}, INVAL), ({"chunk": 0}, INVAL),
    ({"sinks": -1}, INVAL), ({"scale": float("nan")}, INVAL), ({"scale": float("inf")}, INVAL), ({"q": None}, INVAL),
    ({"out": None}, INVAL), ({"out": 0x10000}, INVAL), ({"q_stride": 511}, INVAL), ({"out_stride": 100}, INVAL),
    ({"dtype": 5}, INVAL), ({"q": 0x10002}, ALIGN), ({"q_stride": 514}, ALIGN), ({"lse": 0x30001}, ALIGN),
    ({"n": 2, "rows": 3}, INVAL), ({"starts": 0x10000, "max_new": -1}, INVAL), ({"n": 0, "rows": 0}, 0),
    ({"ids": 0x10001}, ALIGN)])
def test_bad_attention_calls_are_refused(native, kw, code):
    c = make(native)
    a = {"layer": 0, "n": 1, "ids": 0x10000, "starts": None, "rows": 1, "max_new": 1, "heads": 8, "scale": 1.0, "left": -1,
         "chunk": 1, "sinks": 0, "q": 0x10000, "q_stride": 512, "out": 0x20000, "out_stride": 512, "lse": None, "dtype": 1,
         **kw}
    assert native.lib().cac_kv8_attend(ctypes.addressof(c), a["layer"], a["n"], a["ids"], a["starts"], a["rows"],
                                       a["max_new"], a["heads"], a["scale"], a["left"], a["chunk"], a["sinks"], a["q"],
                                       a["q_stride"], a["out"], a["out_stride"], a["lse"], a["dtype"], None, 0,
                                       None) == code


@pytest.mark.parametrize("heads,left", [(4, 250), (4, 540), (4, 980), (1, 280)])
@pytest.mark.parametrize("n,rows", [(1, 64), (3, 150), (8, 8 * 64)])
def test_workspace_of_calls_without_starts(native, heads, left, n, rows):
    """Such a call has rows / n queries of each sequence; the size that is asked for must not go by a smaller max_new."""
    c = make(native, kv_heads=heads, max_pages=4000, max_seqs=600)
    ask = lambda m, left: native.lib().cac_kv8_attend_workspace(ctypes.addressof(c), n, rows, m, heads, left, 1, 0)  # noqa: E731
    for near in range(left - 40, left + 41):     # the border between whole units and shares lies in one of these
        want = ask(rows // n, near)
        assert ask(0, near) == want and ask(1, near) == want and ask(rows, near) >= want


def test_binding_refuses_a_bad_config(native):
    cfg = Kv8Config(1, 4, 64, 32, 10, 4, 4)
    with pytest.raises(ValueError):
        native.Kv8Cache(replace(cfg, code="int4"), device="cuda:0")
    with pytest.raises(ValueError):
        native.Kv8Cache(replace(cfg, head_dim=40), device="cuda:0")
    with pytest.raises(ValueError):
        native.Kv8Cache(cfg, device="cpu")
