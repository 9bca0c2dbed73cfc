"""What is measured of the paged 8-bit K/V cache: writing tokens into it, attention
over it, and its page operations.

The cache of a batch of sequences lies in pages of `page` tokens.  A page holds, for
each K/V head, `page` rows of `head_dim` codes of 8 bits (signed integers, or e4m3
floating point) for K and as many for V, and one fp32 scale for each block of 16
tokens and head: value = scale * code.  `table[s][j]` is the page that holds tokens
j * page .. (j + 1) * page - 1 of sequence s (-1: none), `lens[s]` its length, and
`refs[p]` counts the tables that name page p, since forked sequences share pages.

A case's "op" is one of
  attend  queries of the last tokens of each sequence over its cache, under the
          chunked-causal window of the encoder (left context and chunk, absolute
          positions) with the first `sinks` tokens always visible
  write   new tokens appended, then the last tokens read back as the values that
          the cache holds
  pages   the life of beam hypotheses: fork, append, drop, trim to the window,
          compact the pool, read back
  step    append and attend through several layers, as a model's step does

`own = False` computes all of it with elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16  # tokens that share one scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(name, op, n, kv_heads, group, head_dim, len_lo, len_hi, new_lo, new_hi, left, chunk, sinks, page, code,
          dtype, layers=1):
    return {"name": name, "op": op, "n": n, "kv_heads": kv_heads, "group": group, "head_dim": head_dim,
            "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo, "new_hi": new_hi, "left": left, "chunk": chunk,
            "sinks": sinks, "page": page, "code": code, "dtype": dtype, "layers": layers}


def listed():
    return [
        # one 160 ms push of 256 streams of the 8-head, 64-wide encoder: 2 frames, 70 frames of left context
        _case("attend_stream_push", "attend", 256, 8, 1, 64, 0, 4000, 2, 2, 70, 2, 0, 16, "int8", "f32"),
        # one long conversation, one token: everything hangs on splitting the one cache over the card
        _case("attend_token_one_long", "attend", 1, 8, 4, 128, 120000, 120000, 1, 1, -1, 1, 0, 64, "int8", "bf16"),
        # a serving batch of ragged lengths, one token each
        _case("attend_token_batch", "attend", 64, 8, 4, 128, 1000, 32000, 1, 1, -1, 1, 0, 64, "int8", "bf16"),
        # the same with a sliding window and four tokens that stay visible
        _case("attend_token_window", "attend", 128, 8, 8, 128, 1, 24000, 1, 1, 4095, 1, 4, 32, "e4m3", "bf16"),
        # two whole prompts: as many queries as keys, bound by arithmetic
        _case("attend_prompt", "attend", 2, 8, 4, 128, 0, 0, 5001, 8000, -1, 1, 0, 64, "int8", "bf16"),
        # ragged pieces of prompts beside single tokens, window and sinks, fp32 activations
        _case("attend_pieces", "attend", 24, 4, 4, 64, 0, 9000, 1, 700, 2047, 1, 16, 32, "e4m3", "f32"),
        # one token of each of 256 sequences: nothing but latency
        _case("write_token", "write", 256, 8, 1, 64, 1, 3000, 1, 1, -1, 1, 0, 16, "int8", "f32"),
        # prompts written at once
        _case("write_prompt", "write", 8, 8, 1, 128, 0, 100, 500, 9000, -1, 1, 0, 64, "e4m3", "bf16"),
        # 64 hypotheses of a beam forked and extended by a token, four layers
        _case("pages_beam", "pages", 64, 8, 1, 64, 100, 2000, 1, 3, 511, 1, 4, 16, "int8", "bf16", 4),
        # long sequences forked and extended by a piece, many pages to move
        _case("pages_long", "pages", 96, 8, 1, 128, 1000, 12000, 1, 900, 2047, 1, 16, 64, "int8", "bf16", 2),
        # a push of 256 streams through the 17 layers of the 8-head, 64-wide encoder
        _case("step_stream_push", "step", 256, 8, 1, 64, 0, 1000, 2, 2, 70, 2, 0, 16, "int8", "bf16", 17),
        # a serving step of 32 sequences through four layers
        _case("step_token", "step", 32, 8, 4, 128, 100, 8000, 1, 1, -1, 1, 0, 64, "int8", "bf16", 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "pages", "step"])
    kind = rng.choice(["push", "token", "piece"]) if op == "attend" else "token" if op == "step" else "any"
    kv_heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 4, 5, 7, 8])
    head_dim, page = rng.choice([64, 64, 80, 128, 128]), rng.choice([16, 32, 48, 64])
    left, chunk, sinks = rng.choice([(-1, 1, 0), (70, 2, 0), (rng.randint(100, 5000), 1, rng.randint(0, 20))])
    layers = 1
    if kind == "push":
        n, (new_lo, new_hi), len_hi = _log(rng, 1, 256), rng.choice([(2, 2), (4, 4), (1, 8)]), _log(rng, 50, 4000)
    elif kind == "token":
        n, (new_lo, new_hi), len_hi = _log(rng, 1, 64), (1, 1), _log(rng, 100, 20000)
        layers = rng.randint(1, 8) if op == "step" else 1
    elif kind == "piece":
        n, (new_lo, new_hi), len_hi = _log(rng, 1, 6), (1, _log(rng, 20, 600)), _log(rng, 100, 5000)
    else:
        n, (new_lo, new_hi), len_hi = _log(rng, 2, 96), (1, _log(rng, 1, 600)), _log(rng, 100, 4000)
        layers = rng.randint(1, 3) if op == "pages" else 1
    c = _case("", op, n, kv_heads, group, head_dim, 0 if op == "attend" else 1, len_hi, new_lo, new_hi, left, chunk,
              sinks, page, rng.choice(["int8", "e4m3"]), rng.choice(["f32", "bf16"]), layers)
    del c["name"]
    return c


def _lengths(case):
    """Tokens in the cache before the call, and new ones, of each sequence: spread evenly over the case's ranges."""
    i = np.arange(case["n"])
    a, b = (i * 0.6180339887498949 + 0.37) % 1.0, (i * 0.7548776662466927 + 0.61) % 1.0
    old = case["len_lo"] + np.floor(a * (case["len_hi"] - case["len_lo"] + 1)).astype(np.int64)
    new = case["new_lo"] + np.floor(b * (case["new_hi"] - case["new_lo"] + 1)).astype(np.int64)
    return old, new


def _read_back(case):
    """Tokens read back of each sequence's end: a write's own tokens, some of a hypothesis."""
    return max(16, int(_lengths(case)[1].max())) if case["op"] == "write" else 16


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _keys(gen, shape, gain):
    """Values as projections give them: Gaussian, with channels of unlike sizes."""
    return torch.randn(shape, generator=gen, device="cuda") * gain


def _gain(gen, heads, dim):
    g = torch.exp(0.4 * torch.randn(heads, dim, generator=gen, device="cuda"))
    return g * torch.where(torch.rand(heads, dim, generator=gen, device="cuda") < 0.02, 6.0, 1.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, n, H, D, PT, L = (case[k] for k in ("op", "n", "kv_heads", "head_dim", "page", "layers"))
    old, new = _lengths(case)
    held = old + new if op == "attend" else old  # tokens in the cache when the pass begins
    # each sequence's pages lie anywhere in the pool; forks and appended tokens find free ones
    pages = -(-held // PT)
    grown = -(-(old + new) // PT)
    seqs = 2 * n if op == "pages" else n
    extra = int((new // PT + 2).sum())
    n_pages = int(pages.sum()) + (0 if op == "attend" else extra)
    max_pages = int(grown.max())
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((seqs, max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s in range(n):
        table[s, :pages[s]] = perm[at:at + pages[s]]
        at += int(pages[s])
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[perm[:at].long()] = 1
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    lens[:n] = torch.from_numpy(held.astype(np.int32)).cuda()
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_pages - at] = perm[at:]
    state = {"case": case, "table": table, "refs": refs, "lens": lens, "free": free,
             "n_free": torch.tensor([n_pages - at], dtype=torch.int32, device="cuda")}
    gk, gv, gq = _gain(gen, H, D), _gain(gen, H, D), _gain(gen, H * case["group"], D)
    for name, gain in (("k", gk), ("v", gv)):
        codes = torch.empty(L, n_pages, H, PT, D, dtype=torch.int8, device="cuda")
        scale = torch.empty(L, n_pages, H, PT // BLOCK, dtype=torch.float32, device="cuda")
        for layer in range(L):
            for p in range(0, n_pages, 4096):
                e = min(n_pages, p + 4096)
                x = _keys(gen, (e - p, H, PT // BLOCK, BLOCK, D), gain[:, None, None])
                sc = (x.abs().amax((3, 4)) / _top(case)).clamp_min(2.0 ** -100)
                codes[layer, p:e] = _encode(x * (1 / sc)[..., None, None], case).reshape(e - p, H, PT, D)
                scale[layer, p:e] = sc
                del x, sc
        state[name], state[name + "_scale"] = codes, scale
    T = int(new.sum())
    dt = _dtype(case)
    if op in ("write", "pages", "step"):
        state["k_new"] = [_keys(gen, (T, H, D), gk).to(dt) for _ in range(L)]
        state["v_new"] = [_keys(gen, (T, H, D), gv).to(dt) for _ in range(L)]
    if op in ("attend", "step"):
        state["q"] = [_keys(gen, (T, H * case["group"], D), gq).to(dt) for _ in range(L)]
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    state["ids"], state["starts"] = i32(np.arange(n)), i32(np.concatenate([[0], np.cumsum(new)]))
    state["each"] = int(new[0]) if new.min() == new.max() else 0  # every sequence has as many new tokens
    state["max_new"] = int(new.max())
    state["base"], state["count"] = i32(old), _read_back(case)
    state["first"] = i32(old + new - _read_back(case))
    if op == "pages":
        state["src"] = torch.randint(0, n, (n,), generator=gen, device="cuda").to(torch.int32)
        state["dst"] = state["ids"] + n
        srclen = state["base"][state["src"].long()]
        grown = -(-(srclen + state["starts"].diff()) // PT)  # tables have to hold a long source and a long addition
        wide = int(grown.max())
        if wide > max_pages:
            state["table"] = torch.cat([table, torch.full((seqs, wide - max_pages), -1, dtype=torch.int32, device="cuda")], 1)
        state["odd"] = state["dst"][1::2].contiguous()
        state["odd_len"] = (srclen[1::2] - srclen[1::2] // 3).contiguous()
        state["read_ids"] = torch.cat([state["ids"], state["dst"]])
        after = srclen + state["starts"].diff()
        after[1::2] = state["odd_len"]
        state["read_first"] = torch.cat([state["base"], after]) - _read_back(case)
    if own:
        from cache_aware_conformer_gb300 import native
        from cache_aware_conformer_gb300.config import Kv8Config
        cfg = Kv8Config(n_layers=L, kv_heads=H, head_dim=D, page_tokens=PT, n_pages=n_pages, max_seqs=seqs,
                        max_pages=state["table"].shape[1], code=case["code"])
        state["cache"] = native.Kv8Cache(cfg, tensors={k: state[k] for k in (
            "k", "v", "k_scale", "v_scale", "table", "lens", "refs", "free", "n_free")})
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return {"attend": _run_attend, "write": _run_write, "pages": _run_pages, "step": _run_step}[case["op"]](state)


def _ragged(S):
    return {} if S["each"] else {"starts": S["starts"], "max_new": S["max_new"]}


def _run_attend(S):
    c = S["case"]
    window = {"att_left": c["left"], "att_chunk": c["chunk"], "sinks": c["sinks"]}
    if own:
        out, lse = S["cache"].attend(0, S["ids"], S["q"][0], lse=True, **window, **_ragged(S))
    else:
        out, lse = _attend(S, 0, S["ids"], S["q"][0], S["starts"], **window)
    return {"out": out, "lse": lse}


def _run_write(S):
    if own:
        cache = S["cache"]
        cache.truncate(S["ids"], S["base"])
        cache.extend(S["ids"], each=S["each"], **_ragged(S))
        cache.write(0, S["ids"], S["k_new"][0], S["v_new"][0], **_ragged(S))
        k, v = cache.read(0, S["ids"], S["first"], S["count"], dtype=_dtype(S["case"]))
        return {"k": k, "v": v, "lens": cache.lens}
    _truncate(S, S["ids"], S["base"])
    _extend(S, S["ids"], S["starts"])
    _write(S, 0, S["ids"], S["k_new"][0], S["v_new"][0], S["starts"])
    k, v = _read(S, 0, S["ids"], S["first"], S["count"])
    return {"k": k, "v": v, "lens": S["lens"]}


def _run_pages(S):
    c = S["case"]
    L = c["layers"]
    window = {"att_left": c["left"], "att_chunk": c["chunk"], "sinks": c["sinks"]}
    if own:
        cache = S["cache"]
        cache.fork(S["src"], S["dst"])
        cache.extend(S["dst"], each=S["each"], **_ragged(S))
        for layer in range(L):
            cache.write(layer, S["dst"], S["k_new"][layer], S["v_new"][layer], **_ragged(S))
        cache.truncate(S["odd"], S["odd_len"])
        cache.trim(S["dst"], **window)
        cache.compact()
        k, v = cache.read(L - 1, S["read_ids"], S["read_first"], S["count"], dtype=_dtype(c))
        return {"k": k, "v": v, "lens": cache.lens, "n_free": cache.n_free}
    _fork(S, S["src"], S["dst"])
    _extend(S, S["dst"], S["starts"])
    for layer in range(L):
        _write(S, layer, S["dst"], S["k_new"][layer], S["v_new"][layer], S["starts"])
    _truncate(S, S["odd"], S["odd_len"])
    _trim(S, S["dst"], **window)
    _compact(S)
    k, v = _read(S, L - 1, S["read_ids"], S["read_first"], S["count"])
    return {"k": k, "v": v, "lens": S["lens"], "n_free": (S["refs"] == 0).sum(dtype=torch.int32).reshape(1)}


def _run_step(S):
    c = S["case"]
    window = {"att_left": c["left"], "att_chunk": c["chunk"], "sinks": c["sinks"]}
    outs = []
    if own:
        cache = S["cache"]
        cache.truncate(S["ids"], S["base"])
        cache.extend(S["ids"], each=S["each"], **_ragged(S))
    else:
        _truncate(S, S["ids"], S["base"])
        _extend(S, S["ids"], S["starts"])
    for layer in range(c["layers"]):
        q, k, v = S["q"][layer], S["k_new"][layer], S["v_new"][layer]
        if own:
            cache.write(layer, S["ids"], k, v, **_ragged(S))
            outs.append(cache.attend(layer, S["ids"], q, **window, **_ragged(S)))
        else:
            _write(S, layer, S["ids"], k, v, S["starts"])
            outs.append(_attend(S, layer, S["ids"], q, S["starts"], **window)[0])
    return outs


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _top(case):
    """The largest code."""
    return 127.0 if case["code"] == "int8" else 448.0


def _encode(x, case):
    """Nearest codes (ties to even) of values within the largest code."""
    if case["code"] == "int8":
        return torch.round(x).clamp_(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.int8)


def _decode(codes, case):
    return codes.float() if case["code"] == "int8" else codes.view(torch.float8_e4m3fn).float()


def _tokens(S, name, layer, pages):
    """fp32 values of whole pages [n, m] -> [n, heads, m * page, head_dim]."""
    c = S["case"]
    x = _decode(S[name][layer][pages], c)                      # [n, m, H, PT, D]
    n, m, H, PT, D = x.shape
    x = x.view(n, m, H, PT // BLOCK, BLOCK, D) * S[name + "_scale"][layer][pages][..., None, None]
    return x.view(n, m, H, PT, D).transpose(1, 2).reshape(n, H, m * PT, D)


def _attend(S, layer, ids, q, starts, att_left, att_chunk, sinks):
    c = S["case"]
    PT, H, G, D = c["page"], c["kv_heads"], c["group"], c["head_dim"]
    ids, count = ids.long(), starts.diff().long()
    n, T, Q = len(ids), q.shape[0], S["max_new"]
    lens = S["lens"][ids].long()
    m = S["table"].shape[1]
    pages = S["table"][ids].long()
    there = (pages >= 0).repeat_interleave(PT, 1)
    K, V = (_tokens(S, x, layer, pages.clamp_min(0)) for x in ("k", "v"))
    # queries [n, H, G * Q, D], one row of padding where a sequence has fewer
    i = torch.arange(Q, device=q.device)
    row = (starts[:-1, None].long() + i).clamp_max(T - 1)
    qs = q[row].float().view(n, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(n, H, G * Q, D)
    score = torch.matmul(qs, K.transpose(2, 3)) * (1.0 / math.sqrt(D))
    # query i sits at position len - count + i and sees its chunk, the left context before the chunk, and the sinks
    pos = lens[:, None] - count[:, None] + i
    begin = torch.div(pos, att_chunk, rounding_mode="floor") * att_chunk
    j = torch.arange(m * PT, device=q.device)
    seen = (j < begin[..., None] + att_chunk) & (j < lens[:, None, None]) & there[:, None]
    if att_left >= 0:
        seen &= (j >= begin[..., None] - att_left) | (j < sinks)
    seen &= (pos >= 0)[..., None]
    score = score.view(n, H, G, Q, m * PT).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score.sub_(top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, H, G * Q, m * PT), V).view(n, H, G, Q, D) / torch.where(total == 0, 1.0, total)
    lse = torch.log(total) + top
    real = i < count[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(n, Q, H * G, D)[real].to(q.dtype)
    return out, lse[..., 0].permute(0, 3, 1, 2).reshape(n, Q, H * G)[real]


def _take(S, total):
    """`total` free pages."""
    return (S["refs"] == 0).nonzero()[:total, 0]


def _truncate(S, ids, new_len):
    PT, ids, new_len = S["case"]["page"], ids.long(), new_len.long()
    new_len = torch.minimum(new_len, S["lens"][ids].long())
    rows = S["table"][ids]
    drop = torch.arange(rows.shape[1], device=ids.device) >= (-(-new_len // PT))[:, None]
    _drop(S, ids, rows, drop)
    S["lens"][ids] = new_len.int()


def _drop(S, ids, rows, drop):
    gone = rows[drop & (rows >= 0)].long()
    S["refs"].index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    S["table"][ids] = rows.masked_fill(drop, -1)


def _trim(S, ids, att_left, att_chunk, sinks):
    """Releases the pages that no later query sees: before the window of the next position, and past the sinks."""
    if att_left < 0:
        return
    PT, ids = S["case"]["page"], ids.long()
    lens = S["lens"][ids].long()
    low = torch.div(lens, att_chunk, rounding_mode="floor") * att_chunk - att_left
    j = torch.arange(S["table"].shape[1], device=ids.device)
    drop = ((j + 1) * PT <= low[:, None]) & (j * PT >= sinks)
    _drop(S, ids, S["table"][ids], drop)


def _fork(S, src, dst):
    src, dst = src.long(), dst.long()
    rows = S["table"][dst]
    _drop(S, dst, rows, torch.ones_like(rows, dtype=torch.bool))
    rows = S["table"][src]
    named = rows[rows >= 0].long()
    S["refs"].index_add_(0, named, torch.ones_like(named, dtype=torch.int32))
    S["table"][dst] = rows
    S["lens"][dst] = S["lens"][src]


def _extend(S, ids, starts):
    """Room for the new tokens: fresh pages, and a copy of a last page that others read too and that is not full."""
    PT, ids, count = S["case"]["page"], ids.long(), starts.diff().long()
    n = len(ids)
    lens = S["lens"][ids].long()
    have, want = -(-lens // PT), -(-(lens + count) // PT)
    last = S["table"][ids, (lens // PT).clamp_max(S["table"].shape[1] - 1)].long()
    part = (lens % PT != 0) & (count > 0) & (last >= 0)
    who = torch.arange(n, device=ids.device)
    named = torch.zeros_like(S["refs"], dtype=torch.long).index_add_(0, last[part], torch.ones_like(last[part]))
    keeper = torch.full_like(named, -1).scatter_reduce_(0, last[part], who[part], "amax")
    safe = last.clamp_min(0)
    copy = part & ((S["refs"][safe] > named[safe]) | (keeper[safe] != who))
    fresh = want - have
    take = _take(S, int((fresh.sum() + copy.sum()).item()))
    n_copy = int(copy.sum().item())
    to, new = take[:n_copy], take[n_copy:]
    for x in ("k", "v", "k_scale", "v_scale"):
        S[x][:, to] = S[x][:, last[copy]]
    S["refs"].index_add_(0, last[copy], torch.full_like(to, -1, dtype=torch.int32))
    S["table"][ids[copy], (lens // PT)[copy]] = to.int()
    S["refs"][take] = 1
    s = torch.repeat_interleave(who, fresh)
    k = torch.arange(len(s), device=ids.device) - (fresh.cumsum(0) - fresh)[s]
    S["table"][ids[s], have[s] + k] = new.int()
    S["lens"][ids] = (lens + count).int()


def _write(S, layer, ids, k, v, starts):
    """Quantises the last tokens of each sequence, block by block.  A block that already holds older tokens keeps its
    scale unless the new ones need a larger one; then the old codes are rounded again to that scale."""
    c = S["case"]
    PT, ids, count = c["page"], ids.long(), starts.diff().long()
    base = S["lens"][ids].long() - count
    lo, hi = base // BLOCK, -(-(base + count) // BLOCK)
    blocks = torch.where(count > 0, hi - lo, 0)
    s = torch.repeat_interleave(torch.arange(len(ids), device=ids.device), blocks)
    b = lo[s] + torch.arange(len(s), device=ids.device) - (blocks.cumsum(0) - blocks)[s]
    page = S["table"][ids[s], b * BLOCK // PT].long()
    sub = b % (PT // BLOCK)
    pos = b[:, None] * BLOCK + torch.arange(BLOCK, device=ids.device)
    new = (pos >= base[s][:, None]) & (pos < (base + count)[s][:, None])
    older = pos < base[s][:, None]
    row = (starts[:-1].long()[s][:, None] + pos - base[s][:, None]).clamp(0, k.shape[0] - 1)
    for name, src in (("k", k), ("v", v)):
        codes = S[name][layer].view(-1, c["kv_heads"], PT // BLOCK, BLOCK, c["head_dim"])
        x = src[row].float().transpose(1, 2)                       # [blocks, H, 16, D]
        x = torch.where(new[:, None, :, None], x, 0.0)
        need = (x.abs().amax((2, 3)) / _top(c)).clamp_min(2.0 ** -100)
        before = S[name + "_scale"][layer][page, :, sub]
        scale = torch.where(older.any(1)[:, None], torch.maximum(before, need), need)
        held = codes[page, :, sub]
        again = _encode(_decode(held, c) * (before / scale)[..., None, None], c)
        again = torch.where((scale != before)[..., None, None], again, held)
        fresh = _encode(x * (1 / scale)[..., None, None], c)
        kept = torch.where(new[:, None, :, None], fresh, torch.where(older[:, None, :, None], again, held))
        codes[page, :, sub] = kept
        S[name + "_scale"][layer][page, :, sub] = scale


def _compact(S):
    """Moves the used pages that lie past the number of used ones into the free places before it."""
    used = S["refs"] > 0
    n = used.sum()
    at = torch.arange(len(used), device=used.device)
    to, of = (~used & (at < n)).nonzero()[:, 0], (used & (at >= n)).nonzero()[:, 0]
    for x in ("k", "v", "k_scale", "v_scale"):
        S[x][:, to] = S[x][:, of]
    S["refs"][to], S["refs"][of] = S["refs"][of], torch.zeros_like(S["refs"][of])
    name = at.int().index_copy(0, of, to.int())
    S["table"].copy_(torch.where(S["table"] >= 0, name[S["table"].clamp_min(0).long()], S["table"]))


def _read(S, layer, ids, first, count):
    """Values of tokens first .. first + count - 1 of each sequence; zeros where it has none."""
    c = S["case"]
    PT, ids = c["page"], ids.long()
    pos = first.long()[:, None] + torch.arange(count, device=ids.device)
    j = pos.clamp(0, S["table"].shape[1] * PT - 1)
    page = S["table"].gather(0, ids[:, None].expand(-1, S["table"].shape[1])).gather(1, j // PT).long()
    real = (pos >= 0) & (pos < S["lens"][ids][:, None]) & (page >= 0)
    page, got = page.clamp_min(0), []
    for name in ("k", "v"):
        x = _decode(S[name][layer][page, :, j % PT], c) * S[name + "_scale"][layer][page, :, j % PT // BLOCK][..., None]
        got.append(torch.where(real[..., None, None], x, 0.0).to(_dtype(c)))
    return got


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
class _Sequence:
    """K and V of one sequence and layer as 64-bit codes and scales, token by token."""

    def __init__(self, S, s, layer, length):
        c = S["case"]
        t = np.arange(length)
        page = S["table"][s].cpu().numpy()[t // c["page"]].astype(np.int64)
        t = torch.from_numpy(t % c["page"]).cuda()
        page = torch.from_numpy(page).cuda()
        self.code, self.scale = {}, {}
        for x in ("k", "v"):
            raw = S[x][layer][page, :, t]
            raw = raw if c["code"] == "int8" else raw.view(torch.float8_e4m3fn).float()
            self.code[x] = raw.double()
            self.scale[x] = S[x + "_scale"][layer][page, :, t // BLOCK].double()  # one for each token, alike in a block
        self.case, self.length = c, length

    def nearest(self, x):
        x = x.clamp(-_top(self.case), _top(self.case))
        if self.case["code"] == "int8":
            return torch.round(x)
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
        return torch.round(x / step) * step

    def append(self, new):
        """Tokens [t, H, D] of K and V, by the rule of the blocks' scales."""
        base, t = self.length, new["k"].shape[0]
        for x in ("k", "v"):
            v = new[x].double()
            code = torch.cat([self.code[x], torch.zeros_like(v)])
            scale = torch.cat([self.scale[x], torch.zeros_like(v[..., 0])])
            for b in range(base // BLOCK, -(-(base + t) // BLOCK)):
                lo, hi = max(base, b * BLOCK), min(base + t, (b + 1) * BLOCK)
                y = v[lo - base:hi - base]
                top = (y.abs().amax((0, 2)) / _top(self.case)).clamp_min(2.0 ** -100)
                if lo > b * BLOCK:
                    was = scale[b * BLOCK]
                    top = torch.maximum(top, was)
                    grown = (top > was)[:, None]
                    held = code[b * BLOCK:lo]
                    code[b * BLOCK:lo] = torch.where(grown, self.nearest(held * (was / top)[:, None]), held)
                code[lo:hi] = self.nearest(y / top[:, None])
                scale[b * BLOCK:hi] = top
            self.code[x], self.scale[x] = code, scale
        self.length = base + t

    def cut(self, length):
        for x in ("k", "v"):
            self.code[x], self.scale[x] = self.code[x][:length], self.scale[x][:length]
        self.length = length

    def value(self, x):
        return self.code[x] * self.scale[x][..., None]

    def last(self, x, first, count):
        out = torch.zeros(count, *self.code[x].shape[1:], dtype=torch.float64, device="cuda")
        lo, hi = max(first, 0), min(first + count, self.length)
        if hi > lo:
            out[lo - first:hi - first] = self.value(x)[lo:hi]
        return out

    def attend(self, q):
        c = self.case
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        K, V = self.value("k"), self.value("v")
        at = torch.arange(self.length, device="cuda")
        for lo in range(0, q.shape[0], 1024):
            pos = torch.arange(self.length - q.shape[0], self.length, device="cuda")[lo:lo + 1024]
            begin = pos // c["chunk"] * c["chunk"]
            seen = at < (begin + c["chunk"])[:, None]
            if c["left"] >= 0:
                seen &= (at >= (begin - c["left"])[:, None]) | (at < c["sinks"])
            for h in range(q.shape[1]):
                s = q[lo:lo + 1024, h].double() @ K[:, h // c["group"]].T / math.sqrt(c["head_dim"])
                s = s.masked_fill(~seen, -math.inf)
                lse[lo:lo + 1024, h] = torch.logsumexp(s, 1)
                out[lo:lo + 1024, h] = torch.softmax(s, 1) @ V[:, h // c["group"]]
        return out, lse


def exact(case, seed):
    op, L = case["op"], case["layers"]
    old, new = _lengths(case)
    pairs = int(((old + new) * new).sum()) * case["kv_heads"] * case["group"] * L * (op in ("attend", "step"))
    blocks = int((new // BLOCK + 2).sum()) * L * (op in ("write", "step")) + int((new // BLOCK + 2).sum()) * (op == "pages")
    if pairs * case["head_dim"] * 4 > 4e12 or blocks > 12000 or case["n"] * L * (op == "step") > 5000:
        return None
    S = prepare(case, seed)
    start = S["starts"].tolist()
    piece = lambda x, s: {y: S[y + "_new"][x][start[s]:start[s + 1]] for y in ("k", "v")}  # noqa: E731
    if op == "attend":
        got = [_Sequence(S, s, 0, int(old[s] + new[s])).attend(S["q"][0][start[s]:start[s + 1]]) for s in range(case["n"])]
        return {"out": torch.cat([g[0] for g in got]), "lse": torch.cat([g[1] for g in got])}
    if op == "step":
        outs = []
        for layer in range(L):
            got = []
            for s in range(case["n"]):
                one = _Sequence(S, s, layer, int(old[s]))
                one.append(piece(layer, s))
                got.append(one.attend(S["q"][layer][start[s]:start[s + 1]])[0])
            outs.append(torch.cat(got))
        return outs
    got = {"k": [], "v": [], "lens": None}
    if op == "write":
        for s in range(case["n"]):
            one = _Sequence(S, s, 0, int(old[s]))
            one.append(piece(0, s))
            for x in ("k", "v"):
                got[x].append(one.last(x, int(old[s] + new[s]) - S["count"], S["count"]))
    else:
        got["n_free"] = None
        src, first = S["src"].tolist(), S["read_first"].tolist()
        cut = dict(zip(range(1, case["n"], 2), S["odd_len"].tolist()))
        for s in range(2 * case["n"]):
            fork = s >= case["n"]
            one = _Sequence(S, src[s - case["n"]] if fork else s, L - 1, int(old[src[s - case["n"]] if fork else s]))
            if fork:
                one.append(piece(L - 1, s - case["n"]))
                if s - case["n"] in cut:
                    one.cut(cut[s - case["n"]])
            for x in ("k", "v"):
                y = one.last(x, first[s], S["count"])
                if fork and case["left"] >= 0:  # pages that the trim released read as zeros
                    low = one.length // case["chunk"] * case["chunk"] - case["left"]
                    t = np.arange(first[s], first[s] + S["count"]) // case["page"]
                    gone = ((t + 1) * case["page"] <= low) & (t * case["page"] >= case["sinks"])
                    y[torch.from_numpy(gone).cuda()] = 0
                got[x].append(y)
    return {x: torch.stack(y) if y else None for x, y in got.items()}


# ---------------------------------------------------------------------------
# bytes and operations of one pass
# ---------------------------------------------------------------------------
def _seen(case, old, new):
    """(tokens that any query of the sequence sees, pairs of query and token)."""
    length, chunk = old + new, case["chunk"]
    pos = np.arange(old, length)
    begin = pos // chunk * chunk
    hi = np.minimum(begin + chunk, length)
    if case["left"] < 0:
        return int(length), int(hi.sum())
    lo = np.maximum(begin - case["left"], 0)
    first = np.minimum(lo, case["sinks"])
    return int(min(lo[0], case["sinks"]) + length - lo[0]), int((hi - lo + first).sum())


def work(case):
    op, H, G, D, L, PT = (case[k] for k in ("op", "kv_heads", "group", "head_dim", "layers", "page"))
    old, new = _lengths(case)
    size, T = (2 if case["dtype"] == "bf16" else 4), int(new.sum())
    token = H * 2 * (D + 4 / BLOCK)  # bytes of one token's codes and scales, K and V
    b = f = 0.0
    if op in ("attend", "step"):
        seen = [_seen(case, o, w) for o, w in zip(old, new)]
        b += L * (sum(s for s, _ in seen) * token + T * H * G * (2 * D * size + (4 if op == "attend" else 0)))
        f += L * 4.0 * D * H * G * sum(p for _, p in seen)
    if op in ("write", "pages", "step"):
        b += L * T * (H * 2 * D * size + token)
        f += L * T * H * 2 * D * 4.0
    if op in ("write", "pages"):
        back = np.minimum(old + new, _read_back(case)).sum() if op == "write" else 2 * case["n"] * _read_back(case)
        b += back * (token + H * 2 * D * size)
    if op == "pages":
        # tables copied; a last page copied for each fork whose source does not end with a page; the truncated forks'
        # pages filled again by others
        b += 8.0 * (-(-old // PT)).sum() + L * PT * token * 2 * (case["n"] + (new[1::2] // PT).sum())
    return {"bytes": float(b), "flops": float(f)}
