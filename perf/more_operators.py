"""What is measured of a decoding step over the paged 8-bit K/V cache: products with
weights at 4 bits, the norm and rotation of queries and keys, and attention of
sequences that share a prefix.

A case's "op" is one of
  w4      rows times a weight matrix at 4 bits: W[n][k] = scale[n][k / group] *
          (code[n][k] - zero[n][k / group]), codes 0 .. 15 two to a byte (the even k
          in the low half), zero 8 where there is none, scales bf16
  rotate  queries and keys divided by their root mean square for each head and
          multiplied by a gain (where the case has a norm), then the first `rot`
          elements of each head turned in pairs by position * frequency
  shared  queries of the last tokens of each sequence over its cache, under the
          chunked-causal window with the first `sinks` tokens always visible; the
          sequences of a group have the pages of a prefix in common, as forks have

`own = False` computes all of it with elementary torch operations in 32 bits, the
rotation's angles in 64.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16  # tokens of the cache that share one scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _w4(name, m, n, k, per, zero, bias, dtype):
    return {"name": name, "op": "w4", "m": m, "n": n, "k": k, "per": per, "zero": zero, "bias": bias, "dtype": dtype}


def _rotate(name, n, new_lo, new_hi, pos_hi, kv_heads, group, head_dim, rot, layout, norm, scaling, by, dtype):
    return {"name": name, "op": "rotate", "n": n, "new_lo": new_lo, "new_hi": new_hi, "pos_hi": pos_hi,
            "kv_heads": kv_heads, "group": group, "head_dim": head_dim, "rot": rot, "layout": layout, "norm": norm,
            "scaling": scaling, "by": by, "dtype": dtype}


def _shared(name, groups, n, pre_lo, pre_hi, own_lo, own_hi, new_lo, new_hi, kv_heads, group, head_dim, left, chunk,
            sinks, page, code, dtype):
    return {"name": name, "op": "shared", "groups": groups, "n": n, "pre_lo": pre_lo, "pre_hi": pre_hi,
            "own_lo": own_lo, "own_hi": own_hi, "new_lo": new_lo, "new_hi": new_hi, "kv_heads": kv_heads,
            "group": group, "head_dim": head_dim, "left": left, "chunk": chunk, "sinks": sinks, "page": page,
            "code": code, "dtype": dtype}


def listed():
    return [
        # the 512 -> 2048 feed-forward product of one stream: nothing but latency
        _w4("w4_stream", 1, 2048, 512, 64, False, True, "f32"),
        # one token through a wide feed-forward layer: every byte of the weights for one row
        _w4("w4_token_wide", 1, 32768, 8192, 128, False, False, "bf16"),
        # a serving batch of 16, small groups with zero points
        _w4("w4_batch", 16, 16384, 4096, 32, True, False, "bf16"),
        # 37 rows into the 1,026 classes of the decoder, an odd depth, fp32
        _w4("w4_rows_odd", 37, 1026, 2080, 32, True, True, "f32"),
        # a 160 ms push of 256 streams, 2 frames each, 8 heads of 64
        _rotate("rotate_push", 256, 2, 2, 4000, 8, 1, 64, 64, "half", False, "none", "cache", "f32"),
        # whole prompts, norm and rotation, frequencies scaled for long contexts
        _rotate("rotate_prompt", 8, 500, 5000, 100, 8, 4, 128, 128, "half", True, "ramp", "cache", "bf16"),
        # ragged pieces at far positions, half of each head in neighbouring pairs
        _rotate("rotate_far_partial", 24, 1, 700, 1000000, 4, 4, 128, 64, "pairs", True, "linear", "positions", "f32"),
        # 8 hypotheses that share 30 s of context (375 frames of 80 ms)
        _shared("shared_beam", 1, 8, 375, 375, 1, 60, 1, 1, 8, 1, 64, -1, 1, 0, 16, "int8", "f32"),
        # four answers to one long prompt
        _shared("shared_long", 1, 4, 60000, 60000, 100, 2000, 1, 1, 8, 4, 128, -1, 1, 0, 64, "int8", "bf16"),
        # a serving batch behind one long instruction
        _shared("shared_batch", 1, 64, 32000, 32000, 1, 1000, 1, 1, 8, 4, 128, -1, 1, 0, 64, "int8", "bf16"),
        # several instructions of unlike lengths, a sliding window with four tokens that stay visible
        _shared("shared_groups", 6, 96, 500, 12000, 1, 700, 1, 1, 8, 8, 128, 8191, 1, 4, 32, "e4m3", "bf16"),
        # a few drafted tokens of each sequence checked at once, fp32 activations
        _shared("shared_drafts", 3, 24, 2000, 6000, 1, 300, 1, 8, 4, 4, 64, -1, 1, 0, 48, "e4m3", "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, dtype = rng.choice(["w4", "rotate", "shared", "shared"]), rng.choice(["f32", "bf16"])
    if op == "w4":
        per = rng.choice([32, 64, 128])
        k, n = per * _log(rng, 1, 8192 // per), _log(rng, 16, 32768)
        m = min(_log(rng, 1, 64), max(1, 16 * 16384 * 4096 // (n * k)))  # no more work than the listed ones
        c = _w4("", m, n, k, per, rng.random() < 0.5, rng.random() < 0.5, dtype)
    elif op == "rotate":
        head_dim = rng.choice([64, 64, 80, 128, 128, 256])
        rot = rng.choice([head_dim, head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)])
        n, new_hi = rng.choice([(_log(rng, 1, 256), rng.randint(1, 4)), (_log(rng, 1, 24), _log(rng, 20, 1000))])
        kv_heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 4, 7, 8])
        new_hi = max(1, min(new_hi, 80000000 // (n * kv_heads * (1 + group) * head_dim)))
        c = _rotate("", n, 1, new_hi, _log(rng, 100, 1000000), kv_heads, group, head_dim, rot, rng.choice(["half", "pairs"]), rng.random() < 0.6,
                    rng.choice(["none", "linear", "base", "ramp"]), rng.choice(["cache", "positions"]), dtype)
    else:
        left, chunk, sinks = rng.choice([(-1, 1, 0), (-1, 2, 0), (rng.randint(100, 8000), 1, rng.randint(0, 20))])
        groups = _log(rng, 1, 8)
        n, pre, own_hi, new_hi = _log(rng, groups, 64), _log(rng, 100, 20000), _log(rng, 10, 1000), rng.choice([1, 1, 2, 8])
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 4, 5, 8])
        n = max(groups, min(n, 60000000 // (kv_heads * group * new_hi * (pre + own_hi))))
        c = _shared("", groups, n, rng.choice([pre, pre // 4]), pre, 1, own_hi, 1, new_hi, kv_heads, group,
                    rng.choice([64, 64, 80, 128, 128]), left, chunk, sinks, rng.choice([16, 32, 48, 64]), rng.choice(["int8", "e4m3"]), dtype)
    del c["name"]
    return c


def _spread(n, lo, hi, step, shift):
    """n whole numbers of lo .. hi, spread evenly in no order."""
    return lo + np.floor((np.arange(n) * step + shift) % 1.0 * (hi - lo + 1)).astype(np.int64)


def _lengths(case):
    """Tokens before the call's own, and the call's, of each sequence."""
    n = case["n"]
    new = _spread(n, case["new_lo"], case["new_hi"], 0.7548776662466927, 0.61)
    if case["op"] == "rotate":
        return _spread(n, 0, case["pos_hi"], 0.6180339887498949, 0.37), new
    return _spread(n, case["own_lo"], case["own_hi"], 0.6180339887498949, 0.37), new


def _groups(case):
    """(first sequence of each group, and the end; tokens of each group's prefix)."""
    g, n = case["groups"], case["n"]
    size = 1 + _spread(g, 0, 3, 0.5698402909980532, 0.2)
    first = np.concatenate([[0], np.cumsum(size)]) * n // size.sum()
    return first, _spread(g, case["pre_lo"], case["pre_hi"], 0.6180339887498949, 0.83)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


SCALING = {  # of the rotation's frequencies: kind, base, factor, original length, low and high turns, amplitude
    "none": ("none", 10000.0, 1.0, 0, 1.0, 32.0, 1.0),
    "linear": ("linear", 10000.0, 4.0, 0, 1.0, 32.0, 1.0),
    "base": ("base", 10000.0, 8.0, 0, 1.0, 32.0, 1.0),
    "ramp": ("ramp", 500000.0, 16.0, 8192, 1.0, 32.0, 0.1 * math.log(16.0) + 1.0),
}
EPS = 1e-6


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _gain(gen, heads, dim):
    """Channels of unlike sizes, a few of them far larger, as projections give them."""
    g = torch.exp(0.4 * torch.randn(heads, dim, generator=gen, device="cuda"))
    return g * torch.where(torch.rand(heads, dim, generator=gen, device="cuda") < 0.02, 6.0, 1.0)


def _rows(gen, shape, gain, dt):
    return (torch.randn(shape, generator=gen, device="cuda") * gain).to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    {"w4": _prepare_w4, "rotate": _prepare_rotate, "shared": _prepare_shared}[case["op"]](case, gen, state)
    return state


def _prepare_w4(case, gen, S):
    M, N, K, per = case["m"], case["n"], case["k"], case["per"]
    S["packed"] = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
    S["scale"] = torch.empty(N, K // per, dtype=torch.bfloat16, device="cuda")
    S["zero"] = torch.empty(N, K // per, dtype=torch.uint8, device="cuda") if case["zero"] else None
    for r in range(0, N, 8192):
        e = min(N, r + 8192)
        w = torch.randn(e - r, K // per, per, generator=gen, device="cuda") * (K ** -0.5)
        if case["zero"]:
            lo, hi = w.amin(-1).clamp_max(0), w.amax(-1).clamp_min(0)
            s = ((hi - lo) / 15).to(torch.bfloat16)
            z = torch.round(-lo / s.float()).clamp(0, 15)
            S["zero"][r:e] = z.to(torch.uint8)
        else:
            s = (w.abs().amax(-1) / 7).to(torch.bfloat16)
            z = torch.full_like(s, 8, dtype=torch.float32)
        S["scale"][r:e] = s
        code = torch.round(w / s.float()[..., None] + z[..., None]).clamp(0, 15).to(torch.uint8).view(e - r, K)
        S["packed"][r:e] = code[:, 0::2] | (code[:, 1::2] << 4)
    S["bias"] = 0.1 * torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
    S["a"] = _rows(gen, (M, K), _gain(gen, 1, K), _dtype(case))


def _prepare_rotate(case, gen, S):
    H, G, D = case["kv_heads"], case["group"], case["head_dim"]
    old, new = _lengths(case)
    T = int(new.sum())
    dt = _dtype(case)
    S["q"] = _rows(gen, (T, H * G, D), _gain(gen, H * G, D), dt)
    S["k"] = _rows(gen, (T, H, D), _gain(gen, H, D), dt)
    S["gains"] = [1 + 0.2 * torch.randn(D, generator=gen, device="cuda") for _ in range(2)] if case["norm"] else [None] * 2
    pos = np.concatenate([np.arange(o, o + w) for o, w in zip(old, new)])
    S["positions"], S["ids"], S["starts"] = _i32(pos), _i32(np.arange(case["n"])), _i32(np.concatenate([[0], np.cumsum(new)]))
    S["lens"] = _i32(old + new)
    S["each"] = new.min() == new.max()
    S["max_new"] = int(new.max())
    if own:
        from cache_aware_conformer_gb300 import native
        from cache_aware_conformer_gb300.config import Kv8Config, RotaryConfig
        kind, base, factor, original, low, high, amplitude = SCALING[case["scaling"]]
        cfg = RotaryConfig(head_dim=D, rot_dim=case["rot"], layout=case["layout"], base=base, scaling=kind, factor=factor,
                           original=original, low=low, high=high, amplitude=amplitude, eps=EPS)
        S["rotary"] = native.Rotary(cfg, q_gain=S["gains"][0], k_gain=S["gains"][1])
        if case["by"] == "cache":  # the step's cache, whose sequences have grown by the call's tokens
            shape = Kv8Config(n_layers=1, kv_heads=H, head_dim=D, page_tokens=64, n_pages=1, max_seqs=case["n"],
                              max_pages=int((old + new).max()) // 64 + 1)
            held = {"table": torch.full((case["n"], shape.max_pages), -1, dtype=torch.int32, device="cuda"),
                    "lens": S["lens"], "refs": _i32([0]), "free": _i32([0]), "n_free": _i32([1])}
            S["cache"] = native.Kv8Cache(shape, tensors=held)


def _prepare_shared(case, gen, S):
    H, G, D, PT, n = (case[k] for k in ("kv_heads", "group", "head_dim", "page", "n"))
    first, prefix = _groups(case)
    mine, new = _lengths(case)
    of = np.searchsorted(first, np.arange(n), side="right") - 1  # each sequence's group
    common = prefix // PT                                       # pages that a group's tables name alike
    length = prefix[of] + mine + new
    pages = -(-length // PT)
    n_pages = int((common * (np.diff(first) > 0)).sum() + (pages - common[of]).sum())
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((n, int(pages.max())), -1, dtype=torch.int32, device="cuda")
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    at = 0
    for g in range(case["groups"]):
        if first[g + 1] > first[g]:
            names = perm[at:at + common[g]]
            at += int(common[g])
            table[first[g]:first[g + 1], :common[g]] = names
            refs[names.long()] = int(first[g + 1] - first[g])
    for s in range(n):
        more = int(pages[s] - common[of[s]])
        table[s, common[of[s]]:pages[s]] = perm[at:at + more]
        at += more
    S.update(table=table, refs=refs, lens=_i32(length), free=torch.full((n_pages,), -1, dtype=torch.int32, device="cuda"),
             n_free=_i32([0]), ids=_i32(np.arange(n)), groups=_i32(first), first=first, common=common * PT,
             starts=_i32(np.concatenate([[0], np.cumsum(new)])), start=np.concatenate([[0], np.cumsum(new)]), length=length,
             each=bool(new.min() == new.max()), max_new=int(new.max()))
    for name in ("k", "v"):
        gain = _gain(gen, H, D)
        S[name] = torch.empty(1, n_pages, H, PT, D, dtype=torch.int8, device="cuda")
        S[name + "_scale"] = torch.empty(1, n_pages, H, PT // BLOCK, dtype=torch.float32, device="cuda")
        for p in range(0, n_pages, 2048):
            e = min(n_pages, p + 2048)
            x = torch.randn(e - p, H, PT // BLOCK, BLOCK, D, generator=gen, device="cuda") * gain[:, None, None]
            top = 127.0 if case["code"] == "int8" else 448.0
            sc = (x.abs().amax((3, 4)) / top).clamp_min(2.0 ** -100)
            x = (x * (1 / sc)[..., None, None]).clamp_(-top, top)
            x = torch.round(x).to(torch.int8) if case["code"] == "int8" else x.to(torch.float8_e4m3fn).view(torch.int8)
            S[name][0, p:e] = x.view(e - p, H, PT, D)
            S[name + "_scale"][0, p:e] = sc
    S["q"] = _rows(gen, (int(new.sum()), H * G, D), _gain(gen, H * G, D), _dtype(case))
    if own:
        from cache_aware_conformer_gb300 import native
        from cache_aware_conformer_gb300.config import Kv8Config
        cfg = Kv8Config(n_layers=1, kv_heads=H, head_dim=D, page_tokens=PT, n_pages=n_pages, max_seqs=n,
                        max_pages=table.shape[1], code=case["code"])
        S["cache"] = native.Kv8Cache(cfg, tensors={k: S[k] for k in (
            "k", "v", "k_scale", "v_scale", "table", "lens", "refs", "free", "n_free")})


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return {"w4": _run_w4, "rotate": _run_rotate, "shared": _run_shared}[state["case"]["op"]](state)


def _ragged(S):
    return {} if S["each"] else {"starts": S["starts"], "max_new": S["max_new"]}


def _run_w4(S):
    if own:
        from cache_aware_conformer_gb300 import native
        return native.gemm_w4(S["a"], S["packed"], S["scale"], zero=S["zero"], bias=S["bias"])
    c = S["case"]
    code = torch.stack([S["packed"] & 15, S["packed"] >> 4], -1).view(c["n"], -1, c["per"]).float()
    zero = 8.0 if S["zero"] is None else S["zero"].float()[..., None]
    w = ((code - zero) * S["scale"].float()[..., None]).view(c["n"], c["k"])
    y = torch.matmul(S["a"].float(), w.t())
    if S["bias"] is not None:
        y = y + S["bias"]
    return y.to(S["a"].dtype)


def _run_rotate(S):
    c = S["case"]
    if own:
        if c["by"] == "cache":
            q, k = S["cache"].rotate(S["ids"], S["rotary"], S["q"], S["k"], **_ragged(S))
        else:
            q, k = S["rotary"].rotate(S["positions"], S["q"], S["k"])
        return {"q": q, "k": k}
    # positions of the last tokens of each sequence, from its length
    T, n = S["q"].shape[0], c["n"]
    if c["by"] == "cache":
        count = S["starts"].diff().long()
        seq = torch.repeat_interleave(torch.arange(n, device="cuda"), count, output_size=T)
        pos = (S["lens"].long() - S["starts"][1:].long())[seq] + torch.arange(T, device="cuda")
    else:
        pos = S["positions"].long()
    kind, base, factor, original, low, high, amplitude = SCALING[c["scaling"]]
    i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
    if kind == "base" and c["rot"] > 2:
        base = base * factor ** (c["rot"] / (c["rot"] - 2))
    freq = base ** (-2 * i / c["rot"])
    if kind == "linear":
        freq = freq / factor
    elif kind == "ramp":
        keep = ((original * freq / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
    angle = pos.double()[:, None] * freq
    cos, sin = (amplitude * torch.cos(angle)).float()[:, None], (amplitude * torch.sin(angle)).float()[:, None]
    out = {}
    for name, gain in zip("qk", S["gains"]):
        x = S[name].float()
        if gain is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
        y, R = x.clone(), c["rot"]
        a, b = (x[..., :R // 2], x[..., R // 2:R]) if c["layout"] == "half" else (x[..., 0:R:2], x[..., 1:R:2])
        ra, rb = a * cos - b * sin, a * sin + b * cos
        if c["layout"] == "half":
            y[..., :R // 2], y[..., R // 2:R] = ra, rb
        else:
            y[..., 0:R:2], y[..., 1:R:2] = ra, rb
        out[name] = y.to(S[name].dtype)
    return out


def _run_shared(S):
    c = S["case"]
    if own:
        out, lse = S["cache"].attend_shared(0, S["ids"], S["q"], groups=S["groups"], att_left=c["left"], att_chunk=c["chunk"],
                                            sinks=c["sinks"], lse=True, **_ragged(S))
        return {"out": out, "lse": lse}
    parts = [_attend_group(S, g) for g in range(c["groups"]) if S["first"][g + 1] > S["first"][g]]
    return {"out": torch.cat([p[0] for p in parts]), "lse": torch.cat([p[1] for p in parts])}


def _values(S, name, pages):
    """fp32 values of pages [.., m] -> [.., heads, m * page, head_dim]."""
    c = S["case"]
    x = S[name][0][pages]
    x = x.float() if c["code"] == "int8" else x.view(torch.float8_e4m3fn).float()
    lead, m = pages.shape[:-1], pages.shape[-1]
    H, PT, D = c["kv_heads"], c["page"], c["head_dim"]
    x = x.view(*lead, m, H, PT // BLOCK, BLOCK, D) * S[name + "_scale"][0][pages][..., None, None]
    return x.view(*lead, m, H, PT, D).transpose(-4, -3).reshape(*lead, H, m * PT, D)


def _attend_group(S, g):
    """The common tokens' scores for all queries of the group at once, those of each sequence's other tokens, and one softmax."""
    c = S["case"]
    H, G, D, PT = c["kv_heads"], c["group"], c["head_dim"], c["page"]
    lo, hi = int(S["first"][g]), int(S["first"][g + 1])
    P = int(S["common"][g])
    ids = S["ids"][lo:hi].long()
    n, Q = hi - lo, S["max_new"]
    count, lens = S["starts"].diff()[lo:hi].long(), S["lens"][ids].long()
    i = torch.arange(Q, device="cuda")
    row = (S["starts"][lo:hi, None].long() + i).clamp_max(S["q"].shape[0] - 1)
    q = S["q"][row].float().view(n, Q, H, G, D).permute(0, 2, 3, 1, 4)          # [n, H, G, Q, D]
    pages = S["table"][ids].long()
    m = int(-(-S["length"][lo:hi].max() // PT))
    own_pages = pages[:, P // PT:m].clamp_min(0)
    K, V = _values(S, "k", own_pages), _values(S, "v", own_pages)               # [n, H, t, D]
    score = torch.matmul(q.reshape(n, H, G * Q, D), K.transpose(-1, -2)).view(n, H, G, Q, -1)
    if P:
        Kp, Vp = _values(S, "k", pages[0, :P // PT]), _values(S, "v", pages[0, :P // PT])
        flat = q.permute(1, 0, 2, 3, 4).reshape(H, n * G * Q, D)
        common = torch.matmul(flat, Kp.transpose(-1, -2)).view(H, n, G, Q, P).transpose(0, 1)
        score = torch.cat([common, score], -1)
    score = score * (1.0 / math.sqrt(D))
    pos = lens[:, None] - count[:, None] + i
    begin = torch.div(pos, c["chunk"], rounding_mode="floor") * c["chunk"]
    j = torch.arange(score.shape[-1], device="cuda")
    seen = (j < begin[..., None] + c["chunk"]) & (j < lens[:, None, None])
    if c["left"] >= 0:
        seen &= (j >= begin[..., None] - c["left"]) | (j < c["sinks"])
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score.sub_(top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p[..., P:].reshape(n, H, G * Q, -1), V).view(n, H, G, Q, D)
    if P:
        o = o + torch.matmul(p[..., :P].transpose(0, 1).reshape(H, n * G * Q, P), Vp).view(H, n, G, Q, D).transpose(0, 1)
    o = o / total
    lse = (torch.log(total) + top)[..., 0]
    real = i < count[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(n, Q, H * G, D)[real].to(S["q"].dtype)
    return out, lse.permute(0, 3, 1, 2).reshape(n, Q, H * G)[real]


# ---------------------------------------------------------------------------
# the definitions in 64 bits, apart from the above
# ---------------------------------------------------------------------------
def exact(case, seed):
    S = prepare(case, seed)
    return {"w4": _exact_w4, "rotate": _exact_rotate, "shared": _exact_shared}[case["op"]](case, S)


def _exact_w4(c, S):
    a = S["a"].double()
    out = torch.empty(c["m"], c["n"], dtype=torch.float64, device="cuda")
    for r in range(0, c["n"], 4096):
        byte = S["packed"][r:r + 4096].long()
        w = torch.empty(byte.shape[0], c["k"], dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (byte % 16).double(), (byte // 16).double()
        spread = lambda x: x.double().repeat_interleave(c["per"], 1)  # noqa: E731
        w -= 8.0 if S["zero"] is None else spread(S["zero"][r:r + 4096])
        w *= spread(S["scale"][r:r + 4096])
        out[:, r:r + 4096] = a @ w.T
    return out if S["bias"] is None else out + S["bias"].double()


def _exact_rotate(c, S):
    """A pair as a complex number, turned by a unit one."""
    kind, base, factor, original, low, high, amplitude = SCALING[c["scaling"]]
    R = c["rot"]
    freq = []
    for i in range(R // 2):
        f = (base * factor ** (R / (R - 2)) if kind == "base" and R > 2 else base) ** (-2.0 * i / R)
        if kind == "linear":
            f /= factor
        if kind == "ramp":
            keep = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f *= keep + (1 - keep) / factor
        freq.append(f)
    angle = S["positions"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, amplitude), angle)[:, None]
    first = torch.arange(R // 2, device="cuda") * (1 if c["layout"] == "half" else 2)
    second = first + (R // 2 if c["layout"] == "half" else 1)
    out = {}
    for name, gain in zip("qk", S["gains"]):
        pieces = []
        for r in range(0, S[name].shape[0], 4096):
            x = S[name][r:r + 4096].double()
            if gain is not None:
                x = x * gain.double() / (x.square().sum(-1, keepdim=True) / c["head_dim"] + EPS).sqrt()
            z = torch.complex(x[..., first], x[..., second]) * turn[r:r + 4096]
            x[..., first], x[..., second] = z.real, z.imag
            pieces.append(x)
        out[name] = torch.cat(pieces)
    return out


def _exact_shared(c, S):
    """Each sequence by itself."""
    H, G, D, PT = c["kv_heads"], c["group"], c["head_dim"], c["page"]
    T = S["q"].shape[0]
    out = torch.zeros(T, H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, H * G, dtype=torch.float64, device="cuda")
    start = S["start"]
    for s in range(c["n"]):
        L = int(S["length"][s])
        t = torch.arange(L, device="cuda")
        page = S["table"][s, t // PT].long()
        K, V = ((S[x][0, page, :, t % PT] if c["code"] == "int8" else
                 S[x][0, page, :, t % PT].contiguous().view(torch.float8_e4m3fn)).to(torch.float64) *
                S[x + "_scale"][0, page, :, t % PT // BLOCK].double()[..., None] for x in ("k", "v"))
        m = int(start[s + 1] - start[s])
        begin = torch.arange(L - m, L, device="cuda") // c["chunk"] * c["chunk"]
        seen = t < (begin + c["chunk"])[:, None]
        if c["left"] >= 0:
            seen &= (t >= (begin - c["left"])[:, None]) | (t < c["sinks"])
        q = S["q"][start[s]:start[s + 1]].double().view(m, H, G, D)
        score = torch.einsum("mhgd,thd->hgmt", q, K) / math.sqrt(D)
        score = score.masked_fill(~seen, -math.inf)
        lse[start[s]:start[s + 1]] = torch.logsumexp(score, -1).permute(2, 0, 1).reshape(m, H * G)
        out[start[s]:start[s + 1]] = torch.einsum("hgmt,thd->mhgd", torch.softmax(score, -1), V).reshape(m, H * G, D)
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# bytes and operations of one pass
# ---------------------------------------------------------------------------
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "w4":
        M, N, K, per = case["m"], case["n"], case["k"], case["per"]
        b = N * K / 2 + N * K // per * (3 if case["zero"] else 2) + (M * K + M * N) * size + 4 * N * case["bias"]
        return {"bytes": float(b), "flops": 2.0 * M * N * K}
    H, G, D = case["kv_heads"], case["group"], case["head_dim"]
    mine, new = _lengths(case)
    T = int(new.sum())
    if case["op"] == "rotate":
        heads = T * (H + H * G)
        return {"bytes": float(2 * heads * D * size + 4 * case["n"]), "flops": float(heads * (3 * case["rot"] + 4 * D * case["norm"]))}
    first, prefix = _groups(case)
    of = np.searchsorted(first, np.arange(case["n"]), side="right") - 1
    common = prefix // case["page"] * case["page"]
    length, chunk = prefix[of] + mine + new, case["chunk"]
    held, pairs = np.zeros(case["groups"]), 0
    tokens = 0
    for s in range(case["n"]):
        begin = np.arange(length[s] - new[s], length[s]) // chunk * chunk
        end = np.minimum(begin + chunk, length[s])
        low = np.zeros_like(begin) if case["left"] < 0 else np.maximum(begin - case["left"], 0)
        sinks = np.minimum(low, case["sinks"])
        pairs += int((end - low + sinks).sum())
        c, l0 = int(common[of[s]]), int(low[0])
        seen = max(c - l0, 0) + min(int(sinks[0]), c)   # of the common tokens: read once for the group
        held[of[s]] = max(held[of[s]], seen)
        tokens += int(length[s]) - max(c, l0)
    tokens += int(held.sum())
    return {"bytes": float(tokens * H * 2 * (D + 4 / BLOCK) + T * H * G * (2 * D * size + 4)), "flops": 4.0 * D * H * G * pairs}
