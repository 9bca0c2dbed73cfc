"""The paged 8-bit K/V cache in plain terms, for the parity tests: every sequence
holds its own codes and block scales, nothing is shared.  Codes and scales follow
the documented fp32 rule bit for bit; attention is computed in 64 bits."""
import math

import numpy as np
import torch

TOP = {"int8": 127.0, "e4m3": 448.0}
F = np.float32
MIN_SCALE = F(2.0 ** -100)


def encode(x, code):
    """Nearest code values (ties to even) of fp32 x."""
    x = np.clip(np.where(np.isnan(x), F(0), x), F(-TOP[code]), F(TOP[code]))
    if code == "int8":
        return np.rint(x).astype(F)
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float8_e4m3fn).float().numpy()


class Seq:
    def __init__(self, layers, heads, dim):
        self.code = {(l, w): np.zeros((0, heads, dim), F) for l in range(layers) for w in "kv"}
        self.scale = {(l, w): np.zeros((0, heads), F) for l in range(layers) for w in "kv"}
        self.len = 0
        self.gone = set()   # pages released by trim

    def copy(self):
        s = Seq.__new__(Seq)
        s.code = {k: v.copy() for k, v in self.code.items()}
        s.scale = {k: v.copy() for k, v in self.scale.items()}
        s.len, s.gone = self.len, set(self.gone)
        return s

    def append(self, layer, which, x, code):
        """x fp32 [t, H, D] after self.len tokens (the length is advanced by the caller)."""
        key, base, t = (layer, which), self.len, x.shape[0]
        x = x.astype(F)
        codes = np.concatenate([self.code[key][:base], np.zeros_like(x)])
        nb = -(-(base + t) // 16)
        scale = np.concatenate([self.scale[key][:-(-base // 16)], np.zeros((nb - -(-base // 16), x.shape[1]), F)])
        inv_top = F(1) / F(TOP[code])
        for b in range(base // 16, nb):
            lo, hi = max(base, 16 * b), min(base + t, 16 * b + 16)
            if hi <= lo:
                continue
            y = x[lo - base:hi - base]
            amax = np.where(np.isfinite(y), np.abs(y), F(0)).max((0, 2)).astype(F)
            need = np.maximum(amax * inv_top, MIN_SCALE)
            if lo > 16 * b:
                new = np.maximum(scale[b], need)
                grown = new != scale[b]
                again = encode(codes[16 * b:lo] * (scale[b] / new)[None, :, None], code)
                codes[16 * b:lo] = np.where(grown[None, :, None], again, codes[16 * b:lo])
            else:
                new = need
            with np.errstate(over="ignore", invalid="ignore"):
                codes[lo:hi] = encode(y * (F(1) / new)[None, :, None], code)
            scale[b] = new
        self.code[key], self.scale[key] = codes, scale

    def values(self, layer, which):
        key = (layer, which)
        t = np.arange(self.code[key].shape[0])
        return self.code[key], self.scale[key][t // 16]

    def cut(self, n, page):
        self.len = min(n, self.len)
        for key in self.code:
            self.code[key] = self.code[key][:self.len]
            self.scale[key] = self.scale[key][:-(-self.len // 16)]
        self.gone = {p for p in self.gone if p < -(-self.len // page)}

    def trim(self, left, chunk, sinks, page):
        if left < 0:
            return
        low = self.len // chunk * chunk - left
        self.gone |= {j for j in range(-(-self.len // page)) if (j + 1) * page <= low and j * page >= sinks}


def attend64(seq, layer, q, group, scale, left, chunk, sinks, page):
    """(out, lse, bound pieces) in 64 bits for q [m, heads, D], the last m tokens of seq.  The bound pieces are, per row
    and head: sum_j p_j |v_j| (per column) and scale * max_j sum_d |q_d k_jd|."""
    m, heads, D = q.shape
    q = q.astype(np.float64)
    kc, ks = seq.values(layer, "k")
    vc, vs = seq.values(layer, "v")
    K = kc.astype(np.float64) * ks.astype(np.float64)[..., None]
    V = vc.astype(np.float64) * vs.astype(np.float64)[..., None]
    out, lse = np.zeros((m, heads, D)), np.full((m, heads), -np.inf)
    mass, size = np.zeros((m, heads, D)), np.zeros((m, heads))
    at = np.arange(seq.len)
    there = ~np.isin(at // page, list(seq.gone))
    for r in range(m):
        p = seq.len - m + r
        if p < 0:
            continue
        b = p // chunk * chunk
        seen = there & (at < b + chunk)
        if left >= 0:
            seen &= (at >= b - left) | (at < sinks)
        if not seen.any():
            continue
        for h in range(heads):
            k, v = K[seen, h // group], V[seen, h // group]
            s = scale * (k @ q[r, h])
            top = s.max()
            e = np.exp(s - top)
            out[r, h] = (e / e.sum()) @ v
            lse[r, h] = top + math.log(e.sum())
            mass[r, h] = (e / e.sum()) @ np.abs(v)
            size[r, h] = abs(scale) * (np.abs(k) @ np.abs(q[r, h])).max()
    return out, lse, mass, size


def bounds(out, lse, mass, size, D, keys, dtype):
    """Largest error of the kernel's arithmetic.

    A score is a sum of D products in fp32, times fp32 factors: off by at most (D + 8) 2^-24 of sum |q k| (in units of the
    score, so a relative error of its weight).  The exponent's argument, a difference of numbers no larger than the
    score's bound + 128, adds 2^-23 of those, and the exponential 2^-21.  Weights enter the product with V rounded to
    11 bits for bf16 activations (2^-11), to 21 for fp32 (hi + lo); each is a relative error of a weight (of those over
    2^-21 of the largest; the others are off by 2^-32 of it at most, 2^-38 for fp32, far under what is allowed here).  Sums over the keys in fp32 add keys * 2^-24 at most.  Weight errors
    reach the output twice, in the sum and in its norm.  The output is rounded once."""
    w = (D + 8) * 2.0 ** -24 * size + 2.0 ** -23 * (size + 128) + 2.0 ** -21
    e = w + (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -20) + (keys + 16) * 2.0 ** -24
    half = torch.finfo(dtype).eps / 2
    finite = np.isfinite(lse)
    tol_out = 2 * e[..., None] * mass + half * np.abs(out) + 1e-30
    tol_lse = np.where(finite, w + keys * 2.0 ** -24 + 2.0 ** -22 * (np.abs(np.where(finite, lse, 0)) + 128), 0)
    return tol_out, tol_lse
