"""The 4-bit key/value cache: quantisation, its records bit by bit, and
attention over what the records stand for, in fp64 (integers for codes).

A token's 32 channels x_c of one kv head (bf16): lo = min x, s = bf16((max x -
lo) / 15), code = min(rne((x - lo) / s), 15); s below 2^-125: codes 0
and s = 2^-13 |lo| (0 below 2^-125); a group with a NaN or an infinity as s = NaN, lo = 0.
"""
from __future__ import annotations

import numpy as np

from .attention import widen_bf16

TILE = 16


def round_bf16(x):
    """fp64 -> bf16 bits (uint16), to nearest, ties to even, values in bf16's normal range or zero."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)  # x = m 2^e, 1/2 <= |m| < 1
    r = np.ldexp(np.rint(m * 256.0), e - 8).astype(np.float32)
    return (r.view(np.uint32) >> 16).astype(np.uint16)


def quantise(bits):
    """bf16 bits [..., d] -> (codes uint8 [..., d], scale bits [..., G], minimum bits [..., G])."""
    x = widen_bf16(bits).astype(np.float64)
    g = x.reshape(*x.shape[:-1], -1, 32)
    gb = np.asarray(bits).reshape(g.shape)
    bad = ((gb & 0x7f80) == 0x7f80).any(-1)
    safe = np.where(bad[..., None], 0.0, g)
    lo, hi = safe.min(-1), safe.max(-1)
    s = (hi - lo) / 15.0
    sb = np.where(s < 2.0 ** -127, 0, round_bf16(np.maximum(s, 2.0 ** -127))).astype(np.uint16)
    flat = sb < 0x0100
    sb = np.where(flat, 0, sb).astype(np.uint16)
    scale = widen_bf16(sb).astype(np.float64)
    q = np.divide(safe - lo[..., None], scale[..., None], out=np.zeros_like(safe), where=scale[..., None] > 0)
    codes = np.minimum(np.rint(q), 15).astype(np.uint8)
    lob = np.take_along_axis(gb, safe.argmin(-1)[..., None], -1)[..., 0]
    size = (lob & 0x7fff).astype(np.int64) - (13 << 7)
    sb = np.where(flat, np.where(size >= 0x0100, size, 0), sb)
    sb = np.where(bad, 0x7fc0, sb).astype(np.uint16)
    lob = np.where(bad, 0, lob).astype(np.uint16)
    codes = np.where(bad[..., None], 0, codes)
    return codes.reshape(x.shape), sb, lob


def _places(d, r):
    """For token r of a record: byte and nibble of every K and V code, bytes of the statistics of every group."""
    c = np.arange(d)
    g, G = c // 32, d // 32
    kw = ((g * 8 + r % 8) * 4 + c % 32 // 8) * 8 + r // 8 * 4
    k_byte, k_hi = kw + c % 8 // 2, c % 2
    t, rem = divmod(r % 8, 2)
    vw = 8 * d + ((g * 8 + c % 32 // 4) * 4 + t) * 8 + r // 8 * 4
    n = 4 * rem + c % 4
    v_byte, v_hi = vw + n // 2, n % 2
    gg = np.arange(G)
    stat = ((r % 8 * G + gg) * 2 + r // 8) * 2
    return k_byte, k_hi, v_byte, v_hi, 16 * d + stat, 17 * d + stat, 18 * d + stat, 19 * d + (gg * 16 + r) * 2


def _put16(rec, at, bits):
    rec[at] = bits & 0xff
    rec[at + 1] = bits >> 8


def _get16(rec, at):
    return rec[at].astype(np.uint16) | (rec[at + 1].astype(np.uint16) << 8)


def write_token(rec, r, k_bits, v_bits):
    """Writes token r of a record (uint8 [20 d], in place) from bf16 bits [d] of its key and value."""
    d = rec.size // 20
    kb, kh, vb, vh, ks, kl, vs, vl = _places(d, r)
    for byte, hi, s_at, l_at, bits in ((kb, kh, ks, kl, k_bits), (vb, vh, vs, vl, v_bits)):
        codes, sb, lob = quantise(bits)
        for at, up, code in zip(byte, hi, codes):
            rec[at] = (rec[at] & (0x0f if up else 0xf0)) | (int(code) << (4 if up else 0))
        _put16(rec, s_at, sb)
        _put16(rec, l_at, lob)


def read_token(rec, r):
    """Key and value [d] in fp64 of token r, and their parts:
    (k, v, (k scale, k minimum, v scale, v minimum) [d] each, (k codes, v codes))."""
    d = rec.size // 20
    kb, kh, vb, vh, ks, kl, vs, vl = _places(d, r)
    out, stats, codes = [], [], []
    for byte, hi, s_at, l_at in ((kb, kh, ks, kl), (vb, vh, vs, vl)):
        code = ((rec[byte] >> (4 * hi).astype(np.uint8)) & 15).astype(np.float64)
        s = np.repeat(widen_bf16(_get16(rec, s_at)).astype(np.float64), 32)
        lo = np.repeat(widen_bf16(_get16(rec, l_at)).astype(np.float64), 32)
        out.append(lo + s * code)
        stats += [s, lo]
        codes.append(code)
    return out[0], out[1], stats, codes


def read_cache(pool, table, n, h):
    """Tokens 0 .. n - 1 of the sequence with this table row, kv head h: dict of
    fp64 arrays [n, d]: k, v, ks, kl, vs, vl, kc, vc (scales, minima, codes)."""
    per = pool.shape[2]
    rows = [read_token(pool[table[j // TILE // per], h, j // TILE % per], j % TILE) for j in range(n)]
    d = pool.shape[3] // 20
    get = lambda f: np.array([f(r) for r in rows], np.float64).reshape(n, d)  # noqa: E731
    return {"k": get(lambda r: r[0]), "v": get(lambda r: r[1]), "ks": get(lambda r: r[2][0]),
            "kl": get(lambda r: r[2][1]), "vs": get(lambda r: r[2][2]), "vl": get(lambda r: r[2][3]),
            "kc": get(lambda r: r[3][0]), "vc": get(lambda r: r[3][1])}


def attention_kv4_fp64(q, caches, causal, scale):
    """q [n, Hq, d] (fp64) of one sequence, caches: read_cache of every kv head.
    Returns (O [n, Hq, d], LSE [n, Hq], tol_O, tol_LSE): the last two bound the
    errors of a computation with the codes as operands, see below."""
    n, Hq, d = q.shape
    group = Hq // len(caches)
    O, L = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    tO, tL = np.zeros((n, Hq, d)), np.zeros((n, Hq))
    for h in range(Hq):
        c = caches[h // group]
        N = c["k"].shape[0]
        for i in range(n):
            see = min(N, N - n + i + 1) if causal else N
            if see <= 0:
                continue
            x = scale * (c["k"][:see] @ q[i, h])
            m = x.max()
            p = np.exp(x - m)
            l = p.sum()
            O[i, h] = p @ c["v"][:see] / l
            L[i, h] = m + np.log(l)
            # scores: fp32 sums over d codes and the minima; 32 roundings of 2^-24 of what is summed
            size = scale * ((c["ks"] * c["kc"] + np.abs(c["kl"]))[:see] @ np.abs(q[i, h]))
            ex = 2.0 ** -19 * size.max() + 2.0 ** -20
            # weights are taken against a reference that stands off the largest score by the scales'
            # exponent and at most 8 steps of two more: x - reference and reference + log2(sum) are
            # rounded at that size, 2^-24 of it each (fp32, in units of log 2)
            ex += 2 * 2.0 ** -24 * np.log(2) * (8 + abs(np.log2(max(c["vs"][:see].max(), 2.0 ** -126))))
            w = p / l
            # weights times scales in fp16 (half a step: 2^-11, and 2^-25 of a unit of
            # 2^-7 of the largest scale), weights of the minima in 16 bits, results in bf16
            tiny = 15 * see * 2.0 ** -32 * c["vs"][:see].max() / l
            tO[i, h] = 2.0 ** -8 * np.abs(O[i, h]) + (2.0 ** -11 + 2 * ex) * (w @ (c["vs"] * c["vc"])[:see]) + \
                (2.0 ** -15 + 2 * ex) * (w @ np.abs(c["vl"][:see])) + tiny
            tL[i, h] = ex + 2.0 ** -22 * abs(L[i, h])
    return O, L, tO, tL
