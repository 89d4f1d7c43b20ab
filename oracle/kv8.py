"""The paged 8-bit key/value cache in numpy: the append's bits and the attention's fp64 values.

``append`` follows the fp32 sequence of ``qkq_append_kv8`` (RoPE with the products and sums of its
two fused multiply-adds, the power-of-two step, one rounding to e4m3) on a cache held as e4m3 bytes
and fp32 steps; ``attention`` is the softmax of the definition in float64 over the same bytes.
"""
from __future__ import annotations

import numpy as np

STEP_EXP = 40


def e4m3_values() -> np.ndarray:
    """float64 value of each of the 256 e4m3 codes (sign, 4 exponent bits of bias 7, 3 mantissa
    bits; 0x7f and 0xff are NaN, there are no infinities)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where(c & 128, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


_VALUES = e4m3_values()
_POS = _VALUES[:0x7F]
_MID = (_POS[1:] + _POS[:-1]) / 2


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code, ties to the even code, magnitudes above 448 saturating, NaN to 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    lo = np.searchsorted(_MID, a, side="left")   # a == middle: the lower code
    tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)]) & (lo & 1 == 1)
    code = np.where(np.isnan(x), 0x7F, np.minimum(lo + tie, 0x7E) | (np.signbit(x) * 0x80))
    return code.astype(np.uint8)


def e4m3_decode(code: np.ndarray) -> np.ndarray:
    return _VALUES[code]


def rope_f32(x, cos, sin, rot, style):
    """x [T, H, d] float32, cos / sin [T, rot/2] float32 -> float32 [T, H, d]; a' = fma(a, c,
    -(b*s)), b' = fma(a, s, b*c) (80-bit floats hold the fused product and sum)."""
    x = np.asarray(x, dtype=np.float32)
    y = x.copy()
    if rot == 0:
        return y
    h = rot // 2
    ia, ib = (np.arange(h), np.arange(h) + h) if style == "half" else (np.arange(0, rot, 2), np.arange(1, rot, 2))
    a, b = x[..., ia], x[..., ib]
    c, s = cos[:, None, :], sin[:, None, :]
    L = np.longdouble
    with np.errstate(invalid="ignore"):
        y[..., ia] = (a.astype(L) * c.astype(L) - (b * s).astype(L)).astype(np.float32)
        y[..., ib] = (a.astype(L) * s.astype(L) + (b * c).astype(L)).astype(np.float32)
    return y


def step_of(amax: float) -> np.float32:
    e = -STEP_EXP
    while e < STEP_EXP and amax > 448.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def append_rows(codes, steps, y, table, seq_lens, cu):
    """Rows y [T, Hkv, d] float32 into codes [P, Hkv, ps, d] uint8 / steps [P, Hkv], in place."""
    ps = codes.shape[2]
    for b in range(len(seq_lens)):
        q0, n = int(cu[b]), int(cu[b + 1] - cu[b])
        before = int(seq_lens[b]) - n
        for pi in range(before // ps, (before + n - 1) // ps + 1 if n else 0):
            page = int(table[b, pi])
            lo, hi = max(before, pi * ps), min(before + n, (pi + 1) * ps)
            held = max(0, before - pi * ps)
            rows = y[q0 + lo - before:q0 + hi - before]
            for h in range(codes.shape[1]):
                mag = np.abs(rows[:, h])
                fin = mag[np.isfinite(mag)]
                step = step_of(float(fin.max()) if fin.size else 0.0)
                if held:
                    step = max(step, steps[page, h])
                    if step > steps[page, h]:
                        old = e4m3_decode(codes[page, h, :held]) * (float(steps[page, h]) / float(step))
                        codes[page, h, :held] = e4m3_encode(old)
                steps[page, h] = step
                codes[page, h, lo - pi * ps:hi - pi * ps] = e4m3_encode(rows[:, h].astype(np.float64) / float(step))


def append(cache, k, v, table, seq_lens, cu, cos=None, sin=None, pos=None, rot=0, style="half"):
    """cache = (k codes, v codes, k steps, v steps), updated in place; k, v [T, Hkv, d] float32."""
    if rot:
        if pos is None:
            pos = np.concatenate([np.arange(seq_lens[b] - (cu[b + 1] - cu[b]), seq_lens[b]) for b in range(len(seq_lens))])
        k = k.copy()
        n = len(pos)
        k[:n] = rope_f32(k[:n], cos[pos], sin[pos], rot, style)
    append_rows(cache[0], cache[2], np.asarray(k, np.float32), table, seq_lens, cu)
    append_rows(cache[1], cache[3], np.asarray(v, np.float32), table, seq_lens, cu)


def sequence(codes, steps, table, b, length):
    """float64 [length, Hkv, d] of sequence b's cached rows."""
    ps = codes.shape[2]
    ids = table[b, : -(-length // ps)]
    x = e4m3_decode(codes[ids]) * np.clip(steps[ids].astype(np.float64), 2.0 ** -40, 2.0 ** 40)[..., None, None]
    return x.transpose(0, 2, 1, 3).reshape(-1, codes.shape[1], codes.shape[3])[:length]


def visible(i, length, window, sinks):
    j = np.arange(length)
    see = j <= i
    if window > 0:
        see &= (j > i - window) | (j < sinks)
    return see


def attention(q, cache, table, seq_lens, cu, scale, window=0, sinks=0):
    """float64 (out [T, Hq, d], lse [T, Hq], mag [T, Hq, d], spread [T, Hq]) for q [T, Hq, d]
    float64: mag = sum p |v|, the size that relative errors of the weights act on; spread = the
    largest sum_c |scale q_c k_c| over the visible tokens, the size that errors of the logits act on.
    Rows of no sequence: NaN."""
    T, Hq, d = q.shape
    Hkv = cache[0].shape[1]
    out, mag = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse, spread = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for b in range(len(seq_lens)):
        n, L = int(cu[b + 1] - cu[b]), int(seq_lens[b])
        k, v = (sequence(cache[w], cache[w + 2], table, b, L) for w in (0, 1))
        for t in range(n):
            see = visible(L - n + t, L, window, sinks)
            r = int(cu[b]) + t
            if not see.any():
                out[r], mag[r], lse[r] = 0.0, 0.0, -np.inf
                continue
            for h in range(Hq):
                kk, vv = k[see, h // (Hq // Hkv)], v[see, h // (Hq // Hkv)]
                with np.errstate(invalid="ignore"):
                    s = scale * (kk @ q[r, h])
                    p = np.exp(s - s.max())
                    out[r, h], mag[r, h] = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
                    lse[r, h] = np.log(p.sum()) + s.max()
                    spread[r, h] = abs(scale) * (np.abs(kk) @ np.abs(q[r, h])).max()
    return out, lse, mag, spread
