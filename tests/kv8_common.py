"""Helpers of the paged 8-bit cache's tests: seeded batches, device copies, tolerances."""
import numpy as np

from oracle import kv8 as O


def batch(n, cached, page, Hkv, d, seed, pages_extra=2, max_extra=1):
    """Index arrays of sequences with n new and cached earlier tokens, and a cache whose bytes and
    steps are garbage (NaN codes among them) wherever no sequence has written yet."""
    r = np.random.default_rng(seed)
    n, cached = np.asarray(n), np.asarray(cached)
    lens = (n + cached).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    need = -(-lens // page)
    P = int(need.sum()) + pages_extra
    ids = r.permutation(P).astype(np.int32)
    table = np.full((len(n), max(1, int(need.max())) + max_extra), 2 ** 30, dtype=np.int32)  # unused entries: no page
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    codes = [r.integers(0, 256, (P, Hkv, page, d), dtype=np.uint8) for _ in range(2)]
    steps = [np.exp2(r.integers(-8, 3, (P, Hkv))).astype(np.float32) for _ in range(2)]
    return dict(lens=lens, cu=cu, table=table, cache=[*codes, *steps], n=n, cached=cached, page=page,
                spare=ids[at:])


def fill(bt, Hkv, d, seed, scale=1.0):
    """Writes the sequences' earlier tokens into the batch's cache (by the oracle)."""
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(bt["cached"])]).astype(np.int64)
    k, v = (values((int(cu[-1]), Hkv, d), r) * scale for _ in range(2))
    O.append(bt["cache"], k, v, bt["table"], bt["cached"], cu)
    return k, v


def values(shape, r):
    """Unit normals with a few loud channels."""
    x = r.standard_normal(shape)
    x *= np.where(r.random(shape[1:]) < 0.04, 12.0, 1.0)
    return x.astype(np.float32)


def rounded(x, dtype):
    """float32 values that dtype holds exactly."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dtype).float().numpy()


def dev_cache(cache):
    import torch
    import transform_rope_head_b200 as qkq
    k, v = (torch.from_numpy(c.copy()).cuda().view(torch.float8_e4m3fn) for c in cache[:2])
    ks, vs = (torch.from_numpy(s.copy()).cuda() for s in cache[2:])
    return qkq.KV8Cache(k, v, ks, vs)


def host_cache(c):
    import torch
    return [c.k.view(torch.uint8).cpu().numpy(), c.v.view(torch.uint8).cpu().numpy(),
            c.k_steps.cpu().numpy(), c.v_steps.cpu().numpy()]


def attention_bound(out, mag, spread, L, d, half):
    """How far an output may be from the float64 one of the same codes.

    Weights: rounded to fp16, relative 2^-11; the logits are fp32 sums of d products (twice the
    rounding of each addition: the tensor cores may truncate) scaled in three fp32 roundings, and
    the exponential of a logit x (in units of log 2) is off by 2^-22 and by the rounding of x and of
    its maximum (|x| <= spread log2(e) + 40 for the step's exponent, twice for the difference), each
    acting relatively on p: in numerator and denominator, hence twice.  A weight below fp16's normal
    range is off by 2^-25 absolutely, at most 2^-25 x L of the largest weights' sum, which lies above
    2^-9 of the maximum's slack of 2^8.  Sums of L weights: fp32, at most L / 16 + 64 additions in a
    chain, two roundings each.  Output: rounded to its type."""
    x = spread[..., None] * 1.4427 + 40.0
    logit = 0.6932 * (2 * (d + 3) * 2.0 ** -24 * spread[..., None] * 1.4427 + 2 * x * 2.0 ** -23) + 2.0 ** -22
    rel = 2.0 ** -11 + 2 * logit + 2 * (L / 16 + 64) * 2.0 ** -23
    eps = 2.0 ** -11 if half else 2.0 ** -8
    tiny = 2.0 ** -25 if half else 0.0   # fp16 outputs below its normal range
    return mag * rel * (1 + eps) + np.abs(out) * eps + L * 2.0 ** -25 * 2.0 ** -8 * mag.max() + tiny
