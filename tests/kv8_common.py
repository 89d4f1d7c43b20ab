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


# ---------------------------------------------------------------- batches made on the GPU -----

def dev_batch(n, cached, page, Hkv, d, seed):
    """A batch as ``batch`` makes one, with its cache on the GPU: codes and steps as activations leave them,
    large enough for sequences of thousands of tokens.  Unused table entries name no page."""
    import torch
    import transform_rope_head_b200 as qkq
    r = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n, cached = np.asarray(n), np.asarray(cached)
    lens = (n + cached).astype(np.int32)
    need = -(-lens // page)
    P = int(need.sum()) + 1
    ids = r.permutation(P).astype(np.int32)
    table = np.full((len(n), max(1, int(need.max())) + 1), 2 ** 30, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    codes = [(torch.randn(P, Hkv, page, d, generator=g, device="cuda") * 24.0).clamp_(-400, 400).to(torch.float8_e4m3fn)
             for _ in range(2)]
    steps = [torch.exp2(torch.randint(-6, -3, (P, Hkv), generator=g, device="cuda").float()) for _ in range(2)]
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return dict(cache=qkq.KV8Cache(*codes, *steps), table=put(table), lens=put(lens), cu=put(cu), host_lens=lens, host_cu=cu)


def dev_reference(q, bt, scale, window=0, sinks=0):
    """``oracle.kv8.attention`` of a ``dev_batch`` on the GPU in float64: (out, lse, mag, spread), numpy."""
    import torch
    T, Hq, d = q.shape
    c = bt["cache"]
    Hkv, page = c.k.shape[1:3]
    out, mag = (torch.zeros(T, Hq, d, dtype=torch.float64, device="cuda") for _ in range(2))
    lse = torch.full((T, Hq), -float("inf"), dtype=torch.float64, device="cuda")
    spread = torch.zeros(T, Hq, dtype=torch.float64, device="cuda")
    for b, L in enumerate(bt["host_lens"].tolist()):
        q0, q1 = int(bt["host_cu"][b]), int(bt["host_cu"][b + 1])
        if q0 == q1 or L == 0:
            continue
        ids = bt["table"][b, : -(-L // page)].long()
        k, v = ((x[ids].double() * s[ids].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, d)[:, :L]
                for x, s in ((c.k, c.k_steps), (c.v, c.v_steps)))
        j = torch.arange(L, device="cuda")
        rows = max(1, 2 ** 26 // (Hq * L))
        for t0 in range(q0, q1, rows):
            t1 = min(t0 + rows, q1)
            i = L - (q1 - q0) + torch.arange(t0 - q0, t1 - q0, device="cuda")[:, None]
            see = j <= i
            if window:
                see &= (j > i - window) | (j < sinks)
            x = q[t0:t1].double().view(t1 - t0, Hkv, Hq // Hkv, d)
            s = torch.einsum("thrd,hld->thrl", x, k).mul_(scale).masked_fill_(~see[:, None, None], -float("inf"))
            p = torch.softmax(s, -1).nan_to_num_(0.0)
            put = lambda dst, src: dst[t0:t1].copy_(src.reshape(dst[t0:t1].shape))  # noqa: E731
            put(lse, torch.logsumexp(s, -1))
            put(out, torch.einsum("thrl,hld->thrd", p, v))
            put(mag, torch.einsum("thrl,hld->thrd", p, v.abs()))
            s = torch.einsum("thrd,hld->thrl", x.abs(), k.abs()).mul_(abs(scale)).masked_fill_(~see[:, None, None], 0.0)
            put(spread, s.amax(-1))
    return [x.cpu().numpy() for x in (out, lse, mag, spread)]


def check_dev(n, cached, page, Hq, Hkv, d, dtype="bf16", window=0, sinks=0, seed=0, cu_none=False, repeats=1,
              loud=1.0):
    """attention_kv8 of a ``dev_batch`` against float64: every output within ``attention_bound``, the
    log-sum-exps within theirs, status 0, and each repeat the same bits.  loud: the queries' spread."""
    import torch
    import transform_rope_head_b200 as qkq
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    bt = dev_batch(n, cached, page, Hkv, d, seed)
    T = int(bt["host_cu"][-1])
    g = torch.Generator(device="cuda").manual_seed(int(seed) + 1)
    q = (torch.randn(T, Hq, d, generator=g, device="cuda") * loud).to(dt)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q, bt["cache"], bt["table"], bt["lens"], None if cu_none else bt["cu"])
    got = []
    for _ in range(repeats):  # into outputs that no call has written
        out, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
        qkq.attention_kv8(*args, window=window, sinks=sinks, out=out, lse=lse, status=st)
        got.append((out, lse))
    torch.cuda.synchronize()
    assert st.item() == 0, qkq.status_string(st.item())
    ref, rl, mag, spread = dev_reference(q, bt, d ** -0.5, window, sinks)
    L = int(bt["host_lens"].max())
    out, lse = (x.double().cpu().numpy() for x in got[0])
    bound = attention_bound(ref, mag, spread, L, d, dtype == "fp16")
    assert (np.abs(out - ref) <= bound).all(), f"{np.nanmax(np.abs(out - ref) / bound):.3g} of the bound"
    assert (np.abs(lse - rl) <= lse_bound(rl, spread, L, d)).all()
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def lse_bound(lse, spread, L, d):
    """How far a log-sum-exp may be from float64's: the row sum takes the weights in fp32, before they are
    rounded for their product with the values, so of attention_bound's terms the exponential's 2^-22,
    the sum's additions (at most L / 16 + 64 in a chain, two roundings each) and the logits' remain (the d + 3
    roundings of a product acting on its spread); the result and its two summands (the offset, and the sum's
    logarithm with up to 40 for a value step and 20 for the count) are fp32 numbers."""
    return 2.0 ** -22 * (1 + L / 16 + 64) + 2.0 ** -22 * (np.abs(lse) + 60 + spread * (d + 3) / 2)


def prompt_parts(n, cached, ratio, Hkv, ctas, window=0, sinks=0):
    """The prompt kernel's work split on the host: per CTA the (query rows, token tiles) of its units.  A unit is
    256 query rows of a sequence and key head, its places 3 and one per tile of 128 tokens that some
    row sees; the line of all of them is cut in equal parts."""
    units = []
    for m, c in zip(n, cached):
        for r0 in range(0, m * ratio, 256):
            r1 = min(r0 + 256, m * ratio)
            first, last = c + r0 // ratio, c + (r1 - 1) // ratio
            seen = {j // 128 for j in range(last + 1) if not window or j > first - window or j < sinks}
            units += [(r1 - r0, len(seen))] * Hkv
    total = sum(t + 3 for _, t in units)
    share = -(-total // ctas)
    parts = [[] for _ in range(ctas)]
    at = 0
    for rows, tiles in units:
        for i in range(at // share, (at + tiles + 2) // share + 1):
            k = min(at + 3 + tiles, (i + 1) * share) - max(at + 3, i * share)
            if k > 0:
                parts[i].append((rows, k))
        at += tiles + 3
    return parts
