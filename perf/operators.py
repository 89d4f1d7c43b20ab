"""The paged 8-bit key/value cache (KV8) and the attention over it: cases, plain forms and definitions.

Two operators. "append" writes new keys and values into pages, the position rotation applied on the way,
and rotates the queries; "attend" is causal softmax attention of new queries over the pages, optionally with a
sliding window and a few first tokens that stay visible.  The cache holds e4m3 codes [page, head, token, channel]
and one power-of-two step per page and head.
"""
import math

import torch

own = False

FP8_MAX = 448.0
STEP_EXP = 40  # steps lie in [2^-40, 2^40]


# ---------------------------------------------------------------- cases ------------------------

def _case(name, op, **kw):
    c = dict(op=op, B=1, new=1, cached=0, ragged=False, Hq=32, Hkv=8, d=128, page=16, dtype="bf16",
             rot=0, style="half", window=0, sinks=0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token of one conversation: the launch latency of a decoding step's cache write
        _case("append decode 1", "append", cached=1003, rot=128),
        # 256 decoding sequences at scattered positions (the repository's decode batch)
        _case("append decode 256", "append", B=256, cached=32700, ragged=True, rot=128),
        # eight prompts of 4096 tokens
        _case("append prompt 8x4096", "append", B=8, new=4096, page=64, rot=128),
        # ragged prompt pieces behind cached ones; half of a 64-channel head rotated, interleaved pairs
        _case("append ragged d64", "append", B=5, new=701, cached=300, ragged=True, d=64, page=32,
              dtype="fp16", rot=32, style="interleaved"),
        # one conversation's next token, short cache: latency
        _case("decode 1x1000", "attend", cached=999),
        # one token against a 128K-token cache: the cache split over the whole GPU
        _case("decode 1x131072", "attend", cached=131071, page=64),
        # a serving batch of ragged lengths
        _case("decode 64x8192", "attend", B=64, cached=8191, ragged=True),
        # window and sinks, 64-channel heads
        _case("decode 32 window", "attend", B=32, cached=32000, ragged=True, d=64, page=32,
              dtype="fp16", window=1024, sinks=4),
        # a few drafted tokens checked at once
        _case("verify 16x5", "attend", B=16, new=5, cached=4001, ragged=True, page=32),
        # a 2048-token prompt with 64-channel heads
        _case("prompt 2048 d64", "attend", new=2048, d=64, page=64),
        # a 4096-token piece of a prompt behind 8192 cached tokens
        _case("prompt 4096+8192", "attend", new=4096, cached=8192, page=128),
        # ragged prompts under a window with sinks
        _case("prompts 6 window", "attend", B=6, new=1501, cached=900, ragged=True, window=1000, sinks=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    ratio = rng.choice([1, 2, 3, 4, 6, 8])
    Hkv = rng.choice([1, 2, 4, 8]) if ratio > 4 else rng.choice([2, 4, 8])
    d = rng.choice([64, 128])
    kw = dict(Hq=ratio * Hkv, Hkv=Hkv, d=d, page=rng.choice([16, 32, 64, 128]),
              dtype=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.7)
    kind = rng.choice(["append", "decode", "verify", "prompt"])
    if kind == "append":
        if rng.random() < 0.5:
            kw.update(B=_log(rng, 1, 256), cached=_log(rng, 1, 32000))
        else:
            kw.update(B=rng.randint(1, 8), new=_log(rng, 2, 4096), cached=rng.choice([0, _log(rng, 1, 4000)]))
        kw.update(rot=rng.choice([d, d, d // 2, d // 4]), style=rng.choice(["half", "interleaved"]))
        return _case(None, "append", **kw)
    if rng.random() < 0.4:
        kw.update(window=_log(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 16, 33]))
    if kind == "decode":
        B = _log(rng, 1, 64)
        kw.update(B=B, cached=_log(rng, 1, min(131000, 500000 // B)))
    elif kind == "verify":
        B = _log(rng, 1, 32)
        kw.update(B=B, new=rng.randint(2, 16), cached=_log(rng, 1, min(32000, 200000 // B)))
    else:
        B = rng.randint(1, 6)
        kw.update(B=B, new=_log(rng, 17, 3000 // B + 100), cached=rng.choice([0, _log(rng, 1, 6000)]))
    return _case(None, "attend", **kw)


# ---------------------------------------------------------------- inputs -----------------------

def _lengths(case, seed):
    """New tokens and cached tokens of each sequence, on the host (lists).  Ragged lengths spread evenly over
    their range; the seed says which sequence has which."""
    B, new, cached = case["B"], case["new"], case["cached"]
    if not case["ragged"]:
        return [new] * B, [cached] * B
    # two sequences of well spread fractions (multiples of two irrational numbers, mod 1)
    n = [max(1, int(new * (1.0 - 0.9 * (0.6180339887 * b % 1.0)))) for b in range(B)]
    c = [int(cached * (1.0 - 0.95 * (0.7548776662 * (B - 1 - b) % 1.0))) for b in range(B)]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(7919 + int(seed))).tolist()
    return [n[b] for b in order], [c[b] for b in order]


def _values(shape, g, dtype, heads_dim):
    """Activations with a few loud channels per head and a magnitude per token, as keys and values have."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    loud = torch.rand(shape[heads_dim:], generator=g, device="cuda") < 0.03
    x = x * torch.where(loud, 12.0, 1.0)
    return x.to(dtype)


def _rope_rows(max_pos, rot, theta=5e5):
    w = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * w
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def prepare(case, seed):
    n, c = _lengths(case, seed)
    B, Hq, Hkv, d, ps = case["B"], case["Hq"], case["Hkv"], case["d"], case["page"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    T = sum(n)
    cu = torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    lens = torch.tensor([a + b for a, b in zip(n, c)], dtype=torch.int32).cuda()
    pages = [-(-(a + b) // ps) for a, b in zip(n, c)]
    most = max(pages)
    # of a sequence's pages, an append needs only those from the first new token on: the ones before point at page 0
    first = [b // ps if case["op"] == "append" else 0 for b in c]
    have = [p - f for p, f in zip(pages, first)]
    P = sum(have) + 1
    ids = (torch.randperm(P - 1, generator=g, device="cuda") + 1).to(torch.int32)
    col = torch.arange(most, device="cuda")[None, :]
    f, p = (torch.tensor(v, device="cuda")[:, None] for v in (first, pages))
    start = torch.tensor([0] + have, device="cuda").cumsum(0)[:-1, None]
    at = (start + col - f).clamp(0, P - 2)
    table = torch.where((col >= f) & (col < p), ids[at], torch.zeros_like(ids[at])).contiguous()
    # steps around 2^-5, as those of unit-variance activations with loud channels, and codes of that spread
    step = torch.exp2(torch.randint(-6, -3, (2, P, Hkv), generator=g, device="cuda").float())
    codes = []
    for _ in range(2):
        x = torch.randn((P, Hkv, ps, d), generator=g, device="cuda", dtype=torch.bfloat16)
        codes.append((x * 24.0).clamp_(-400, 400).to(torch.float8_e4m3fn))
    s = dict(case=case, cu=None if T == B and max(n) == 1 else cu, cu_all=cu, lens=lens, table=table, k_codes=codes[0],
             v_codes=codes[1], k_steps=step[0].contiguous(), v_steps=step[1].contiguous(), longest=max(a + b for a, b in zip(n, c)),
             most_new=max(n))
    if case["op"] == "append":  # one projection's output: queries, keys and values are parts of each token's row
        qkv = _values((T, Hq + 2 * Hkv, d), g, dtype, 1)
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hkv, Hkv], 1)
        s["cos"], s["sin"] = _rope_rows(s["longest"], case["rot"])
    else:
        s["q"] = _values((T, Hq, d), g, dtype, 1)
    return s


# ---------------------------------------------------------------- plain forms ------------------

def _tokens(s, T):
    """Sequence, index in the cache and the sequence's cached length of each new token."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(s["cu_all"][1:].contiguous(), t.int(), right=True)
    before = s["lens"] - (s["cu_all"][1:] - s["cu_all"][:-1])
    return t, b, (before[b] + t - s["cu_all"][b]).long(), before


def _rotate(x, cos, sin, rot, style):
    """fp32 rotation of pairs of the first `rot` channels, products and sums taken in 64 bits and rounded
    where the definition rounds: b*s to fp32, then a*c - that to fp32 (codes lie next to rounding borders)."""
    r = x[..., :rot].double()
    a, b = (r[..., : rot // 2], r[..., rot // 2 :]) if style == "half" else (r[..., 0::2], r[..., 1::2])
    c, s = cos[:, None, :].double(), sin[:, None, :].double()
    p = (a * c - (b * s).float().double()).float()
    q = (a * s + (b * c).float().double()).float()
    y = torch.cat([p, q], -1) if style == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([y, x[..., rot:].float()], -1)


def _step_of(amax):
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    k = torch.where(amax > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -STEP_EXP))
    return torch.exp2(k.clamp(-STEP_EXP, STEP_EXP).float())


def _store(y, codes, steps, s, b, at, before, ps):
    """Writes rows y [T, Hkv, d] (fp32) into codes / steps at cache index `at` of sequence b."""
    page, off = s["table"][b, at // ps].long(), at % ps
    need = torch.zeros_like(steps).index_reduce_(0, page, y.abs().amax(-1), "amax")
    touched = torch.zeros(steps.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    # pages that were partly full: the one of each sequence that holds its last cached token
    held = (before % ps).long()
    seqs = torch.arange(len(held), device="cuda")
    p0 = torch.where(held > 0, s["table"][seqs, (before // ps).long().clamp(max=s["table"].shape[1] - 1)].long(), 0)
    part = torch.zeros(steps.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, p0, True)
    part[0] = False  # page 0 holds no new tokens
    fresh = _step_of(need)
    new = torch.where(touched[:, None], torch.where(part[:, None], torch.maximum(steps, fresh), fresh), steps)
    old = codes[p0].float()
    again = (old * (steps[p0] / new[p0])[:, :, None, None]).to(torch.float8_e4m3fn)
    row = torch.arange(ps, device="cuda")[None, None, :, None] < held[:, None, None, None]
    keep = torch.where(row & part[p0][:, None, None, None], again.view(torch.uint8), codes[p0].view(torch.uint8))
    codes.view(torch.uint8)[p0] = keep
    codes.view(torch.uint8)[page, :, off] = (y / new[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    steps.copy_(new)


def _plain_append(s):
    c = s["case"]
    t, b, at, before = _tokens(s, s["k"].shape[0])
    cos, sin = s["cos"][at], s["sin"][at]
    _store(_rotate(s["k"], cos, sin, c["rot"], c["style"]), s["k_codes"], s["k_steps"], s, b, at, before, c["page"])
    _store(s["v"].float(), s["v_codes"], s["v_steps"], s, b, at, before, c["page"])
    return _rotate(s["q"], cos, sin, c["rot"], c["style"]).to(s["q"].dtype)


def _gathered(s, codes, steps):
    """[B, Hkv, tokens, d] fp32 of every sequence's pages, in order."""
    x = codes[s["table"].long()].float() * steps[s["table"].long()][..., None, None]  # [B, pages, Hkv, ps, d]
    return x.transpose(1, 2).flatten(2, 3)[:, :, : s["longest"]]


def _plain_attend(s):
    c = s["case"]
    T, Hq, d = s["q"].shape
    t, b, at, before = _tokens(s, T)
    slot = t - s["cu_all"][b]
    q = torch.zeros((c["B"], s["most_new"], Hq, d), device="cuda")
    q[b, slot] = s["q"].float()
    q = q.unflatten(2, (c["Hkv"], -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, ratio * new, d]
    S = (q @ _gathered(s, s["k_codes"], s["k_steps"]).transpose(-1, -2)) * d ** -0.5
    i = (before[:, None] + torch.arange(s["most_new"], device="cuda"))[:, None, :, None]
    j = torch.arange(S.shape[-1], device="cuda")
    see = j <= i
    if c["window"]:
        see &= (j > i - c["window"]) | (j < c["sinks"])
    see &= j < s["lens"][:, None, None, None]
    S = S.unflatten(2, (Hq // c["Hkv"], -1)).masked_fill_(~see[:, None], -math.inf)
    top = S.amax(-1, keepdim=True).clamp_min(-1e30)
    P = S.sub_(top).exp_()
    total = P.sum(-1, keepdim=True)
    v = _gathered(s, s["v_codes"], s["v_steps"])
    live = (j < s["lens"][:, None])[:, None, :, None]
    O = (P.flatten(2, 3) @ torch.where(live, v, 0.0)).unflatten(2, (Hq // c["Hkv"], -1)) / total.clamp_min(1e-30)
    O = O.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, new, Hq, d]
    return O[b, slot].to(s["q"].dtype)


def run(state):
    c = state["case"]
    if own:
        import transform_rope_head_b200 as qkq
        cache = qkq.KV8Cache(state["k_codes"], state["v_codes"], state["k_steps"], state["v_steps"])
        if c["op"] == "append":
            q = qkq.append_kv8(state["k"], state["v"], cache, state["table"], state["lens"], state["cu"],
                               q=state["q"], cos_tab=state["cos"], sin_tab=state["sin"], rope_style=c["style"])
        else:
            return qkq.attention_kv8(state["q"], cache, state["table"], state["lens"], state["cu"],
                                     window=c["window"], sinks=c["sinks"])
    elif c["op"] == "append":
        q = _plain_append(state)
    else:
        return _plain_attend(state)
    return dict(q=q, k=state["k_codes"], v=state["v_codes"], k_steps=state["k_steps"], v_steps=state["v_steps"])


# ---------------------------------------------------------------- definition -------------------

def _e4m3_exact(x):
    """Nearest e4m3 value of a float64 tensor, ties to even, |x| <= 448."""
    _, e = torch.frexp(x)
    ulp = torch.exp2((e - 4).clamp(min=-9).double())
    return (x / ulp).round() * ulp


def exact(case, seed):
    s = prepare(case, seed)
    n, c = _lengths(case, seed)
    ps, Hkv, d = case["page"], case["Hkv"], case["d"]
    cu = [0]
    for v in n:
        cu.append(cu[-1] + v)
    if case["op"] == "append":
        half, rot = case["rot"] // 2, case["rot"]
        first = [2 * i for i in range(half)] if case["style"] == "interleaved" else list(range(half))
        second = [2 * i + 1 for i in range(half)] if case["style"] == "interleaved" else [half + i for i in range(half)]
        at = torch.cat([torch.arange(b, a + b) for a, b in zip(n, c)]).cuda()

        def turned(x):
            y = x.double().clone()
            C, S = s["cos"][at].double()[:, None], s["sin"][at].double()[:, None]
            A, B = x[..., first].double(), x[..., second].double()
            y[..., first], y[..., second] = A * C - B * S, A * S + B * C
            return y
        out = dict(q=turned(s["q"]))
        seqs = range(case["B"])
        # every page that gets tokens: (sequence, page of it)
        todo = [(b, p) for b in seqs for p in range(c[b] // ps, (c[b] + n[b] - 1) // ps + 1)]
        ids = s["table"].cpu()
        page = torch.tensor([int(ids[b, p]) for b, p in todo], device="cuda")
        fill = torch.tensor([[cu[b] + p * ps + r - c[b] if c[b] <= p * ps + r < c[b] + n[b] else -1 for r in range(ps)]
                             for b, p in todo], device="cuda")
        held = torch.tensor([max(0, c[b] - p * ps) for b, p in todo], device="cuda")
        for name, y in (("k", turned(s["k"])), ("v", s["v"].double())):
            codes, steps = s[name + "_codes"].to(torch.float32), s[name + "_steps"].double()
            codes = codes.double() if codes.numel() < 3e8 else codes
            new = torch.where((fill >= 0)[:, :, None, None], y[fill.clamp(min=0)], 0.0).transpose(1, 2)  # [todo, Hkv, ps, d]
            amax = new.abs().amax((-1, -2))
            ends = FP8_MAX * torch.exp2(torch.arange(-STEP_EXP, STEP_EXP, device="cuda").double())
            want = torch.exp2((torch.searchsorted(ends, amax) - STEP_EXP).double())  # smallest 2^e with amax <= 448 2^e
            old = torch.where((held > 0)[:, None], steps[page], 0.0)
            step = torch.maximum(old, want)
            was = codes[page].double()
            kept = torch.where((old > 0)[..., None, None], _e4m3_exact(was * (old / step)[..., None, None]), was)
            r = torch.arange(ps, device="cuda")[None, None, :, None]
            now = torch.where((fill >= 0)[:, None, :, None], _e4m3_exact((new / step[..., None, None])),
                              torch.where(r < held[:, None, None, None], kept, was))
            codes[page] = now.to(codes.dtype)
            steps[page] = step
            out[name], out[name + "_steps"] = codes.double(), steps
        return out
    out = torch.zeros((cu[-1], case["Hq"], d), dtype=torch.float64, device="cuda")
    ratio = case["Hq"] // Hkv
    table = s["table"].long()
    for b in range(case["B"]):
        L = n[b] + c[b]
        own_pages = table[b, : -(-L // ps)]
        i = c[b] + torch.arange(n[b], device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        hidden = j > i
        if case["window"]:
            hidden |= (j <= i - case["window"]) & (j >= case["sinks"])
        for h in range(Hkv):
            k, v = ((s[w + "_codes"][own_pages, h].double() * s[w + "_steps"][own_pages, h].double()[:, None, None])
                    .reshape(-1, d)[:L] for w in ("k", "v"))
            q = s["q"][cu[b]:cu[b + 1], h * ratio:(h + 1) * ratio].double()
            S = torch.einsum("thc,jc->htj", q, k) / math.sqrt(d)
            S.masked_fill_(hidden, -math.inf)
            out[cu[b]:cu[b + 1], h * ratio:(h + 1) * ratio] = torch.einsum("htj,jc->thc", torch.softmax(S, -1), v)
    return out


# ---------------------------------------------------------------- work -------------------------

def work(case):
    """Bytes and operations that no implementation can leave out."""
    B, Hq, Hkv, d, ps = (case[k] for k in ("B", "Hq", "Hkv", "d", "page"))
    n, c = _lengths(case, 0)
    T = sum(n)
    if case["op"] == "append":
        io = T * (4 * Hq * d + 2 * 2 * Hkv * d + 2 * Hkv * d) + T * case["rot"] * 4 + 8 * B * Hkv
        return {"bytes": io, "flops": T * (Hq + Hkv) * case["rot"] * 3 + T * Hkv * d * 4}
    W, S = case["window"], case["sinks"]
    cache, pairs = 0, 0
    for a, b in zip(n, c):
        L = a + b
        if W:
            low = max(0, b - W + 1)  # first key in the first row's window
            cache += (L - low) + min(S, low)
            full = sum(min(i + 1, W + min(S, max(0, i + 1 - W))) for i in range(b, L))
        else:
            cache += L
            full = a * b + a * (a + 1) // 2
        pairs += full
    io = 4 * T * Hq * d + cache * (2 * Hkv * d) + cache * Hkv * 8 // ps
    return {"bytes": io, "flops": 4 * d * Hq * pairs}
