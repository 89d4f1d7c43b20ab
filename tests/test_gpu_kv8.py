"""GPU tests of the paged 8-bit cache: qkq_append_kv8 bit for bit against the oracle's sequence,
qkq_attention_kv8 within its rounding bound of the float64 definition over the same bytes."""
import numpy as np
import pytest

from tests import kv8_common as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import transform_rope_head_b200 as qkq  # noqa: E402
from oracle import kv8 as O  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def tables(max_pos, rot, seed=0):
    a = np.arange(max_pos)[:, None] * 1e4 ** (-np.arange(0, rot, 2) / rot)[None]
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


# ---------------------------------------------------------------- append ---------------------

def run_append(n, cached, page, Hq, Hkv, d, rot, style, dtype, seed, cu_none=False, pos=False, strided=False, spare=0,
               poke=None):
    """Append through the binding and through the oracle; every byte of the cache has to agree."""
    r = np.random.default_rng(seed)
    bt = C.batch(n, cached, page, Hkv, d, seed + 1)
    C.fill(bt, Hkv, d, seed + 2, scale=0.25)   # quieter than what comes: steps of partly full pages grow
    T = int(bt["cu"][-1]) + spare
    tt = DT[dtype]
    qkv = C.rounded(C.values((T, Hq + 2 * Hkv, d), r), tt)
    if poke:
        poke(qkv)
    q, k, v = np.split(qkv, [Hq, Hq + Hkv], axis=1)
    cos, sin = tables(int(bt["lens"].max()) + 3, rot) if rot else (None, None)
    p = r.integers(0, cos.shape[0], T).astype(np.int32) if pos else None
    cache = C.dev_cache(bt["cache"])
    fused = dev(qkv).to(tt)
    parts = fused.split([Hq, Hkv, Hkv], 1)
    if not strided:
        parts = [x.contiguous() for x in parts]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((T, Hq, d), 7.0, dtype=tt, device="cuda")
    res = qkq.append_kv8(parts[1], parts[2], cache, dev(bt["table"]), dev(bt["lens"]), None if cu_none else dev(bt["cu"]),
                         q=parts[0], q_out=q_out, pos=None if p is None else dev(p), cos_tab=None if cos is None else dev(cos),
                         sin_tab=None if sin is None else dev(sin), rope_style=style, status=status)
    assert res is q_out
    torch.cuda.synchronize()
    want = [a.copy() for a in bt["cache"]]
    live = int(bt["cu"][-1])
    pl = None if p is None else p[:live]
    O.append(want, k[:live], v[:live], bt["table"], bt["lens"], bt["cu"], cos, sin, pl, rot, style)
    for got, ref, name in zip(C.host_cache(cache), want, ("k codes", "v codes", "k steps", "v steps")):
        np.testing.assert_array_equal(got, ref, err_msg=name)
    at = pl if p is not None else np.concatenate([np.arange(c, c + m) for m, c in zip(n, cached)])
    qr = q[:live]
    if rot:
        qr = O.rope_f32(qr, cos[at], sin[at], rot, style)
    qr = torch.from_numpy(np.ascontiguousarray(qr)).to(tt)
    assert torch.equal(q_out[:live].cpu().view(torch.int16), qr.view(torch.int16))
    assert (q_out[live:] == 7.0).all()
    return int(status.item())


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,rot,style,dtype", [(128, 128, "half", "bf16"), (128, 128, "interleaved", "fp16"),
                                               (128, 48, "half", "bf16"), (64, 64, "half", "fp16"),
                                               (64, 32, "interleaved", "bf16"), (64, 16, "half", "bf16"),
                                               (128, 0, "half", "bf16")])
def test_append_ragged(page, d, rot, style, dtype):
    """Prompt pieces and single tokens in one batch, starts and ends inside and at the ends of pages,
    an empty sequence, rows behind the last one."""
    n = [1, 0, page, page + 3, 5, 2 * page + 1, 1, 1]
    cached = [0, 9, page, 3, page - 5, page - 1, page - 1, 2 * page]
    assert run_append(n, cached, page, 6, 2, d, rot, style, dtype, seed=page + d + rot, spare=3) == 0


@pytest.mark.parametrize("page,d,Hq,Hkv", [(16, 128, 32, 8), (64, 64, 5, 5), (128, 128, 3, 1), (32, 64, 71, 1)])
@pytest.mark.parametrize("pos", [False, True])
def test_append_decode(page, d, Hq, Hkv, pos):
    """One token a sequence, no cu_new; parts of a fused projection as they are."""
    cached = [0, 1, page - 1, page, 3 * page + 7, 40, 15, 16, 17]
    assert run_append([1] * 9, cached, page, Hq, Hkv, d, d, "half", "bf16", seed=page + pos, cu_none=True, pos=pos,
                      strided=True) == 0


def test_append_many_sequences():
    """More sequences than a warp's search takes in one round."""
    r = np.random.default_rng(5)
    n, cached = r.integers(0, 4, 1100), r.integers(0, 50, 1100)
    assert run_append(list(n), list(cached), 16, 1, 1, 64, 64, "half", "bf16", seed=8, spare=1) == 0


def test_append_nonfinite_and_overflow():
    def poke(x):
        x[0, 2, 3] = np.inf       # a key
        x[1, 3, 5] = np.nan       # a value
        x[2, 2, :] = -np.inf      # a row with nothing finite
    st = run_append([3, 2], [4, 0], 16, 2, 1, 64, 0, "half", "bf16", seed=3, poke=poke)
    assert qkq.status_string(st) == "nonfinite"

    def huge(x):
        x[0, 2, 3] = 3e38
    assert qkq.status_string(run_append([1], [0], 16, 2, 1, 64, 0, "half", "bf16", seed=3, poke=huge)) == "scale_overflow"


def test_append_positions_outside_the_table():
    bt = C.batch([2], [0], 16, 1, 64, 1)
    cos, sin = tables(8, 64)
    k = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    qkq.append_kv8(k, k.clone(), C.dev_cache(bt["cache"]), dev(bt["table"]), dev(bt["lens"]), dev(bt["cu"]),
                   pos=dev(np.array([3, 9], np.int32)), cos_tab=dev(cos), sin_tab=dev(sin), status=st)
    assert qkq.status_string(st.item()) == "pos_range"


@pytest.mark.parametrize("what", ["page", "negative page", "length", "short length", "rows"])
def test_append_bad_index(what):
    """What lies outside the buffers is left out and reported; the other sequence is written."""
    bt = C.batch([2, 3], [5, 20], 16, 2, 64, 4)
    want = [a.copy() for a in bt["cache"]]
    lens, cu, table = bt["lens"].copy(), bt["cu"].copy(), bt["table"].copy()
    r = np.random.default_rng(9)
    k, v = (C.rounded(C.values((5, 2, 64), r), torch.bfloat16) for _ in range(2))
    O.append_rows(want[0], want[2], k[:2], table[:1], lens[:1], cu[:2])
    O.append_rows(want[1], want[3], v[:2], table[:1], lens[:1], cu[:2])
    if what == "page":
        table[1, 1] = want[0].shape[0]
    elif what == "negative page":
        table[1, 1] = -1
    elif what == "length":
        lens[1] = 16 * table.shape[1] + 1
    elif what == "short length":
        lens[1] = 2
    else:
        cu[2] = 6
    cache, st = C.dev_cache(bt["cache"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    qkq.append_kv8(dev(k).bfloat16(), dev(v).bfloat16(), cache, dev(table), dev(lens), dev(cu), status=st)
    assert qkq.status_string(st.item()) == "cache_index"
    for got, ref in zip(C.host_cache(cache), want):
        np.testing.assert_array_equal(got, ref)


# ---------------------------------------------------------------- attention ------------------

def run_attention(n, cached, page, Hq, Hkv, d, dtype="bf16", window=0, sinks=0, seed=0, cu_none=False, spare=0, scale=None,
                  lens=None, loud=1.0, poke=None, steps=None):
    r = np.random.default_rng(seed)
    bt = C.batch(np.asarray(n), np.asarray(cached), page, Hkv, d, seed + 1)
    both = dict(bt, cached=bt["n"] + bt["cached"])
    C.fill(both, Hkv, d, seed + 2)
    if steps:
        steps(bt["cache"])
    if lens is not None:
        bt["lens"] = np.asarray(lens, np.int32)
    if poke:
        poke(bt)
    live = int(bt["cu"][-1])
    T = live + spare
    q = C.rounded(r.standard_normal((T, Hq, d)) * loud, DT[dtype])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((T, Hq, d), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, Hq), 7.0, dtype=torch.float32, device="cuda")
    qkq.attention_kv8(dev(q).to(DT[dtype]), C.dev_cache(bt["cache"]), dev(bt["table"]), dev(bt["lens"]),
                      None if cu_none else dev(bt["cu"]), window=window, sinks=sinks, out=out, lse=lse, status=st, scale=scale)
    torch.cuda.synchronize()
    scale = d ** -0.5 if scale is None else scale
    ref, rl, mag, spread = O.attention(q[:live].astype(np.float64), bt["cache"], bt["table"], bt["lens"], bt["cu"], scale, window, sinks)
    got, gl = out.float().cpu().numpy(), lse.cpu().numpy()
    assert (got[live:] == 7.0).all() and (gl[live:] == 7.0).all()
    got, gl = got[:live], gl[:live]
    nan = np.isnan(ref)
    np.testing.assert_array_equal(np.isnan(got), nan)
    L = int(max(bt["lens"].max(), 1))
    bound = C.attention_bound(np.nan_to_num(ref), np.nan_to_num(mag), np.nan_to_num(spread), L, d, dtype == "fp16")
    err = np.abs(np.where(nan, 0.0, got - ref))
    assert (err <= bound).all(), f"{np.nanmax(err / bound):.3g} of the bound"
    empty = np.isneginf(rl)
    np.testing.assert_array_equal(np.isneginf(gl), empty)
    assert (got[empty] == 0).all()
    fin = np.isfinite(rl)
    # the statistics' relative error (as for the weights, without their rounding) and fp32's of the result
    tol = 2.0 ** -9 * 2.0 ** -2 + 2.0 ** -22 * (np.abs(rl[fin]) + 60 + spread[fin] * (d + 3) / 2)
    assert (np.abs(gl[fin] - rl[fin]) <= tol).all()
    return int(st.item())


@pytest.mark.parametrize("page,Hq,Hkv,d,dtype", [(16, 8, 2, 128, "bf16"), (32, 4, 4, 64, "fp16"), (64, 6, 1, 128, "fp16"),
                                                 (128, 8, 1, 64, "bf16"), (16, 12, 1, 128, "bf16"), (16, 9, 3, 64, "bf16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 0), (33, 3), (1, 17), (100000, 4)])
def test_decode(page, Hq, Hkv, d, dtype, window, sinks):
    """One query token a sequence: caches of one token, around tile and page ends, long enough for
    several parts; every head grouping of one and two n-tiles."""
    cached = [0, 1, 14, 15, 16, 31, 63, 64, 127, 128, 300, 1111]
    assert run_attention([1] * len(cached), cached, page, Hq, Hkv, d, dtype, window, sinks, seed=page + Hq, cu_none=True) == 0


@pytest.mark.parametrize("Hq,Hkv,d,page,window,sinks", [(8, 2, 128, 16, 0, 0), (8, 2, 64, 64, 0, 0), (4, 4, 128, 32, 17, 2),
                                                        (6, 1, 64, 16, 40, 5), (20, 1, 128, 128, 0, 0), (16, 2, 64, 32, 3, 1)])
def test_ragged_queries(Hq, Hkv, d, page, window, sinks):
    """Prompts, pieces behind cached tokens, single tokens and empty sequences in one batch; rows
    behind the last one left alone."""
    n = [3, 0, 1, 17, 40, 5, 130, 0]
    cached = [0, 4, 200, 100, 0, 31, 70, 0]
    assert run_attention(n, cached, page, Hq, Hkv, d, "bf16", window, sinks, seed=Hq + d, spare=5) == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 3)])
def test_prompt(dtype, d, window, sinks):
    assert run_attention([389, 260], [0, 133], 32, 4, 2, d, dtype, window, sinks, seed=d + window) == 0


def test_long_cache_splits():
    """A cache whose slices go to every part of the grid; the parts' sums are joined."""
    assert run_attention([1], [20000], 64, 8, 2, 128, seed=2, cu_none=True) == 0
    assert run_attention([1, 1, 1], [7000, 0, 9000], 16, 2, 1, 64, seed=3, cu_none=True) == 0
    assert run_attention([4], [9000], 128, 4, 1, 128, seed=4) == 0


def test_rows_that_see_nothing():
    """Padded entries: no cached tokens at all, and fewer than the new ones (negative indices)."""
    assert run_attention([1, 1, 1], [0, 50, 0], 16, 4, 2, 64, seed=5, cu_none=True, lens=[0, 51, 0]) == 0
    assert run_attention([6, 4, 20], [0, 3, 0], 16, 4, 2, 128, seed=6, lens=[2, 7, 0]) == 0


def test_large_and_small_logits():
    """Loud queries (one token takes the whole weight), a zero scale, a negative one."""
    run_attention([1, 9], [300, 100], 16, 4, 2, 128, seed=7, loud=300.0)
    run_attention([1, 9], [300, 100], 16, 4, 2, 128, seed=7, loud=1e-3)
    run_attention([1, 9], [300, 100], 16, 4, 2, 64, seed=8, scale=0.0)
    run_attention([1, 9], [300, 100], 16, 4, 2, 64, "fp16", seed=9, scale=-0.3)


def test_steps_of_very_different_pages():
    """Value and key steps far apart between pages, and steps outside the range that is read."""
    def steps(cache):
        r = np.random.default_rng(1)
        cache[2][:] = np.exp2(r.integers(-12, -4, cache[2].shape)).astype(np.float32)
        cache[3][:] = np.exp2(r.integers(-35, 12, cache[3].shape)).astype(np.float32)
    assert run_attention([1, 40], [200, 90], 16, 4, 2, 64, seed=11, steps=steps) == 0

    def ends(cache):
        cache[3][0::3] = 0.0
        cache[2][1::3] = 0.0
    assert run_attention([1, 40], [200, 90], 16, 4, 2, 128, seed=12, steps=ends) == 0


@pytest.mark.parametrize("n,cached,window,sinks", [([1], [70], 30, 2), ([50], [30], 0, 0), ([140], [20], 30, 4)])
def test_nan_codes_reach_only_rows_that_see_them(n, cached, window, sinks):
    """NaN in a cached key makes every row that sees it NaN, in a cached value one channel of those
    rows; rows that do not see it, and NaN behind the sequence's end, change nothing."""
    def poke(bt):
        page = bt["page"]
        for j, c, which in ((45, 5, 1), (68, 40, 1), (10, 0, 1), (1, 3, 1)):
            bt["cache"][which][bt["table"][0, j // page], 1, j % page, c] = 0xFF
        bt["cache"][0][bt["table"][0, 60 // page], 0, 60 % page, 9] = 0x7F
    assert run_attention(n, cached, 16, 4, 2, 64, window=window, sinks=sinks, seed=13, poke=poke) == 0


def test_attention_bad_index():
    """A page id outside the cache is left out, a length outside the table empties its rows, a row
    range outside the batch is left alone; each is reported."""
    bt = C.batch([1, 1, 1], [40, 40, 3], 16, 2, 64, 21)
    C.fill(dict(bt, cached=bt["n"] + bt["cached"]), 2, 64, 22)
    table, lens = bt["table"].copy(), bt["lens"].copy()
    table[0, 1] = 10 ** 6
    lens[1] = 16 * table.shape[1] + 1
    r = np.random.default_rng(23)
    q = C.rounded(r.standard_normal((3, 4, 64)), torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = C.dev_cache(bt["cache"])
    out = qkq.attention_kv8(dev(q).bfloat16(), cache, dev(table), dev(lens), status=st)
    assert qkq.status_string(st.item()) == "cache_index"
    assert (out[1] == 0).all()
    ref, _, mag, spread = O.attention(q.astype(np.float64), bt["cache"], bt["table"], bt["lens"], [0, 1, 2, 3], 0.125)
    b = C.attention_bound(ref, mag, spread, 64, 64, False)
    assert (np.abs(out[2].float().cpu().numpy() - ref[2]) <= b[2]).all()
    # sequence 0 without the page's 16 tokens: a shorter table row in its place
    keep = np.delete(table[:1], 1, axis=1)
    kept = O.attention(q[:1].astype(np.float64), bt["cache"], keep, [lens[0] - 16], [0, 1], 0.125)
    b = C.attention_bound(kept[0], kept[2], kept[3], 64, 64, False)
    assert (np.abs(out[0].float().cpu().numpy() - kept[0][0]) <= b[0]).all()
    st.zero_()
    out = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qkq.attention_kv8(dev(q).bfloat16(), cache, dev(bt["table"][:2]), dev(bt["lens"][:2]), dev(np.array([0, 1, 4], np.int32)),
                      out=out, status=st)
    assert qkq.status_string(st.item()) == "cache_index"
    assert (out[1:] == 7.0).all() and not (out[0] == 7.0).any()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes per buffer, the sequence's pages at its far end."""
    P, Hkv, page, d = 2 ** 21 + 64, 16, 1, 128
    page = 16
    P = 2 ** 32 // (Hkv * page * d) + 64
    cache = qkq.kv8_cache(P, Hkv, page, d)
    ids = np.arange(P - 5, P).astype(np.int32)[::-1].copy()
    r = np.random.default_rng(31)
    k, v = (C.rounded(C.values((70, Hkv, d), r), torch.bfloat16) for _ in range(2))
    q = C.rounded(r.standard_normal((70, Hkv, d)), torch.bfloat16)
    table, lens, cu = dev(ids[None]), dev(np.array([70], np.int32)), dev(np.array([0, 70], np.int32))
    qkq.append_kv8(dev(k).bfloat16(), dev(v).bfloat16(), cache, table, lens, cu)
    out = qkq.attention_kv8(dev(q).bfloat16(), cache, table, lens, cu).float().cpu().numpy()
    last = qkq.attention_kv8(dev(q[69:]).bfloat16(), cache, table, lens).float().cpu().numpy()
    small = [np.zeros((5, Hkv, page, d), np.uint8), np.zeros((5, Hkv, page, d), np.uint8), np.ones((5, Hkv), np.float32), np.ones((5, Hkv), np.float32)]
    tab = np.arange(5)[::-1].astype(np.int32)[None]
    O.append(small, k, v, tab, [70], [0, 70])
    np.testing.assert_array_equal(cache.k[P - 5:].view(torch.uint8).cpu().numpy(), small[0])
    np.testing.assert_array_equal(cache.v[P - 5:].view(torch.uint8).cpu().numpy(), small[1])
    ref, _, mag, spread = O.attention(q.astype(np.float64), small, tab, [70], [0, 70], 128 ** -0.5)
    bound = C.attention_bound(ref, mag, spread, 70, d, False)
    assert (np.abs(out - ref) <= bound).all() and (np.abs(last - ref[69:]) <= bound[69:]).all()


# ---------------------------------------------------------------- together -------------------

@pytest.mark.parametrize("d,style,dtype", [(128, "half", "bf16"), (64, "interleaved", "fp16")])
def test_prompt_then_decoding_steps(d, style, dtype):
    """As a server runs them: prompts appended and attended, then single tokens, then a mixed batch;
    the cache after every step is the oracle's, the outputs the definition's over it."""
    r = np.random.default_rng(41)
    B, Hq, Hkv, page = 3, 8, 2, 16
    tt = DT[dtype]
    cos, sin = qkq.rope_table(128, d, 1e4)
    cosn, sinn = cos.cpu().numpy(), sin.cpu().numpy()
    cache = qkq.kv8_cache(30, Hkv, page, d)
    mine = C.host_cache(cache)
    table = r.permutation(30)[:24].reshape(B, 8).astype(np.int32)
    lens = np.zeros(B, np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in ([20, 1, 37], [1, 1, 1], [1, 1, 1], [1, 30, 2], [1, 1, 1]):
        n = np.array(n)
        lens = (lens + n).astype(np.int32)
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T = int(cu[-1])
        x = C.rounded(C.values((T, Hq + 2 * Hkv, d), r), tt)
        q, k, v = dev(x).to(tt).split([Hq, Hkv, Hkv], 1)
        cud = None if (n == 1).all() else dev(cu)
        qr = qkq.append_kv8(k, v, cache, dev(table), dev(lens), cud, q=q, cos_tab=cos, sin_tab=sin, rope_style=style, status=st)
        out = qkq.attention_kv8(qr, cache, dev(table), dev(lens), cud, window=25, sinks=2, status=st)
        O.append(mine, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], table, lens, cu, cosn, sinn, None, d, style)
        for got, ref in zip(C.host_cache(cache), mine):
            np.testing.assert_array_equal(got, ref)
        qd = qr.double().cpu().numpy()
        ref, _, mag, spread = O.attention(qd, mine, table, lens, cu, d ** -0.5, 25, 2)
        bound = C.attention_bound(ref, mag, spread, int(lens.max()), d, dtype == "fp16")
        assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
    assert st.item() == 0


def test_graphs_and_streams():
    """Two captured graphs of the step (each call with a workspace of its own) replayed on two streams
    at once give what eager calls give, bit for bit; so does a call on a side stream."""
    B, Hq, Hkv, d, page = 4, 8, 2, 128, 16
    bt = C.batch([1] * B, [500, 3, 90, 1000], page, Hkv, d, 51)
    C.fill(dict(bt, cached=bt["n"] + bt["cached"]), Hkv, d, 52)
    cache = C.dev_cache(bt["cache"])
    table, lens = dev(bt["table"]), dev(bt["lens"])
    q = [torch.randn(B, Hq, d, device="cuda").bfloat16() for _ in range(2)]
    want = [qkq.attention_kv8(x, cache, table, lens) for x in q]
    again = [qkq.attention_kv8(x, cache, table, lens) for x in q]
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    graphs, outs = [], []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qkq.attention_kv8(x, cache, table, lens))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = qkq.attention_kv8(q[0], cache, table, lens, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0])


def test_in_place():
    """q as its own output, rotated and attended."""
    bt = C.batch([7, 1], [30, 100], 16, 2, 64, 61)
    C.fill(dict(bt, cached=bt["n"] + bt["cached"]), 2, 64, 62)
    cache = C.dev_cache(bt["cache"])
    args = (cache, dev(bt["table"]), dev(bt["lens"]), dev(bt["cu"]))
    q = torch.randn(8, 8, 64, device="cuda").half()
    k = torch.randn(8, 2, 64, device="cuda").half()
    cos, sin = (dev(t) for t in tables(128, 64))
    qr = qkq.append_kv8(k, k.clone(), *args, q=q, cos_tab=cos, sin_tab=sin)
    out = qkq.attention_kv8(qr, *args)
    x = q.clone()
    assert qkq.append_kv8(k, k.clone(), *args, q=x, q_out=x, cos_tab=cos, sin_tab=sin) is x and torch.equal(x, qr)
    assert torch.equal(qkq.attention_kv8(x, *args, out=x), out)
