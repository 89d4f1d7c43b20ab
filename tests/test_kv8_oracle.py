"""CPU checks of the paged 8-bit cache: the oracle's e4m3 and steps, and the boundary's refusals."""
import ctypes

import numpy as np
import pytest

from oracle import kv8 as O

qkq = pytest.importorskip("transform_rope_head_b200")
torch = pytest.importorskip("torch")


def test_e4m3_codes_are_torchs():
    c = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(c).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(O.e4m3_values(), ref.astype(np.float64))
    r = np.random.default_rng(0)
    x = (r.standard_normal(20000) * np.exp2(r.integers(-12, 8, 20000))).astype(np.float32)
    x = np.clip(np.concatenate([x, O._MID, -O._MID, O._POS]), -448, 448).astype(np.float32)
    got = O.e4m3_encode(x)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(got, want)
    assert list(O.e4m3_encode(np.array([1e9, -1e9, np.inf, np.nan]))) == [0x7E, 0xFE, 0x7E, 0x7F]


@pytest.mark.parametrize("amax,exp", [(0.0, -40), (448.0, 0), (448.1, 1), (224.0, -1), (224.1, 0),
                                      (1e-30, -40), (3e38, 40), (1.0, -8), (0.875, -9)])
def test_step(amax, exp):
    assert O.step_of(amax) == 2.0 ** exp


def test_append_grows_a_partly_full_page():
    """A louder token doubles the step of a partly full page; what it held is rounded again."""
    codes, steps = np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.float32)
    table = np.zeros((1, 1), np.int32)
    y = np.full((1, 1, 64), 100.0, np.float32)
    O.append_rows(codes, steps, y, table, [1], [0, 1])
    assert steps[0, 0] == 0.25 and (O.e4m3_decode(codes[0, 0, 0]) == 384.0).all()  # 400: between 384 and 416, even is 384
    O.append_rows(codes, steps, y * 16, table, [2], [0, 1])
    assert steps[0, 0] == 4.0
    assert (O.e4m3_decode(codes[0, 0, 0]) * 4 == 96.0).all()
    # the page's next owner starts it afresh
    O.append_rows(codes, steps, y / 64, table, [1], [0, 1])
    assert steps[0, 0] == 2.0 ** -8


def test_attention_definition_against_torch():
    r = np.random.default_rng(3)
    cache = [r.integers(0, 0x7F, (3, 2, 16, 64), dtype=np.uint8) for _ in range(2)] + [np.full((3, 2), 2.0 ** -9, np.float32)] * 2
    table = np.array([[2, 0, 1]], np.int32)
    q = r.standard_normal((4, 4, 64))
    out, lse, _, _ = O.attention(q, cache, table, [37], [0, 4], 0.125, window=9, sinks=2)
    k, v = (torch.from_numpy(O.sequence(cache[w], cache[w + 2], table, 0, 37)).repeat_interleave(2, 1).transpose(0, 1) for w in (0, 1))
    i, j = np.arange(33, 37)[:, None], np.arange(37)[None]
    mask = torch.from_numpy((j <= i) & ((j > i - 9) | (j < 2)))
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).transpose(0, 1), k, v, attn_mask=mask, scale=0.125)
    np.testing.assert_allclose(out, ref.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)


# ---- refusals, before anything touches a device ------------------------------------------

V = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731


def _append(**over):
    a = dict(q=0x100000, qs=512, k=0x200000, ks=128, v=0x300000, vs=128, dtype=0, pos=None, T=4, cu=0x400000, lens=0x410000,
             B=2, table=0x420000, mp=4, P=8, ps=16, Hq=8, Hkv=2, d=64, rot=64, style=0, cos=0x500000, sin=0x510000, max_pos=64,
             out=0x600000, kc=0x700000, vc=0x800000, kst=0x900000, vst=0x910000, status=None)
    a.update(over)
    return qkq.lib().qkq_append_kv8(
        V(a["q"]), a["qs"], V(a["k"]), a["ks"], V(a["v"]), a["vs"], a["dtype"], V(a["pos"]), a["T"], V(a["cu"]), V(a["lens"]),
        a["B"], V(a["table"]), a["mp"], a["P"], a["ps"], a["Hq"], a["Hkv"], a["d"], a["rot"], a["style"], V(a["cos"]),
        V(a["sin"]), a["max_pos"], V(a["out"]), V(a["kc"]), V(a["vc"]), V(a["kst"]), V(a["vst"]), V(a["status"]), None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(kc=None), -1), (dict(vst=None), -1),
    (dict(out=None), -1), (dict(q=None), -1), (dict(cos=None), -1), (dict(lens=None), -1), (dict(table=None), -1),
    (dict(style=2), -1), (dict(style=0x100), -5),
    (dict(d=96), -2), (dict(d=256), -2), (dict(ps=8), -2), (dict(ps=48), -2), (dict(ps=256), -2), (dict(Hq=7), -2),
    (dict(Hkv=0), -2), (dict(T=-1), -2), (dict(B=-1), -2), (dict(mp=0), -2), (dict(mp=2 ** 26 + 1), -2), (dict(P=0), -2), (dict(cu=None), -2),
    (dict(rot=8), -2), (dict(rot=80), -2), (dict(rot=-16), -2), (dict(max_pos=0), -2), (dict(T=2 ** 31), -2),
    (dict(ks=64), -2), (dict(ks=132), -2), (dict(qs=100), -2), (dict(vs=127), -2),
    (dict(k=0x200008), -3), (dict(out=0x600008), -3), (dict(vc=0x800004), -3), (dict(cos=0x500004), -3),
    (dict(kst=0x900002), -3), (dict(status=0x2), -3), (dict(pos=0x2), -3),
    (dict(out=0x100000 + 64), -1),             # overlaps q without being it
    (dict(out=0x100000, qs=1024), -1),         # q in place must be contiguous
    (dict(out=0x200000), -1),                  # overlaps k
    (dict(vc=0x700000 + 2048), -1),            # K and V codes overlap
    (dict(T=0, B=0, cu=None, k=None), 0), (dict(T=0), 0), (dict(B=0), 0),
])
def test_append_refusals(over, code):
    assert _append(**over) == code


def _attend(**over):
    a = dict(q=0x100000, dtype=0, T=4, cu=0x400000, lens=0x410000, B=2, table=0x420000, mp=4, P=8, ps=16, kc=0x700000,
             vc=0x800000, kst=0x900000, vst=0x910000, Hq=8, Hkv=2, d=64, scale=0.125, window=0, sinks=0, out=0x600000,
             lse=None, ws=0xA00000, wsb=1 << 40, status=None)
    a.update(over)
    return qkq.lib().qkq_attention_kv8(
        V(a["q"]), a["dtype"], a["T"], V(a["cu"]), V(a["lens"]), a["B"], V(a["table"]), a["mp"], a["P"], a["ps"], V(a["kc"]),
        V(a["vc"]), V(a["kst"]), V(a["vst"]), a["Hq"], a["Hkv"], a["d"], a["scale"], a["window"], a["sinks"], V(a["out"]),
        V(a["lse"]), V(a["ws"]), a["wsb"], V(a["status"]), None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=-1), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(vc=None), -1), (dict(kst=None), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(window=-1), -1), (dict(sinks=-1), -1),
    (dict(d=32), -2), (dict(Hq=9), -2), (dict(ps=20), -2), (dict(T=5, cu=None), -2),
    (dict(q=0x100002), -3), (dict(out=0x600004), -3), (dict(lse=0x2), -3), (dict(ws=0xA00008), -3),
    (dict(out=0x100000 + 128), -1), (dict(ws=None), -6), (dict(wsb=64), -6),
    (dict(T=0), 0), (dict(B=0, T=0, cu=None, q=None), 0),
])
def test_attention_refusals(over, code):
    assert _attend(**over) == code


def test_workspace_bytes():
    f = qkq.attention_kv8_workspace_bytes
    assert f(0, 1, 8, 2, 64) == 0 and f(1, 0, 8, 2, 64) == 0 and f(1, 1, 9, 2, 64) == 0 and f(1, 1, 8, 2, 96) == 0
    assert f(1, 1, 8, 2, 64) > 0


def test_status_names():
    assert qkq.status_string(128) == "cache_index"
    assert qkq.status_string(129) == "nonfinite|cache_index"
    assert qkq.status_string(192) == "unknown status bits"
    assert qkq.status_string(256) == "unknown status bits"


def _tensors():
    c = qkq.kv8_cache(4, 2, 16, 64, device="cpu")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    return c, k, torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)


@pytest.mark.parametrize("change", [
    lambda a: a.update(k=a["k"].float()), lambda a: a.update(v=a["v"].half()), lambda a: a.update(v=a["v"][:2]),
    lambda a: a.update(table=a["table"].long()), lambda a: a.update(lens=a["lens"].long()),
    lambda a: a.update(lens=torch.ones(2, dtype=torch.int32)), lambda a: a.update(cu=None),
    lambda a: a.update(cu=torch.zeros(3, dtype=torch.int32)), lambda a: a.update(cache=a["cache"]._replace(k=a["cache"].k.view(torch.uint8))),
    lambda a: a.update(cache=a["cache"]._replace(k_steps=a["cache"].k_steps[:, :1])),
    lambda a: a.update(k=a["k"].transpose(0, 1).contiguous().transpose(0, 1)),
    lambda a: None,                            # as they are: not on a CUDA device
])
def test_binding_refuses(change):
    c, k, table, lens, cu = _tensors()
    a = dict(cache=c, k=k, v=k.clone(), table=table, lens=lens, cu=cu)
    change(a)
    with pytest.raises(ValueError):
        qkq.append_kv8(a["k"], a["v"], a["cache"], a["table"], a["lens"], a["cu"])
