"""GPU tests of qkq_attention_kv8 on batches long enough that a CTA's part holds several units and each of them
many tiles, as a server's batches are: the start of a part found in every way, rings that go round."""
import numpy as np
import pytest

from tests import kv8_common as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import transform_rope_head_b200 as qkq  # noqa: E402


@pytest.mark.parametrize("B,most,Hq,Hkv,d,dtype", [(256, 6000, 8, 2, 128, "bf16"), (600, 3000, 4, 1, 64, "fp16"),
                                                   (129, 5000, 24, 1, 128, "bf16")])
def test_decoding_batches_of_long_sequences(B, most, Hq, Hkv, d, dtype):
    """More sequences than a CTA of the few-rows kernel has threads, each with thousands of cached tokens: a part
    begins anywhere inside a sequence, and its start is found by the search over all sequences."""
    r = np.random.default_rng(B)
    C.check_dev([1] * B, r.integers(1, most, B), 64, Hq, Hkv, d, dtype, seed=B, cu_none=True, repeats=4)


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 4)])
def test_drafted_tokens_in_several_units(window, sinks):
    """Sequences whose drafted tokens fill two units beside ones with one: the part's start lies in the second."""
    r = np.random.default_rng(3)
    n = r.integers(1, 9, 40)
    n[::5] = 12
    C.check_dev(n, r.integers(100, 3000, 40), 32, 8, 2, 128, "bf16", window, sinks, seed=4, repeats=4)


# ---------------------------------------------------------------- the prompt kernel ------------

def prompts(n, cached, Hkv, d, dtype, window=0, sinks=0, page=64, seed=0, loud=1.0, long=True):
    """A batch for the prompt kernel (4 query heads a key head).  long: its line of tiles is long enough that
    CTAs have several units, and in the mean 20 places."""
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    parts = C.prompt_parts(n, cached, 4, Hkv, ctas, window, sinks)
    if long:
        assert sum(3 + k for part in parts for _, k in part) >= 20 * ctas
        assert max(len(part) for part in parts) > 1
    C.check_dev(n, cached, page, 4 * Hkv, Hkv, d, dtype, window, sinks, seed=seed, repeats=3, loud=loud)
    return parts


def skips(part):
    """Whether the second query tile's warps have nothing of some unit and go on to another of the part."""
    return any(rows <= 128 and tiles == 1 for rows, tiles in part[:-1])


HEADS = pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16"), (128, "fp16")])


@HEADS
def test_short_prompts_between_long_ones(d, dtype):
    """Eight units of one query tile and one token tile in a row, wide units of many tiles around them."""
    parts = prompts([3000, 20, 3000], [0, 30, 0], 8, d, dtype, seed=d)
    assert any(skips(part) for part in parts)


@HEADS
def test_sixteen_prompts(d, dtype):
    r = np.random.default_rng(d)
    n = np.exp(r.uniform(np.log(16), np.log(2000), 16)).astype(int)
    n[3], n[9] = 16, 2000
    prompts(n, [0] * 16, 8, d, dtype, page=16, seed=d + 1)


@HEADS
@pytest.mark.parametrize("behind", [30, 100, 300])
def test_decoding_tokens_beside_prompts(d, dtype, behind):
    """Decoding tokens behind short caches in the same call as prompts of 2000 tokens, before, between and after them."""
    n = [1] * 9 + [2000] + [1] * 12 + [2100] + [31] + [1] * 5
    cached = [behind] * 9 + [0] + [behind + 7] * 12 + [500] + [300] + [behind] * 5
    parts = prompts(n, cached, 8, d, dtype, page=32, seed=behind)
    if behind < 128:
        assert any(skips(part) for part in parts)


@HEADS
def test_odd_and_even_narrow_units_in_a_row(d, dtype):
    """Units of one query tile with 7 and 9 token tiles, some with 8, 2 and 1: the streams change places."""
    n = [32, 32, 20, 32, 7, 32, 32, 32] * 6
    cached = [800, 1040, 850, 1100, 20, 1100, 900, 200] * 6
    parts = prompts(n, cached, 8, d, dtype, seed=d + 2)
    odd = sum(rows <= 128 and tiles % 2 == 1 and i + 1 < len(part) for part in parts for i, (rows, tiles) in enumerate(part))
    assert odd > 20


@HEADS
def test_ragged_prompts_under_a_window(d, dtype):
    prompts([1501, 700, 333, 1100, 40, 1400], [900, 0, 600, 300, 800, 20], 8, d, dtype, 1000, 3, page=16, seed=d + 3)


@HEADS
def test_rescaled_rows_of_many_tiles(d, dtype):
    """Loud queries: a later tile's logits pass the running maximum, in wide units and in both streams of narrow ones."""
    prompts([1100, 30, 1100, 32, 32, 25], [3000, 5000, 1000, 7000, 3000, 1000], 8, d, dtype, page=128, seed=d + 4, loud=12.0)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_batches(seed):
    """Batches of every kind of unit, in any order."""
    r = np.random.default_rng(seed)
    B = int(r.integers(6, 40))
    n = np.where(r.random(B) < 0.5, r.integers(1, 40, B), np.exp(r.uniform(np.log(2), np.log(1500), B)).astype(int))
    n[r.integers(0, B)] = 1500
    cached = np.where(r.random(B) < 0.3, 0, np.exp(r.uniform(0, np.log(4000), B)).astype(int))
    window, sinks = [(0, 0), (int(r.integers(50, 1500)), int(r.integers(0, 200)))][seed % 2]
    prompts(n, cached, int(r.choice([2, 8])), int(r.choice([64, 128])), str(r.choice(["bf16", "fp16"])), window, sinks,
            page=int(r.choice([16, 32, 64, 128])), seed=seed, long=False)


@pytest.mark.parametrize("piece,behind", [(700, 0), (300, 2500), (1500, 1000)])
def test_single_tokens_and_a_piece_in_one_call_and_in_two(piece, behind):
    """255 decoding tokens and a piece of a prompt, which one kernel takes together (the few-rows one but for the
    longest piece) and two kernels apart, as the documentation advises."""
    B, Hq, Hkv, d = 255, 8, 2, 128
    r = np.random.default_rng(piece)
    n, cached = [1] * B + [piece], list(r.integers(1, 3000, B)) + [behind]
    C.check_dev(n, cached, 32, Hq, Hkv, d, seed=piece, repeats=2)
    bt = C.dev_batch(n, cached, 32, Hkv, d, piece)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(sum(n), Hq, d, generator=g, device="cuda").bfloat16()
    ref, _, mag, spread = C.dev_reference(q, bt, d ** -0.5)
    c, table, lens, cu = (bt[k] for k in ("cache", "table", "lens", "cu"))
    out = torch.cat([qkq.attention_kv8(q[:B], c, table[:B], lens[:B]),
                     qkq.attention_kv8(q[B:], c, table[B:], lens[B:], cu[B:] - B)])
    bound = C.attention_bound(ref, mag, spread, int(bt["host_lens"].max()), d, False)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


@HEADS
@pytest.mark.parametrize("window,sinks", [(0, 0), (400, 3)])
def test_nan_codes_in_batches_of_many_units(d, dtype, window, sinks):
    """NaN codes scattered over values and a few keys, in tiles that all, some and no rows see: a NaN value makes one
    channel of the rows that see it NaN, a NaN key whole rows, and nothing else changes."""
    n, cached = [900, 20, 31, 1100, 5, 1, 1500], [300, 30, 1100, 0, 2000, 700, 10]
    Hkv, ratio = 8, 4
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    bt = C.dev_batch(n, cached, 32, Hkv, d, d)
    g = torch.Generator(device="cuda").manual_seed(d)
    q = torch.randn(sum(n), Hkv * ratio, d, generator=g, device="cuda").to(dt)
    bad = [torch.rand(bt["cache"].k.shape, generator=g, device="cuda") < r for r in (2e-7, 4e-6)]
    clean = [torch.where(b, 0, c.view(torch.uint8)) for b, c in zip(bad, bt["cache"][:2])]
    for b, c in zip(bad, bt["cache"][:2]):
        c.view(torch.uint8)[b] = 0x7F
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):
        qkq.attention_kv8(q, bt["cache"], bt["table"], bt["lens"], bt["cu"], window=window, sinks=sinks, out=out, lse=lse, status=st)
    assert st.item() == 0
    ref, rl, mag, spread = C.dev_reference(q, dict(bt, cache=qkq.KV8Cache(*(c.view(torch.float8_e4m3fn) for c in clean), *bt["cache"][2:])),
                                           d ** -0.5, window, sinks)
    row_nan = torch.zeros(sum(n), Hkv, dtype=torch.bool, device="cuda")
    val_nan = torch.zeros(sum(n), Hkv, d, dtype=torch.bool, device="cuda")
    for b, L in enumerate(bt["host_lens"].tolist()):
        q0, q1 = bt["host_cu"][b:b + 2].tolist()
        ids = bt["table"][b, : -(-L // 32)].long()
        kb, vb = (x[ids].transpose(0, 1).reshape(Hkv, -1, d)[:, :L] for x in bad)
        i, j = L - (q1 - q0) + torch.arange(q1 - q0, device="cuda")[:, None], torch.arange(L, device="cuda")
        see = (j <= i) & ((j > i - window) | (j < sinks) if window else j >= 0)
        row_nan[q0:q1] = torch.einsum("tl,hl->th", see.float(), kb.any(-1).float()) > 0
        val_nan[q0:q1] = torch.einsum("tl,hld->thd", see.float(), vb.float()) > 0
    want = (val_nan | row_nan[..., None]).repeat_interleave(ratio, 1)
    assert want.any() and not want.all()
    assert torch.equal(torch.isnan(out), want)
    assert torch.equal(torch.isnan(lse), row_nan.repeat_interleave(ratio, 1))
    keep = ~want.cpu().numpy()
    bound = C.attention_bound(ref, mag, spread, int(bt["host_lens"].max()), d, dtype == "fp16")
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound)[keep].all()
    rows = ~torch.isnan(lse).cpu().numpy()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= C.lse_bound(rl, spread, int(bt["host_lens"].max()), d))[rows].all()
