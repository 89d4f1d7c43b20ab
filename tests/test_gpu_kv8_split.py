"""GPU tests of qkq_attention_kv8's work split and kernels at the sizes where they change: more sequences
than a CTA has threads, units of 8, 16, 24 and 256 query rows, tiles and pages that end inside one
another, parts of a unit on several CTAs.  Same bound as in test_gpu_kv8 (its derivation: kv8_common)."""
import numpy as np
import pytest

from tests import kv8_common as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import transform_rope_head_b200 as qkq  # noqa: E402
from tests.test_gpu_kv8 import DT, dev, run_attention  # noqa: E402


@pytest.mark.parametrize("B", [129, 700])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 1)])
def test_many_decoding_sequences(B, window, sinks):
    r = np.random.default_rng(B)
    assert run_attention([1] * B, list(r.integers(0, 60, B)), 16, 2, 1, 64, "bf16", window, sinks, seed=B, cu_none=True) == 0


@pytest.mark.parametrize("B,mean", [(600, 3), (530, 30)])
def test_many_ragged_sequences(B, mean):
    """Few rows a sequence (the register kernel) and more than 24 (tensor memory), empty ones among them."""
    r = np.random.default_rng(B)
    n = r.integers(0, 2 * mean, B)
    n[::7] = 0
    assert run_attention(list(n), list(r.integers(0, 40, B)), 16, 1, 1, 64, "fp16", seed=B, spare=3) == 0


@pytest.mark.parametrize("ratio", [1, 3, 8, 9, 16, 17, 24, 25, 32, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_one_token(ratio, d):
    """One token's heads in units of 8, 16 and 24 rows and in the prompt kernel."""
    assert run_attention([1] * 5, [0, 3, 17, 130, 900], 32, ratio, 1, d, "bf16", seed=ratio + d, cu_none=True) == 0


@pytest.mark.parametrize("n", [6, 7, 31, 32, 33, 63, 64, 65, 128, 129, 200])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_prompt_rows_around_the_tiles(n, d, dtype):
    """Rows that end inside and at the ends of the 128-row tiles and 256-row units, behind a cache that ends
    inside a tile of 128 tokens."""
    assert run_attention([n], [n % 5 * 40], 16, 4, 1, d, dtype, seed=n + d) == 0


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (140, 2)])
def test_prompt_wide_and_narrow_units(d, dtype, window, sinks):
    """Units of two query tiles and of one, whose token tiles go to two streams: one tile, two, odd counts, many."""
    n = [70, 10, 33, 64, 31, 97, 8, 40, 32, 65]
    cached = [0, 500, 95, 64, 1000, 160, 120, 0, 224, 300]
    assert run_attention(n, cached, 32, 4, 1, d, dtype, window, sinks, seed=d + window) == 0


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 0), (129, 5), (300, 200)])
def test_prompt_windows(page, window, sinks):
    """Windows shorter and longer than a tile, sinks inside the first tile and behind it, pages of every size."""
    assert run_attention([150, 1, 77], [260, 513, 0], page, 4, 2, 128, "bf16", window, sinks, seed=page + window) == 0


@pytest.mark.parametrize("d,dtype", [(128, "fp16"), (64, "bf16")])
def test_prompt_scales_and_loud_queries(d, dtype):
    for kw in (dict(scale=-0.2), dict(scale=0.0), dict(loud=200.0), dict(loud=1e-3)):
        run_attention([90, 40], [100, 0], 32, 4, 2, d, dtype, seed=d, **kw)


def test_prompt_long_cache_in_many_parts():
    """One unit's tiles on many CTAs, and rows whose first parts lie before all that they see."""
    assert run_attention([9], [9000], 64, 4, 1, 64, seed=71) == 0
    assert run_attention([9], [9000], 64, 4, 1, 128, "bf16", 50, 3, seed=72) == 0


def prompt(seed=81, d=128):
    bt = C.batch([300, 90], [200, 0], 32, 2, d, seed)
    C.fill(dict(bt, cached=bt["n"] + bt["cached"]), 2, d, seed + 1)
    return (C.dev_cache(bt["cache"]), dev(bt["table"]), dev(bt["lens"]), dev(bt["cu"]))


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_graphs_streams_and_repeats(d):
    """The same bits from a repeat, a side stream, and two captured graphs replayed at once."""
    args = prompt(d=d)
    q = [torch.randn(390, 8, d, device="cuda").bfloat16() for _ in range(2)]
    want = [qkq.attention_kv8(x, *args) for x in q]
    assert torch.equal(qkq.attention_kv8(q[0], *args), want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = qkq.attention_kv8(q[1], *args, stream=side, want_lse=True)
    side.synchronize()
    assert torch.equal(out, want[1]) and torch.isfinite(lse).all()
    graphs, outs = [], []
    for x in q:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qkq.attention_kv8(x, *args))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_graph_replays_follow_the_lengths():
    """A captured decoding step reads its lengths when it runs: appended tokens count at the next replay."""
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    cache = qkq.kv8_cache(60, Hkv, page, d)
    table = torch.arange(60, dtype=torch.int32, device="cuda").view(B, 20)
    lens = torch.tensor([1, 40, 100], dtype=torch.int32, device="cuda")
    k = torch.randn(141, Hkv, d, device="cuda").half()
    v = torch.randn(141, Hkv, d, device="cuda").half()
    cu = torch.tensor([0, 1, 41, 141], dtype=torch.int32, device="cuda")
    qkq.append_kv8(k, v, cache, table, lens, cu)
    q = torch.randn(B, Hq, d, device="cuda").half()
    qkq.attention_kv8(q, cache, table, lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens.add_(1)
        qkq.append_kv8(k[:B], v[:B], cache, table, lens)
        out = qkq.attention_kv8(q, cache, table, lens)
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [21, 60, 120]
    assert torch.equal(out, qkq.attention_kv8(q, cache, table, lens))


def test_no_tokens():
    cache = qkq.kv8_cache(2, 1, 16, 64)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.empty(0, 1, dtype=torch.int32, device="cuda")
    assert qkq.attention_kv8(q, cache, table, none).shape == q.shape
    assert qkq.append_kv8(q[:, :1].contiguous(), q[:, :1].contiguous(), cache, table, none, q=q).shape == q.shape


def test_fewer_checks_do_not_reach_the_device():
    """What the binding refuses with tensors on the device: nothing is launched, the outputs stay."""
    cache, table, lens, cu = prompt(d=64)
    q = torch.randn(390, 8, 64, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    for bad in (dict(out=out.half()), dict(out=out[:, :, :32]), dict(out=out, lse=torch.empty(3, device="cuda")),
                dict(out=out, workspace=torch.empty(4, dtype=torch.uint8)), dict(out=out, status=torch.zeros(1)),
                dict(out=out, window=2 ** 40)):
        with pytest.raises(ValueError):
            qkq.attention_kv8(q, cache, table, lens, cu, **bad)
    for bad in (dict(scale=float("nan")), dict(window=-1), dict(sinks=-1),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(qkq.QKQError):
            qkq.attention_kv8(q, cache, table, lens, cu, out=out, **bad)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
