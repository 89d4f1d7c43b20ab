"""GPU tests of append_kv8 and attention_kv8 on a stream that is not the current one: what the calls allocate is
neither taken from work that is still queued on the current stream nor given away while that stream uses it."""
import pytest

from tests import kv8_common as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import transform_rope_head_b200 as qkq  # noqa: E402

HOLD = 200_000_000  # clocks that the current stream is held for: a tenth of a second, calls take a thousandth


def case(what):
    """A call on a side stream, and tensors of the sizes that it allocates."""
    T, Hq, Hkv, d = 1500, 8, 2, 128
    bt = C.dev_batch([T], [0], 32, Hkv, d, 1)
    idx = (bt["table"], bt["lens"], bt["cu"])
    q = torch.randn(T, Hq, d, device="cuda").bfloat16()
    k = torch.randn(T, Hkv, d, device="cuda").bfloat16()
    if what == "append":
        return lambda s: qkq.append_kv8(k, k, bt["cache"], *idx, q=q, stream=s), [q.shape], [q.dtype]
    need = qkq.attention_kv8_workspace_bytes(T, 1, Hq, Hkv, d)
    return (lambda s: qkq.attention_kv8(q, bt["cache"], *idx, want_lse=True, stream=s),
            [q.shape, (T, Hq), (need,)], [q.dtype, torch.float32, torch.uint8])


@pytest.mark.parametrize("what", ["append", "attention"])
def test_freed_blocks_that_queued_work_still_reads(what):
    call, shapes, types = case(what)
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.full(s, 3, dtype=t, device="cuda") for s, t in zip(shapes, types)]
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)
    read = [x.clone() for x in old]  # queued: read when the stream goes on
    del old
    made = call(side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # the call was done first
    torch.cuda.synchronize()
    assert all((x == 3).all() for x in read)
    del made


@pytest.mark.parametrize("what", ["append", "attention"])
def test_returned_tensors_that_the_current_stream_still_reads(what):
    call, _, _ = case(what)
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    made = call(side)
    torch.cuda.synchronize()
    made = made if isinstance(made, tuple) else (made,)
    want = [x.clone() for x in made]
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)
    read = [x.clone() for x in made]
    shapes = [(x.shape, x.dtype) for x in made]
    del made
    with torch.cuda.stream(side):  # what asks next on the side stream
        other = [torch.full(s, 5, dtype=t, device="cuda") for s, t in shapes for _ in range(3)]
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want))
    del other


@pytest.mark.parametrize("what", ["append", "attention"])
def test_the_same_results_as_on_the_current_stream(what):
    call, _, _ = case(what)
    side = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    got = call(side)
    side.synchronize()
    for a, b in zip(*(x if isinstance(x, tuple) else (x,) for x in (want, got))):
        assert torch.equal(a, b)
