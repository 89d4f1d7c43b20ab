"""GPU tests of qkq_attention_kv8's waits when they run out: one thread block of the prompt kernel waits for a tile
that never comes, all its waits end by their limit of 2 ms.  The kernel ends, the status says so, the rows
that the block had a part in are NaN and every other row is as ever."""
import pytest

from tests import kv8_common as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import transform_rope_head_b200 as qkq  # noqa: E402


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("n,cached", [([40], [1000]), ([600, 20, 31, 900], [0, 30, 1100, 300]),
                                      ([3000, 20, 32, 5, 3000], [0, 30, 1000, 900, 100])])
@pytest.mark.parametrize("cta", [0, 1, 5, 73, 75, 147, 100000])
def test_rows_whose_waits_ran_out(n, cached, d, dtype, cta):
    bt = C.dev_batch(n, cached, 32, 2, d, 3)
    T = sum(n)
    q = torch.randn(T, 8, d, device="cuda").to(dtype)
    args = (q, bt["cache"], bt["table"], bt["lens"], bt["cu"])
    want, want_lse = qkq.attention_kv8(*args, want_lse=True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((T, 8), 7.0, device="cuda")
    silent = torch.full_like(q, 7.0)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    parts = C.prompt_parts(n, cached, 4, 2, ctas)
    rows = sum(r for r, _ in parts[cta]) if cta < ctas else 0
    torch.cuda.synchronize()
    try:
        assert qkq.lib().qkq_selftest_attention_kv8_stall(2_000_000, cta) == 0
        qkq.attention_kv8(*args, out=out, lse=lse, status=st)
        qkq.attention_kv8(*args, out=silent)  # no status: the rows say it
    finally:
        assert qkq.lib().qkq_selftest_attention_kv8_stall(0, 0) == 0
    torch.cuda.synchronize()
    assert qkq.status_string(st.item()) == ("timeout" if cta < ctas else "ok")
    lost = torch.isnan(out)
    assert torch.equal(lost.all(-1), lost.any(-1)) and int(lost.all(-1).sum()) == rows
    assert torch.equal(torch.isnan(lse), lost.all(-1)) and torch.equal(torch.isnan(silent), lost)
    assert torch.equal(out[~lost], want[~lost]) and torch.equal(silent[~lost], want[~lost])
    assert torch.equal(lse[~lost.all(-1)], want_lse[~lost.all(-1)])
    # the context is as before
    st.zero_()
    again, again_lse = qkq.attention_kv8(*args, want_lse=True, status=st)
    assert st.item() == 0 and torch.equal(again, want) and torch.equal(again_lse, want_lse)
