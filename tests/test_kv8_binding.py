"""Refusals of the compiled binding of append_kv8 and attention_kv8 that need no GPU: each names its argument."""
import pytest

torch = pytest.importorskip("torch")

import transform_rope_head_b200 as qkq  # noqa: E402


def cpu():
    cache = qkq.kv8_cache(2, 1, 16, 64, device="cpu")
    return dict(q=torch.zeros(1, 2, 64, dtype=torch.bfloat16), k=torch.zeros(1, 1, 64, dtype=torch.bfloat16), cache=cache,
                table=torch.zeros(1, 1, dtype=torch.int32), lens=torch.ones(1, dtype=torch.int32))


def attention(**over):
    a = {**cpu(), **over}
    return qkq.attention_kv8(a["q"], a["cache"], a["table"], a["lens"])


def append(**over):
    a = {**cpu(), **over}
    return qkq.append_kv8(a["k"], a["k"], a["cache"], a["table"], a["lens"], rope_style=a.get("style", "half"))


@pytest.mark.parametrize("call", [attention, append])
def test_tensors_off_the_gpu(call):
    with pytest.raises(ValueError, match="CUDA device"):
        call()


def test_types():
    with pytest.raises(ValueError, match="q must be bfloat16 or float16"):
        attention(q=torch.zeros(1, 2, 64))
    with pytest.raises(ValueError, match="k must be bfloat16 or float16"):
        append(k=torch.zeros(1, 1, 64))
    with pytest.raises(ValueError, match="q must be"):
        attention(q=torch.zeros(1, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="block_table must be a tensor"):
        attention(table=None)
    with pytest.raises(TypeError, match="k must be a tensor"):
        append(k=[1, 2])
    with pytest.raises(KeyError):
        append(style="other")


def test_the_binding_is_built():
    """The module that the calls need exists beside the library (there is no other path)."""
    assert qkq._binding().append and qkq._binding().attention
