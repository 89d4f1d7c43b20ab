"""GPU tests of qkq_attention_kv8 on batches long enough that a CTA's part holds several units and each of them
many tiles, as a server's batches are: the start of a part found in every way, rings that go round."""
import numpy as np
import pytest

from tests import kv8_common as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


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
