"""GPU tests of qkq_attention_kv8's weights where they lie far apart: a first token that takes nearly all of the
softmax and has no value to give, and pages whose value steps differ by 2^20."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import transform_rope_head_b200 as qkq  # noqa: E402
from tests import kv8_common as C  # noqa: E402

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def sequence(L, d, page, seed):
    """A cache of one sequence and key head, keys zero, values between 1/2 and 2, steps 1."""
    cache = qkq.kv8_cache(-(-L // page), 1, page, d)
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.rand(cache.v.shape, generator=g, device="cuda") * 1.5 + 0.5
    cache.v.copy_(v.to(torch.float8_e4m3fn))
    cache.k_steps.fill_(1.0)
    cache.v_steps.fill_(1.0)
    return cache, torch.arange(cache.k.shape[0], dtype=torch.int32, device="cuda")[None], torch.tensor([L], dtype=torch.int32, device="cuda")


def check(cache, table, lens, n, ratio, d, dtype):
    """Queries (1, 1, 0, ..) and the scale log 2: a token's weight is 2 to the sum of its first two key channels,
    exactly.  What may go wrong: a weight times value step rounded to fp16 (2^-11 of it, or 2^-25 where the
    row's largest stands at 2^7 or more, hence 2^-32 of that), 2^-22 for each exponential, the sums' additions (L / 16 +
    64 in a chain, twice 2^-24 each, in numerator and denominator), the output's rounding."""
    L = int(lens)
    q = torch.zeros(n, ratio, d, device="cuda", dtype=dtype)
    q[..., :2] = 1.0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = qkq.attention_kv8(q, cache, table, lens, cu, scale=float(np.log(2.0)), want_lse=True, status=st)
    assert st.item() == 0
    k, v = (x.float().double().transpose(0, 1).reshape(-1, d)[:L] for x in (cache.k, cache.v))
    vs = cache.v_steps.double().repeat_interleave(cache.v.shape[2])[:L, None]
    s = k[:, 0] + k[:, 1]
    for t in range(n):
        see = slice(0, L - n + t + 1)
        p = torch.exp2(s[see])
        ref = (p @ (v * vs)[see]) / p.sum()
        mag = (p @ (v * vs).abs()[see]) / p.sum()
        w = p * vs[see, 0]
        floor = 2.0 ** -32 * w.max() * v[see].abs().sum(0) / p.sum()
        rel = 2.0 ** -11 + 2 * 2.0 ** -22 + 2 * (L / 16 + 64) * 2.0 ** -23
        bound = (mag * rel + floor) * (1 + EPS[dtype]) + ref.abs() * EPS[dtype] + 2.0 ** -25
        err = (out[t].double() - ref).abs()
        assert (err <= bound).all(), f"token {t}: {float((err / bound).max()):.3g} of the bound, {float((err / ref.abs()).max()):.3g} of the value"
        want = torch.log(p.sum())
        assert ((lse[t].double() - want).abs() <= 2.0 ** -22 * (1 + L / 16 + 64) + 2.0 ** -22 * (want.abs() + 60)).all()


# one token over the few-rows kernel (one n-tile, three), pieces over the prompt kernel (one query tile, two)
SHAPES = pytest.mark.parametrize("n,ratio,L", [(1, 4, 700), (1, 24, 5000), (1, 1, 60000), (20, 4, 3000), (90, 4, 2000)])
TYPES = pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])


@SHAPES
@TYPES
@pytest.mark.parametrize("loud", [20.5, 23.25, 24.5, 25.5, 27.0])
@pytest.mark.parametrize("at", [0, 40, 650])
def test_a_token_that_takes_the_weight_and_gives_nothing(n, ratio, L, d, dtype, loud, at):
    """Its logit is 2^loud of every other's: the output is what the others have to say."""
    cache, table, lens = sequence(L, d, 64, 1)
    page, row = at // 64, at % 64
    whole = 16.0 if loud < 24 else 24.0
    cache.k[page, 0, row, 0], cache.k[page, 0, row, 1] = whole, loud - whole
    cache.v.view(torch.uint8)[page, 0, row] = 0
    check(cache, table, lens, n, ratio, d, dtype)


@SHAPES
@TYPES
@pytest.mark.parametrize("above", [7.5, 8.0, 9.0])
def test_a_logit_just_within_what_the_maximum_lets_pass(n, ratio, L, d, dtype, above):
    """A later logit 2^7.5 to 2^9 over the first tokens': at most 2^15 in fp16, below its largest number."""
    cache, table, lens = sequence(L, d, 64, 2)
    cache.k[5:8, 0, :, 0] = 8.0
    cache.k[5:8, 0, :, 1] = above - 8.0
    check(cache, table, lens, n, ratio, d, dtype)


@SHAPES
@TYPES
def test_value_steps_far_apart(n, ratio, L, d, dtype):
    """One page has a loud value channel; the other channels come from the other pages."""
    cache, table, lens = sequence(L, d, 64, 3)
    cache.v.view(torch.uint8)[3] = 0
    cache.v[3, 0, :, 5] = 1.0
    cache.k[3, 0, :, 0] = 0.75
    cache.v_steps[3] = 2.0 ** (20 if dtype == torch.bfloat16 else 13)
    check(cache, table, lens, n, ratio, d, dtype)


@SHAPES
@TYPES
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 25, 2.0 ** 26, 2.0 ** 28, -2.0 ** 25])
@pytest.mark.parametrize("above", [4.0, 8.0, 16.0])
def test_logits_beyond_fp32s_fractions(n, ratio, L, d, dtype, size, above):
    """Logits so large that fp32 holds no fractions of them, a later page's `above` higher: no weight overflows,
    and the output lies among the values (1/2 to 2; a factor of 1.01 for the roundings)."""
    cache, table, lens = sequence(L, d, 64, 4)
    cache.k[:, 0, :, 2] = 256.0 if size > 0 else -256.0
    cache.k_steps.fill_(abs(size) / 256.0 / 64.0)  # the query's channel holds 64
    cache.k[5:8, 0, :, 0] = above / float(cache.k_steps[0, 0])
    q = torch.zeros(n, ratio, d, device="cuda", dtype=dtype)
    q[..., 0], q[..., 2] = 1.0, 64.0
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out, lse = qkq.attention_kv8(q, cache, table, lens, cu, scale=float(np.log(2.0)), want_lse=True)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert out.min() >= 0.5 / 1.01 and out.max() <= 2.0 * 1.01


@pytest.mark.parametrize("below", [28, 31, 34])
@pytest.mark.parametrize("n,ratio,L", [(1, 4, 700), (1, 24, 900), (40, 4, 900)])
def test_one_loud_query_channel(n, ratio, L, below):
    """A bf16 query channel 2^below over the others, where the keys are zero: the logits come from the others, which
    are exact down to 2^-31 of the loud one and off by at most 2^-39 of it under that (in the few-rows kernel)."""
    d = 128
    bt = C.dev_batch([n], [L - n], 32, 1, d, below)
    bt["cache"].k.view(torch.uint8)[..., 7] = 0
    g = torch.Generator(device="cuda").manual_seed(below)
    q = (torch.rand(n, ratio, d, generator=g, device="cuda") + 1.0) * torch.where(torch.rand(n, ratio, d, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    q[..., 7] = 2.0 ** below
    q = q.bfloat16()
    got = qkq.attention_kv8(q, bt["cache"], bt["table"], bt["lens"], bt["cu"])
    ref, _, mag, spread = C.dev_reference(q, bt, d ** -0.5)
    bound = C.attention_bound(ref, mag, spread, L, d, False)
    if below > 31 and n * ratio <= 24:
        # every other channel is at least 1: the logit is off by 2^(below - 39) of its spread, the weights in
        # numerator and denominator by that
        bound += mag * 2 * 2.0 ** (below - 39) * spread[..., None]
    assert (np.abs(got.double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
@pytest.mark.parametrize("n", [1, 40])
def test_log_sum_exps_take_the_weights_unrounded(n, d, dtype):
    """Short caches and small logits: the bound (152 x 2^-22 here) lies below what weights rounded to fp16 (2^-11 of
    them, of two to five about as large) would add to their sum."""
    C.check_dev([n] * 64, [1, 2, 3, 4] * 16 if n == 1 else [0] * 64, 16, 8, 2, d, dtype, seed=n, cu_none=n == 1, loud=0.05)
