"""GPU tests of append_kv8 and attention_kv8 behind one another without a pause, as a captured step of many layers runs
them: each kernel starts while the one before ends, and has to see all that it wrote."""
import pytest

from tests import kv8_common as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import transform_rope_head_b200 as qkq  # noqa: E402


@pytest.mark.parametrize("Hkv,d,page", [(32, 64, 16), (8, 128, 64)])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_that_grow_from_token_to_token(Hkv, d, page, captured):
    """Each token is louder than the one before, so that every append rewrites its page's steps and codes, which the
    attention behind it reads at once; after each token the same call on an idle GPU gives the same bits."""
    B, L = 12, 40
    table = torch.randperm(B * (-(-L // page)), device="cuda").int().view(B, -1)
    caches = [qkq.kv8_cache(table.numel(), Hkv, page, d) for _ in range(3)]  # three layers
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = torch.empty(3, B, 3 * Hkv, d, dtype=torch.bfloat16, device="cuda")
    noise = [torch.randn(x.shape, generator=g, device="cuda") for _ in range(L)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        outs = []
        for layer, cache in enumerate(caches):
            q, k, v = x[layer].split(Hkv, 1)
            qr = qkq.append_kv8(k, v, cache, table, lens, q=q, status=st)
            outs.append(qkq.attention_kv8(qr, cache, table, lens, status=st))
        return outs

    graph, held = None, None
    for i in range(L):
        x.copy_(noise[i] * 1.37 ** i)
        x[:, :, :Hkv].copy_(noise[i][:, :, :Hkv] * 1.37 ** -i)  # queries: logits of one size
        lens.fill_(i + 1)
        torch.cuda.synchronize()
        if captured and graph is None:
            before = [[t.clone() for t in c] for c in caches]
            step()  # warms up; the cache as it was for the captured run
            torch.cuda.synchronize()
            for c, b in zip(caches, before):
                for t, o in zip(c, b):
                    t.view(torch.uint8).copy_(o.view(torch.uint8))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                held = step()
        if captured:
            graph.replay()
            outs = [o.clone() for o in held]
        else:
            outs = step()
        torch.cuda.synchronize()
        for layer, cache in enumerate(caches):
            again = qkq.attention_kv8(x[layer][:, :Hkv].contiguous(), cache, table, lens)
            torch.cuda.synchronize()
            assert torch.equal(outs[layer], again), (i, layer)
    assert st.item() == 0


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
def test_prompts_on_two_streams_at_once(d, dtype):
    """Two captured prompt batches of several units a CTA, replayed at once: the same bits as alone."""
    args, want = [], []
    for seed, n, cached in ((1, [2000, 20, 900, 31], [0, 30, 500, 1100]), (2, [31, 1500, 1, 1800], [800, 100, 60, 0])):
        bt = C.dev_batch(n, cached, 32, 8, d, seed)
        q = torch.randn(sum(n), 32, d, device="cuda").to(dtype)
        args.append((q, bt["cache"], bt["table"], bt["lens"], bt["cu"]))
        want.append(qkq.attention_kv8(*args[-1]))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in args:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(qkq.attention_kv8(*a))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("ratio", [256, 300, 513])
def test_heads_beyond_a_unit(ratio):
    """A token whose heads fill more than a unit of 256 query rows."""
    C.check_dev([1, 3, 1], [700, 40, 0], 16, ratio, 1, 64, seed=ratio)
