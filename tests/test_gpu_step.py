"""GPU test of a generation step's operators together: in the example's layer
(one prompt, then several answers to it, step by step) the packed embedding, the
heads' norm and rotation and the attention behind the shared prompt are recorded
and checked against their definitions on the inputs that they got, with the
bounds of their own tests."""
import numpy as np
import pytest
import torch

import synth
from conftest import assert_bit_exact
from test_gpu_embed import expected, words
from test_gpu_example import _example
from test_gpu_rope import compare
from test_gpu_serving import attend_ref
from test_gpu_serving_paths import side_calls, values

pytestmark = pytest.mark.gpu

import quantized_weight_block_gb300 as ndq  # noqa: E402

DEV = "cuda"


@pytest.mark.parametrize("width", [20, 20000])  # (the wide tables' steps take the shared kernels)
@pytest.mark.parametrize("fmt", ["gguf:q8_0", "gguf:q4_k"])
def test_steps_stage_by_stage(fmt, width, orc, monkeypatch):
    ex = _example()
    hidden, vocab, R = 512, 300, 5
    layer = ex.AttentionLayer(fmt=fmt, num_blocks=80, hidden=hidden, q_heads=8, kv_heads=2, rotate=True, vocab=vocab)
    reqs = ex.Requests(R, 80, width)
    seen = {}

    def record(name):
        fn = getattr(ndq, name)

        def call(*a, **kw):
            before = [x.clone() if isinstance(x, torch.Tensor) else x for x in a]
            y = fn(*a, **kw)
            seen[name] = (before, kw, tuple(z.clone() for z in y) if isinstance(y, tuple) else y.clone())
            return y

        monkeypatch.setattr(ndq, name, call)

    for name in ("embed_packed", "qk_norm_rope", "attention_prefix_kv8", "attention_kv8"):
        record(name)
    shared, g = None, torch.Generator().manual_seed(3)
    none = [-1]
    for step in range(4):
        fresh = [200] + [0] * (R - 1) if step == 0 else [1, 3, 1, 2, 1]
        T = sum(fresh)
        seen.clear()
        plan = reqs.plan(fresh, 16)
        ids = torch.randint(0, vocab, (T,), generator=g)
        x = layer.embed(ids.to(DEV))
        assert_bit_exact(words(x), words(expected(orc, fmt, (vocab, hidden), synth.payload(fmt, (vocab, hidden), seed=9), ids, 1.0, "bfloat16")), "bfloat16")
        layer(x, torch.tensor(none * T, dtype=torch.int32, device=DEV), plan, reqs.table, max(fresh), shared)
        (q, k, pos, freq, qw, kw), _, (qo, ko) = seen["qk_norm_rope"]
        assert pos.tolist() == [reqs.cached.tolist()[r] - f + i for r, f in enumerate(fresh) for i in range(f)]
        compare(qo, q, pos, freq, qw, 1e-6, False, qo)
        compare(ko, k, pos, freq, kw, 1e-6, False, ko)
        name = "attention_kv8" if step == 0 else "attention_prefix_kv8"
        (q, _, table, kv_len, *_), _, got = seen[name]
        c = layer.cache
        want, bound, _ = attend_ref(q, c.k, c.k_scale, c.v, c.v_scale, table.cpu().numpy(), kv_len.tolist(),
                                    np.concatenate([[0], np.cumsum(fresh)]).tolist(), 16, 128 ** -0.5, 0, torch.bfloat16)
        assert ((got.double() - want).abs() <= bound).all()
        if step == 0:
            shared = reqs.share(192, 16)
            reqs.cached[0] = 192  # (the prompt's last tokens are not shared: every request brings its own)
    assert ndq.get_device_fault() == 0


def test_calls_on_another_stream_own_what_they_make():
    call, _, _ = side_calls()["attention"]
    call()
    g = torch.Generator(device=DEV).manual_seed(4)
    w, ids = torch.from_numpy(synth.payload("gguf:q8_0", (50, 1024), seed=1)).to(DEV), torch.randint(0, 50, (700,), device=DEV, generator=g)
    q, k = (torch.randn(700, h, 128, device=DEV, generator=g).to(torch.bfloat16) for h in (16, 4))
    pos, freq = torch.arange(700, dtype=torch.int32, device=DEV), torch.rand(64, device=DEV, generator=g)
    calls = [lambda **kw: ndq.embed_packed("gguf:q8_0", w, 50, 1024, ids, **kw), lambda **kw: torch.cat([y.flatten() for y in ndq.qk_norm_rope(q, k, pos, freq, **kw)]) if not kw else ndq.qk_norm_rope(q, k, pos, freq, **kw)]
    for call in calls:
        want = call()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        # freed memory of every size on the current stream, still to be written there
        junk = [torch.empty(1 << i, dtype=torch.uint8, device=DEV) for i in range(9, 26) for _ in range(3)]
        torch.cuda._sleep(100_000_000)
        for z in junk:
            z.fill_(255)
        del junk
        got = call(stream=side)
        torch.cuda.synchronize()
        got = torch.cat([y.flatten() for y in got]) if isinstance(got, tuple) else got
        assert torch.equal(got, want)


def test_prefix_workspace_made_for_another_stream_is_that_streams(monkeypatch):
    from test_gpu_prefix import Case
    c = Case([4], [512], [30, 0, 90, 5], [1] * 4, 8, 2, 128, 16, seed=5)
    cache, args = c.cache(), c.args()
    want = ndq.attention_prefix_kv8(c.q, cache, **args)
    seen = []
    raw = ndq._lib.ndq_attention_prefix_kv8
    monkeypatch.setattr(ndq._lib, "ndq_attention_prefix_kv8", lambda *a: (seen.append(a), raw(*a))[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = ndq.attention_prefix_kv8(c.q, cache, stream=side, **args)
    at, nbytes = seen[0][19], seen[0][20]
    later = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in [1 << i for i in range(9, 27)] + [nbytes] for _ in range(2)]
    assert all(z.data_ptr() + z.numel() <= at or z.data_ptr() >= at + nbytes for z in later)
    torch.cuda.synchronize()
    assert torch.equal(values(got).view(torch.int16), values(want).view(torch.int16))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fresh,bits", [([1, 1, 1, 1], 8 | 32), ([60, 1, 2, 1], 8 | 32)])
def test_prefix_copies_that_never_land(code, D, fresh, bits):
    # the kernels' failure path, without a GPU fault: waits for copies that are said to bring more than they do run out
    from test_gpu_prefix import Case
    c = Case([4], [700], [300, 40, 90, 500], fresh, 8, 2, D, 16, code, seed=6)
    cache, args, start = c.cache(), c.args(), torch.tensor(c.start, dtype=torch.int32, device=DEV)
    ws = ndq.attention_prefix_workspace(cache, c.q.shape[0], 8)

    def call():
        out = ndq.attention_prefix_kv8(c.q, cache, q_start=start, max_q=max(fresh), workspace=ws, **args)
        assert int(ws[:4096].count_nonzero()) == 0
        return out

    torch.cuda.synchronize()
    ndq.get_device_fault()
    try:
        want = call()
        torch.cuda.synchronize()
        assert ndq.get_device_fault() == 0
        assert ndq.ndq_test_lose_copies(2000) == 0
        call()
        torch.cuda.synchronize()
        assert ndq.get_device_fault() == bits
        for _ in range(2):  # the request was for one call
            got = call()
            torch.cuda.synchronize()
            assert ndq.get_device_fault() == 0
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    finally:
        ndq.ndq_test_lose_copies(0)
        torch.cuda.synchronize()
        ndq.get_device_fault()
