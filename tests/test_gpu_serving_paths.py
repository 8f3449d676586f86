"""GPU tests of the serving operators along the paths that only larger, cut or
unusual calls take, with the definitions and bounds of test_gpu_serving.py.
"""
import numpy as np
import pytest
import torch

from test_gpu_serving import DEV, attend_case, attend_ref, dev32, random_cache

pytestmark = pytest.mark.gpu

import quantized_weight_block_gb300 as ndq  # noqa: E402


# ---- attention: calls that compute only some of a request's queries ----------------


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("n,most", [([3, 1, 2], 1), ([9, 2, 4], 4), ([300, 5, 70], 64), ([300, 150, 290], 260)])
def test_attend_queries_beyond_max_q_leave_the_others_in_place(n, most, window):
    # (the queries that are computed keep their positions, and the rest of out stays as it was)
    kv, D, bs = [400, 333, 290], 128, 16
    q, kc, ks, vc, vs, table, start = attend_case(kv, n, 8, 2, D, bs, "e4m3", torch.bfloat16, 71)
    want, bound, lse_want = attend_ref(q, kc, ks, vc, vs, table, kv, start, bs, D ** -0.5, window, torch.bfloat16)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
    ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start),
                      max_q=most, window=window, out=out, lse=lse)
    for r, a in enumerate(start[:-1]):
        c = a + min(n[r], most)
        assert ((out[a:c].double() - want[a:c]).abs() <= bound[a:c]).all(), r
        assert ((lse[a:c] - lse_want[a:c]).abs() <= 2.0 ** -13).all(), r
        assert (out[c:start[r + 1]] == 7).all() and (lse[c:start[r + 1]] == 7).all(), r


@pytest.mark.parametrize("fresh,n_tokens", [([1, 4, 3], 6), ([40, 2, 200], 100), ([700, 5], 512)])
def test_plan_append_and_attention_with_room_for_fewer_tokens(fresh, n_tokens):
    # a plan keeps the true lengths of a request that brings more tokens than there is room for
    bs, H, D, cached = 16, 2, 64, [33, 0, 50][:len(fresh)]
    R = len(fresh)
    blocks = [-(-(c + f) // bs) for c, f in zip(cached, fresh)]
    nb = sum(blocks) + 2
    table = np.full((R, max(blocks) + 1), -1, dtype=np.int32)
    at = 0
    for r, c in enumerate(cached):
        table[r, :-(-c // bs)] = np.arange(at, at - (-c // bs))
        at += -(-c // bs)
    tt = torch.from_numpy(table).to(DEV)
    kc, ks = random_cache(nb, H, bs, D, "int8", 81)
    vc, vs = random_cache(nb, H, bs, D, "int8", 82)
    cache = ndq.KvCache(kc, vc, ks, vs)
    plan = ndq.kv_plan(dev32(cached), dev32(fresh), bs, dev32(range(at, nb)), dev32([nb - at]), tt, n_tokens=n_tokens)
    g = torch.Generator(device=DEV).manual_seed(83)
    q = torch.randn(n_tokens, 4, D, device=DEV, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(n_tokens, H, D, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    ndq.kv_append(cache, k, v, plan.slots)
    out = ndq.attention_kv8(q, cache, tt, plan.kv_len, q_start=plan.q_start, max_q=max(fresh))
    # the same rows as queries of requests of just so many tokens
    start = [min(int(s), n_tokens) for s in plan.q_start.tolist()]
    kv = [c + start[r + 1] - start[r] for r, c in enumerate(cached)]
    want, bound, _ = attend_ref(q, kc, ks, vc, vs, tt.cpu().numpy(), kv, start, bs, D ** -0.5, 0, torch.bfloat16)
    err = (out.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


# ---- what a call on another stream makes for itself --------------------------------


def side_calls():
    """Calls without outputs or workspaces, each as (call, the library's
    function, which of its arguments is the workspace)."""
    bs, D, kv, n = 16, 128, [5000, 41], [2, 60]
    q, kc, ks, vc, vs, table, start = attend_case(kv, n, 8, 2, D, bs, "e4m3", torch.bfloat16, 91)
    cache, tt, kl, qs = ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), dev32(start)
    g = torch.Generator(device=DEV).manual_seed(92)
    x, a, b = (torch.randn(s, device=DEV, generator=g).to(torch.bfloat16) for s in ((300, 1024), (2, 16, 1024), (2, 512, 16)))
    base, index = torch.randn(300, 512, device=DEV, generator=g), dev32([i % 2 for i in range(300)])
    ranks, scales = dev32([16, 16]), torch.ones(2, device=DEV)
    plan = (dev32([3, 40]), dev32([700, 1]), bs, dev32(range(60)), dev32([60]), torch.arange(100, dtype=torch.int32, device=DEV).reshape(2, 50))

    return {
        "attention": (lambda **kw: ndq.attention_kv8(q, cache, tt, kl, q_start=qs, max_q=60, **kw), "ndq_attention_kv8", 16),
        "adapters": (lambda **kw: ndq.lora_add(x, a, b, ranks, scales, index, base, **kw), "ndq_lora_add", 14),
        "plan": (lambda **kw: ndq.kv_plan(*plan, n_tokens=701, **kw), "ndq_kv_plan", None),
    }


def values(y):
    return y if isinstance(y, torch.Tensor) else torch.cat([z.long() for z in (y.q_start, y.kv_len, y.positions, y.slots, y.free_left)])


@pytest.mark.parametrize("name", ["attention", "adapters", "plan"])
def test_a_call_on_another_stream_owns_what_it_makes(name, monkeypatch):
    call, fn, ws_arg = side_calls()[name]
    want = values(call())
    seen = []
    raw = getattr(ndq._lib, fn)
    monkeypatch.setattr(ndq._lib, fn, lambda *args: (seen.append(args), raw(*args))[1])
    side = torch.cuda.Stream()
    # freed memory of every size on the current stream, still to be written there
    torch.cuda.synchronize()
    sizes = [1 << i for i in range(9, 26)] + [ndq.ndq_attention_workspace_bytes(128)]
    junk = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
    torch.cuda._sleep(100_000_000)
    for z in junk:
        z.fill_(255)
    del junk
    got = call(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(values(got), want)
    # the workspace, while the call's kernels have not run: not for the current stream
    if ws_arg is not None:
        seen.clear()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
        got = call(stream=side)
        at, nbytes = seen[0][ws_arg], seen[0][ws_arg + 1]
        later = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes + [nbytes] for _ in range(3)]
        assert all(z.data_ptr() + z.numel() <= at or z.data_ptr() >= at + nbytes for z in later)
        torch.cuda.current_stream().synchronize()
        side.synchronize()
        assert torch.equal(got, want)


# ---- block tables: outputs beside the inputs ---------------------------------------


def test_plan_outputs_next_to_its_inputs():
    # arrays that touch without overlapping are taken; kv_len and free_left go on as the next step's cached and count
    R, T, bs, W = 3, 6, 16, 4
    buf = torch.zeros(200, dtype=torch.int32, device=DEV)
    parts, at = {}, 0
    for name, n in (("slots", 2 * T), ("cached", R), ("kv_len", R), ("fresh", R), ("q_start", R + 1), ("free", 20), ("table", R * W),
                    ("count", 1), ("positions", T), ("left", 1)):
        parts[name] = buf[at:at + n]
        at += n
    parts["cached"].copy_(dev32([15, 0, 40])), parts["fresh"].copy_(dev32([2, 3, 1]))
    parts["free"].copy_(torch.arange(20, device=DEV)), parts["count"].fill_(20)
    parts["table"].view(R, W)[:] = dev32([[30, -1, -1, -1], [-1] * 4, [31, 32, 33, -1]])
    out = ndq.KvPlan(parts["q_start"], parts["kv_len"], parts["positions"], parts["slots"].view(torch.int64), parts["left"])
    table = parts["table"].view(R, W)
    ndq.kv_plan(parts["cached"], parts["fresh"], bs, parts["free"], parts["count"], table, out=out)
    assert out.q_start.tolist() == [0, 2, 5, 6] and out.kv_len.tolist() == [17, 3, 41] and out.free_left.tolist() == [18]
    assert out.slots.tolist() == [30 * 16 + 15, 19 * 16, 18 * 16, 18 * 16 + 1, 18 * 16 + 2, 33 * 16 + 8]
    with pytest.raises(ndq.NdqError):
        ndq.kv_plan(out.kv_len, parts["fresh"], bs, parts["free"], parts["count"], table, out=out)
    second = ndq.kv_plan(out.kv_len, parts["fresh"], bs, parts["free"], out.free_left, table, n_tokens=T)
    assert second.kv_len.tolist() == [19, 6, 42] and second.positions.tolist() == [17, 18, 3, 4, 5, 41]
    assert second.slots.tolist() == [19 * 16 + 1, 19 * 16 + 2, 18 * 16 + 3, 18 * 16 + 4, 18 * 16 + 5, 33 * 16 + 9]
    assert second.free_left.tolist() == [18]
