"""GPU tests of the serving operators along the paths that only larger, cut or
unusual calls take, with the definitions and bounds of test_gpu_serving.py.
"""
import numpy as np
import pytest
import torch

from test_gpu_serving import CODES, DEV, attend_case, attend_ref, check_append, check_attend, check_lora, dev32, random_cache

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


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("n,over", [([1, 1, 1], 1), ([4, 3, 1], 2), ([4, 4, 4], 40), ([200, 130, 70], 60), ([300, 40, 300], 500)])
def test_attend_tokens_past_the_table_are_not_seen(code, window, n, over):
    # (a plan whose table is too narrow: such tokens have no blocks, and the queries keep their positions)
    bs, D, W = 16, 128, 30
    kv = [W * bs + over, 300, W * bs + 2 * over]
    q, kc, ks, vc, vs, table, start = attend_case(kv, n, 8, 2, D, bs, code, torch.bfloat16, 181)
    narrow = np.ascontiguousarray(table[:, :W])
    hidden = table.copy()
    hidden[:, W:] = -1
    want, bound, lse_want = attend_ref(q, kc, ks, vc, vs, hidden, kv, start, bs, D ** -0.5, window, torch.bfloat16)
    if code == "e4m3":  # a NaN at the table's end reaches those that see it
        vc.view(torch.int8)[int(table[0, W - 1]), 0, bs - 1, 3] = 0x7f
    lse = torch.empty(q.shape[:2], device=DEV)
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(narrow).to(DEV), dev32(kv), q_start=dev32(start), window=window, lse=lse)
    nan = torch.zeros_like(out, dtype=torch.bool)
    if code == "e4m3":
        pos = torch.arange(kv[0] - n[0], kv[0], device=DEV)
        sees = (pos >= W * bs - 1) & ((pos < W * bs - 1 + window) if window else True)
        nan[:n[0], :4, 3] = sees[:, None]
    assert torch.equal(out.isnan(), nan)
    assert (((out.double() - want).abs() <= bound) | nan).all()
    none = torch.isinf(lse_want)
    assert torch.equal(torch.isinf(lse), none) and ((lse - lse_want)[~none].abs() <= 2.0 ** -13).all()


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


# ---- append: calls of more tokens, heads, K and V than one warp each (7296) ---------


def append_slots(spans, bs, skip=()):
    """Slots of requests of (tokens before, new tokens); those in `skip` have none."""
    blocks = [-(-(a + n) // bs) for a, n in spans]
    ids = np.random.default_rng(bs + len(spans)).permutation(sum(blocks) + 3)
    slots, at = [], 0
    for i, ((a, n), nb) in enumerate(zip(spans, blocks)):
        slots += [-1 if i in skip else int(ids[at + p // bs]) * bs + p % bs for p in range(a, a + n)]
        at += nb
    return slots, len(ids)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,D,bs", [(torch.bfloat16, 64, 16), (torch.float16, 128, 32), (torch.float16, 64, 64), (torch.bfloat16, 128, 128)])
@pytest.mark.parametrize("spans,skip", [
    ([(5, 220), (0, 129), (127, 1), (70, 200)] + [(i * 17 % 200, 1) for i in range(30)], (1, 9)),  # prompts and steps
    ([(i * 37 % 300, 1) for i in range(470)], (0, 17, 18, 469)),                                   # steps alone
    ([(i % 41, 1 + i % 7) for i in range(130)], (3,))])                                             # a few tokens each
def test_append_many(code, dtype, D, bs, spans, skip):
    heads = 8
    slots, nb = append_slots(spans, bs, skip)
    assert len(slots) * 2 * heads > 7296
    g = torch.Generator(device=DEV).manual_seed(D + bs)
    rows = torch.randn(len(slots), 2, heads, D, device=DEV, generator=g)
    rows = (rows * torch.exp(torch.randn(len(slots), 2, heads, 1, device=DEV, generator=g))).to(dtype)
    kc, ks = random_cache(nb, heads, bs, D, code, 101)
    vc, vs = random_cache(nb, heads, bs, D, code, 102, 0.2)
    check_append(rows[:, 0], rows[:, 1], slots, kc, ks, vc, vs, bs, code)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("bs", [16, 128])
def test_append_many_special_values(code, bs):
    heads, D = 8, 128
    slots, nb = append_slots([(5, 300), (40, 60), (0, 128)], bs)
    k, v = (torch.randn(len(slots), heads, D, device=DEV).to(torch.bfloat16) for _ in range(2))
    k[0, 0, 5], k[1, 0, 7], k[100, 1, 0], k[200, 1, 127], k[310, 7, 3] = float("nan"), float("inf"), -float("inf"), 3e38, -3e38
    v[20:60], v[330:] = 0.0, 0.0
    v[70, 2] = float("inf")
    v[100:140, 3], k[350:, 4] = 1e-38, float("nan")
    kc, ks = random_cache(nb, heads, bs, D, code, 103)
    vc, vs = random_cache(nb, heads, bs, D, code, 104)
    vs[::3] = 0.0
    vc.view(torch.int8)[::3] = 0
    check_append(k, v, slots, kc, ks, vc, vs, bs, code)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("growth", [0.0, 0.15])
def test_tokens_appended_one_by_one_stay_near_their_values(code, growth):
    # Every append of a larger value rounds the block's codes again.  A rounding
    # adds half a step: s / 2 (INT8); 2^-4 of the value, or 2^-10 s if that is
    # more (E4M3).  (2^-18 of it for the products and quotients in binary32.)
    bs, heads, D = 32, 2, 64
    g = torch.Generator(device=DEV).manual_seed(105)
    x = torch.randn(2, bs, heads, D, device=DEV, generator=g) * torch.exp(growth * torch.arange(bs, device=DEV))[:, None, None]
    x = x.to(torch.bfloat16)
    cache = ndq.KvCache.empty(2, heads, bs, D, CODES[code], DEV)
    err = torch.zeros(2, heads, bs, D, dtype=torch.float64, device=DEV)
    before = torch.zeros(2, heads, dtype=torch.float64, device=DEV)
    for i in range(bs):
        ndq.kv_append(cache, x[0, i:i + 1], x[1, i:i + 1], torch.tensor([bs + i], device=DEV))
        scale = torch.stack([cache.k_scale[1], cache.v_scale[1]]).double()
        rounded = torch.zeros_like(err, dtype=torch.bool)
        rounded[:, :, :i] = (scale > before)[:, :, None, None]
        rounded[:, :, i] = True
        s = scale[:, :, None, None]
        size = x.double().transpose(1, 2).abs() + err
        step = s / 2 if code == "int8" else torch.maximum(size * 2.0 ** -4, s * 2.0 ** -10)
        err += torch.where(rounded, step * (1 + 2.0 ** -18) + size * 2.0 ** -18, 0.0)
        before = scale
    got = torch.stack([cache.k[1].double() * cache.k_scale[1, :, None, None].double(), cache.v[1].double() * cache.v_scale[1, :, None, None].double()])
    assert ((got - x.double().transpose(1, 2)).abs() <= err).all()


# ---- attention: long shares, long prompts --------------------------------------------


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,n", [((8, 2), 1), ((32, 2), 1), ((8, 2), 4)])
def test_attend_shares_of_many_tiles(code, D, heads, n):
    # more than 4096 tokens of a request to a CTA, blocks missing far behind
    bs, R, L = 32, 40, 21000
    kv = [L - 37 * i for i in range(R)]
    q, kc, ks, vc, vs, table, start = attend_case(kv, [n] * R, *heads, D, bs, code, torch.bfloat16, 111)
    table[3, 400:420] = -1
    table[7, 150] = 1 << 30
    table[11, 17::50] = -5
    want, bound, _ = attend_ref(q, kc, ks, vc, vs, table, kv, start, bs, D ** -0.5, 0, torch.bfloat16)
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start), max_q=n)
    err = (out.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1700])
@pytest.mark.parametrize("kv,n,heads", [([3000, 2500, 90], [300, 1100, 1], (32, 8)),   # as many units as SMs: one CTA each
                                        ([40000], [64], (8, 2))])                       # few: their tokens split
def test_attend_long_prompts(code, D, window, kv, n, heads):
    bs = 16
    q, kc, ks, vc, vs, table, start = attend_case(kv, n, *heads, D, bs, code, torch.bfloat16, 121)
    table[0, 100:104] = -1
    want, bound, lse_want = attend_ref(q, kc, ks, vc, vs, table, kv, start, bs, D ** -0.5, window, torch.bfloat16)
    lse = torch.empty(q.shape[:2], device=DEV)
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start), max_q=max(n),
                            window=window, lse=lse)
    err = (out.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())
    assert ((lse - lse_want).abs() <= 2.0 ** -13).all()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_steps_and_prompts_together(code, dtype):
    n = [1] * 30 + [400] + [1] * 7 + [5, 0, 33]
    kv = [100 * i + 7 for i in range(30)] + [3000] + [50 * i for i in range(7)] + [900, 44, 33]
    check_attend(kv, n, 32, 8, 128, 16, code, dtype, seed=131)


# ---- adapters: many tiles to a CTA -----------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,N,nA,rank", [(2000, 512, 8192, 5, 16), (1500, 256, 8200, 3, 64), (1999, 64, 4099, 4, 8), (700, 128, 6000, 6, 128)])
def test_lora_many_tiles(dtype, M, K, N, nA, rank):
    rng = np.random.default_rng(M)
    runs = np.sort(rng.integers(-1, nA, M)).tolist()
    check_lora(M, K, N, nA, rank, dtype, runs)
    check_lora(M, K, N, nA, rank, dtype, rng.permutation(runs).tolist(), seed=1)
    check_lora(M, K, N, nA, rank, dtype, [(i // 23) % (nA + 1) - 1 for i in range(M)], seed=2, inplace=True)


def test_lora_more_tiles_than_are_weighed():
    check_lora(140000, 64, 264, 3, 8, torch.bfloat16, [(i // 999) % 4 - 1 for i in range(140000)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("which", ["base", "out", "both"])
def test_lora_tiles_with_outputs_off_16_bytes(dtype, which):
    M, K, N, nA, rank = 500, 256, 1024, 3, 16
    g = torch.Generator(device=DEV).manual_seed(141)
    x, a, b = (torch.randn(s, device=DEV, generator=g).to(torch.bfloat16) for s in ((M, K), (nA, rank, K), (nA, N, rank)))
    base = torch.randn(M, N, device=DEV, generator=g).to(dtype)
    index, ranks, scales = dev32([i * 5 // M - 1 for i in range(M)]), dev32([16, 9, 16]), torch.tensor([1.0, 0.5, 2.0], device=DEV)
    want = ndq.lora_add(x, a, b, ranks, scales, index, base)

    def off(t):
        buf = torch.zeros(M * N + 1, dtype=dtype, device=DEV)
        buf[1:] = t.flatten()
        return buf[1:].view(M, N)

    out = off(torch.zeros_like(base)) if which != "base" else torch.zeros_like(base)
    ndq.lora_add(x, a, b, ranks, scales, index, off(base) if which != "out" else base, out=out)
    assert torch.equal(out, want)  # (the same products in the same order)


# ---- attention: V's scales over their whole range ------------------------------------


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("n", [1, 4, 140])
@pytest.mark.parametrize("spread", ["random", "rising", "falling", "small with zeros", "large with zeros", "zeros first", "zeros"])
def test_attend_scales_of_v_over_their_range(code, n, spread):
    # A block counts in the denominator whatever its scale, and blocks of zeros
    # take no bits from the others.  (In tiles of 128 tokens and in small ones.)
    bs, D = 16, 128
    kv = [700, 3500]
    q, kc, ks, vc, vs, table, start = attend_case(kv, [n, n], 8, 2, D, bs, code, torch.bfloat16, 151)
    g = torch.Generator(device=DEV).manual_seed(152)
    nb = vs.shape[0]
    where = torch.full((nb,), -1.0, device=DEV)  # a block's place in its request, 0 .. 1
    for r in range(2):
        m = -(-kv[r] // bs)
        where[torch.from_numpy(table[r, :m].astype(np.int64)).to(DEV)] = torch.linspace(0, 1, m, device=DEV)
    one = torch.rand(vs.shape, device=DEV, generator=g) + 0.5
    power = {"random": torch.randint(-99, 99, vs.shape, device=DEV, generator=g).float(), "rising": (198 * where - 99).round()[:, None],
             "falling": (99 - 198 * where).round()[:, None], "small with zeros": -80.0, "large with zeros": 98.0, "zeros first": -70.0,
             "zeros": 0.0}[spread]
    vs.copy_(torch.ldexp(one, torch.as_tensor(power, device=DEV).int()))
    if spread.endswith("with zeros"):
        vs[::3] = 0.0
    elif spread == "zeros first":
        vs[where < 0.6] = 0.0
    elif spread == "zeros":
        vs.zero_()
    if code == "e4m3":  # codes of blocks of zeros may be anything but NaN
        vc.view(torch.int8)[(vc.view(torch.int8) & 0x7f) == 0x7f] = 0x11
    want, bound, lse_want = attend_ref(q, kc, ks, vc, vs, table, kv, start, bs, D ** -0.5, 0, torch.bfloat16)
    lse = torch.empty(q.shape[:2], device=DEV)
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start), lse=lse)
    err = (out.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())
    # (the logarithm's parts are of up to 108, in binary32)
    assert ((lse - lse_want).abs() <= 2.0 ** -13).all()


@pytest.mark.parametrize("n", [1, 4, 140])
def test_attend_nan_in_a_block_of_small_scale(n):
    bs, D, kv = 16, 128, [600]
    q, kc, ks, vc, vs, table, start = attend_case(kv, [n], 8, 2, D, bs, "e4m3", torch.bfloat16, 161)
    b = int(table[0, 9])
    vs[b] = 2.0 ** -95
    vc.view(torch.int8)[b, 1, 3, 17] = -1
    vc.view(torch.int8)[b, 1, 12, 80] = 0x7f
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start))
    expect = torch.zeros_like(out, dtype=torch.bool)
    expect[:, 4:, 17] = expect[:, 4:, 80] = True
    assert torch.equal(out.isnan(), expect)


@pytest.mark.parametrize("n", [1, 64])
def test_attend_nan_far_below_the_largest_score(n):
    # split over CTAs: a part whose weights vanish beside the others' still holds its NaN
    bs, D, kv = 16, 64, [20000]
    q, kc, ks, vc, vs, table, start = attend_case(kv, [n], 2, 1, D, bs, "e4m3", torch.bfloat16, 171)
    ks[torch.from_numpy(table[0, :1200].astype(np.int64)).to(DEV)] = 0.0  # score 0
    q[:] = 8.0
    late = torch.from_numpy(table[0, 1200:1250].astype(np.int64)).to(DEV)
    kc[late] = torch.full((), 256.0, device=DEV).to(torch.float8_e4m3fn)
    ks[late] = 1.0
    vc.view(torch.int8)[int(table[0, 2]), 0, 5, 33] = 0x7f
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start))
    expect = torch.zeros_like(out, dtype=torch.bool)
    expect[:, :, 33] = True
    assert torch.equal(out.isnan(), expect)
