"""GPU tests of the serving operators: block tables and slot maps, append to
the 8-bit cache, attention over it and low-rank adapters, each against its
definition evaluated apart from the library (whole numbers and codes exactly,
sums in 64 bits).

Attention's bound.  A weight 2^(t - m) f enters the product as binary16: one
rounding of at most 2^-11 of it, or 2^-25 of the largest weight when it is
that small.  A score is a binary32 sum of D products whose error is below
eps = 2^-20 * scale * sum |q k| (tensor-core sums may truncate), plus 2^-21 of
the score itself from the exponent's rounding, and moves a weight by at most
2 eps of it, in the numerator and in the denominator.  Hence
    |out - ref| <= (2^-11 + 2^-13 + 4 eps) sum p |v| + n 2^-24 max |v|
plus one rounding of the output (2^-8 bfloat16, 2^-11 binary16).

Adapters' bound.  Sums of K and then of rank binary32 terms, each term
rounded a few times: (K + 16) 2^-23 |B| (|A| |x|) + (rank + 16) 2^-23 |B| |t|
plus the addition of base and the output's rounding.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import quantized_weight_block_gb300 as ndq  # noqa: E402

DEV = "cuda"
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {"e4m3": 448.0, "int8": 127.0}
I32 = dict(dtype=torch.int32, device=DEV)


def dev32(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).tolist(), **I32)


# ---- block tables and slot maps ------------------------------------------------


def plan_ref(cached, fresh, bs, free, table, n_tokens):
    table = table.copy()
    q_start, kv, pos, slots, taken = [0], [], [], [], 0
    for r, (c, f) in enumerate(zip(cached, fresh)):
        c, f = max(c, 0), max(f, 0)
        had, need = -(-c // bs), -(-(c + f) // bs)
        ids = {}
        for b in range(had, need):
            ids[b] = free[len(free) - 1 - taken] if taken < len(free) else -1
            taken += 1
        for i in range(f):
            p = c + i
            b = p // bs
            ident = -1
            if b < table.shape[1]:
                ident = ids[b] if b >= had else table[r, b]
                if b >= had and len(pos) < n_tokens and p % bs == 0:
                    table[r, b] = ident
            pos.append(p)
            slots.append(ident * bs + p % bs if ident >= 0 else -1)
        q_start.append(q_start[-1] + f)
        kv.append(c + f)
    pos = (pos + [-1] * n_tokens)[:n_tokens]
    slots = (slots + [-1] * n_tokens)[:n_tokens]
    return q_start, kv, pos, slots, len(free) - taken, table


def check_plan(cached, fresh, bs, free, width, n_tokens, capacity=None, stream=None):
    R = len(cached)
    rng = np.random.default_rng(R + bs)
    table = rng.integers(0, 1 << 20, (R, width)).astype(np.int32)
    want = plan_ref(cached, fresh, bs, list(free), table, n_tokens)
    stack = np.concatenate([np.asarray(free, dtype=np.int64), np.full((capacity or len(free)) - len(free), 7777)])
    tt = torch.from_numpy(table).to(DEV)
    out = ndq.kv_plan_buffers(R, n_tokens)
    for x in (out.q_start, out.kv_len, out.positions, out.slots, out.free_left):
        x.fill_(-999)
    args = (dev32(cached), dev32(fresh), bs, dev32(stack), dev32([len(free)]), tt)
    torch.cuda.synchronize()
    for _ in range(2):  # the same inputs again write the same values
        got = ndq.kv_plan(*args, out=out, stream=stream)
    torch.cuda.synchronize()
    assert got.q_start.tolist() == want[0]
    assert got.kv_len.tolist() == want[1]
    assert got.positions.tolist() == want[2]
    assert got.slots.tolist() == want[3]
    assert got.free_left.tolist() == [want[4]]
    assert np.array_equal(tt.cpu().numpy(), want[5])


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("R,longest,most", [(1, 40, 1), (1, 3000, 5000), (7, 300, 70), (255, 900, 1), (2047, 500, 3),
                                            (2048, 100, 2), (2049, 90, 1), (5000, 60, 4)])
def test_plan(bs, R, longest, most):
    rng = np.random.default_rng(R * bs + most)
    cached = rng.integers(0, longest + 1, R).tolist()
    fresh = (rng.integers(0, most + 1, R) if most > 1 else np.ones(R, int)).tolist()
    need = sum(-(-(c + f) // bs) - -(-c // bs) for c, f in zip(cached, fresh))
    free = rng.permutation(1 << 20)[:need + 5].tolist()
    check_plan(cached, fresh, bs, free, (longest + most) // bs + 1, sum(fresh), capacity=need + 9)


def test_plan_edges():
    # requests without tokens, negative lengths, block edges, padding
    check_plan([0, 16, 15, 31, -5, 32], [0, 1, 1, 2, 3, 0], 16, list(range(100, 120)), 4, 20)
    check_plan([0] * 2100 + [5], [0] * 2100 + [40], 16, list(range(9)), 3, 40)   # a token far behind empty requests
    check_plan([3, 4], [50, 60], 16, [11, 12, 13], 10, 110)                       # the stack runs out
    check_plan([3, 4], [50, 60], 16, [], 10, 110, capacity=1)                     # it was empty
    check_plan([3, 4], [50, 60], 16, list(range(30)), 2, 110)                     # the table is too narrow
    check_plan([3, 4], [50, 60], 16, list(range(30)), 10, 60)                     # more tokens than the buffers
    check_plan([3, 4], [0, 0], 16, list(range(3)), 10, 0)


def test_plan_without_requests():
    out = ndq.kv_plan_buffers(0, 5)
    got = ndq.kv_plan(dev32([]), dev32([]), 16, dev32([1, 2]), dev32([2]), torch.empty(0, 4, **I32), out=out)
    assert got.q_start.tolist() == [0] and got.free_left.tolist() == [2] and got.slots.tolist() == [-1] * 5


# ---- append ----------------------------------------------------------------------


def encode(x, s, code):
    """Codes of binary32 x over s (0 where s is 0), as int8 bit patterns."""
    y = torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))
    if code == "int8":
        return torch.where(y.isnan(), 0.0, y.round().clamp(-127, 127)).to(torch.int8)
    c = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.int8)
    return torch.where(y.isnan(), torch.tensor(0x7f, dtype=torch.int8), c)


def append_ref(codes, scales, x, slots, bs, code):
    """On the CPU, run by run, in binary32 as defined."""
    codes, scales = codes.clone(), scales.clone()
    raw = codes.view(torch.int8)
    limit = codes.shape[0] * bs
    t = 0
    while t < len(slots):
        b = slots[t] // bs
        if slots[t] < 0 or slots[t] >= limit:
            t += 1
            continue
        e = t
        while e < len(slots) and slots[e] // bs == b:
            e += 1
        off = slots[t] % bs
        for h in range(codes.shape[1]):
            rows = x[t:e, h].float()
            mag = rows.abs()
            amax = mag[mag.isfinite()].max() if mag.isfinite().any() else torch.tensor(0.0)
            fresh = (amax / torch.tensor(QMAX[code])).clamp(2.0 ** -100, 2.0 ** 100) if amax > 0 else torch.tensor(0.0)
            old = scales[b, h] if off else torch.tensor(0.0)
            s = torch.maximum(old, fresh)
            if old > 0 and s > old:
                raw[b, h, :off] = encode(codes[b, h, :off].float() * old, s, code)
            for i in range(t, e):
                raw[b, h, slots[i] % bs] = encode(rows[i - t], s, code)
            scales[b, h] = s
        t = e
    return codes, scales


def random_cache(nb, heads, bs, D, code, seed, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(nb, heads, bs, D, device=DEV, generator=g) * size
    s = x.abs().amax((2, 3)) / QMAX[code]
    c = x / s[..., None, None]
    c = c.clamp(-448, 448).to(torch.float8_e4m3fn) if code == "e4m3" else c.round().to(torch.int8)
    return c, s


def same_codes(got, want):
    g, w = got.cpu().view(torch.int8), want.view(torch.int8)
    if got.dtype == torch.float8_e4m3fn:  # every NaN code is NaN
        g, w = (torch.where((z & 0x7f) == 0x7f, torch.tensor(0x7f, dtype=torch.int8), z) for z in (g, w))
    return torch.equal(g, w)


def check_append(x, v, slots, kc, ks, vc, vs, bs, code):
    wk = append_ref(kc.cpu(), ks.cpu(), x.cpu(), slots, bs, code)
    wv = append_ref(vc.cpu(), vs.cpu(), v.cpu(), slots, bs, code)
    cache = ndq.KvCache(kc, vc, ks, vs)
    ndq.kv_append(cache, x, v, torch.tensor(slots, dtype=torch.int64, device=DEV))
    torch.cuda.synchronize()
    for (c, s), gc, gs in ((wk, kc, ks), (wv, vc, vs)):
        assert torch.equal(gs.cpu().view(torch.int32), s.view(torch.int32))
        assert same_codes(gc, c)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,heads,bs", [(128, 8, 16), (64, 3, 32), (128, 1, 64), (64, 2, 128), (128, 2, 128)])
@pytest.mark.parametrize("spans", [[(3, 1)], [(0, 1), (15, 1), (16, 1), (31, 1)], [(0, 200), (7, 33), (120, 140), (9, 0), (64, 64)],
                                   [(i % 37, 1 + i % 5) for i in range(90)]])
def test_append(code, dtype, D, heads, bs, spans):
    # spans: (tokens before, new tokens) of each request
    g = torch.Generator(device=DEV).manual_seed(len(spans) * D + bs)
    blocks = [-(-(a + n) // bs) for a, n in spans]
    ids = np.random.default_rng(bs).permutation(sum(blocks) + 3)
    slots, at = [], 0
    for (a, n), nb in zip(spans, blocks):
        slots += [int(ids[at + p // bs]) * bs + p % bs for p in range(a, a + n)]
        at += nb
    T = len(slots)
    rows = torch.randn(T, 2, heads, D, device=DEV, generator=g) * torch.exp(torch.randn(T, 2, heads, 1, device=DEV, generator=g))
    rows = rows.to(dtype)
    kc, ks = random_cache(len(ids), heads, bs, D, code, 1)
    vc, vs = random_cache(len(ids), heads, bs, D, code, 2, 0.2)
    check_append(rows[:, 0], rows[:, 1], slots, kc, ks, vc, vs, bs, code)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_append_special_values(code):
    bs, heads, D = 16, 2, 128
    kc, ks = random_cache(8, heads, bs, D, code, 3)
    vc, vs = random_cache(8, heads, bs, D, code, 4)
    vs[5] = 0.0  # a block of zeros so far
    vc.view(torch.int8)[5] = 0
    k = torch.randn(40, heads, D, device=DEV).to(torch.bfloat16)
    v = torch.randn(40, heads, D, device=DEV).to(torch.bfloat16)
    k[0, 0, 5], k[1, 0, 7], k[2, 1, 0], k[3, 1, 1] = float("nan"), float("inf"), -float("inf"), 3e38
    k[20:], v[20:30] = 0.0, 0.0           # rows of zeros
    k[30, 0, 0] = 1e-38                   # a scale at its lower end
    v[31] = float("inf")                  # no finite value at all in its block's head 0 beside these
    slots = [2 * 16 + 5 + i for i in range(11)] + [-1, 8 * 16, 1 << 40] + [5 * 16 + 2 + i for i in range(6)] + \
            [7 * 16 + i for i in range(10)] + [3 * 16, 4 * 16] + [6 * 16 + 15] + [-7] * 7
    assert len(slots) == 40
    check_append(k, v, slots, kc, ks, vc, vs, bs, code)


@pytest.mark.parametrize("grow", [1.0 + 2.0 ** -10, 1.01, 3.0])
def test_append_rescales_every_code(grow):
    # a block whose earlier tokens hold every code there is (also -128, and the NaN codes), under a scale that grows
    bs, D = 16, 64
    for code in ("int8", "e4m3"):
        kc = torch.zeros(2, 1, bs, D, dtype=torch.int8, device=DEV)
        kc[1, 0, :4] = torch.arange(-128, 128, dtype=torch.int8, device=DEV).reshape(4, D)
        kc = kc.view(CODES[code])
        ks = torch.full((2, 1), 0.0123, device=DEV)
        x = torch.zeros(3, 1, D, device=DEV)
        x[1, 0, 7] = -0.0123 * QMAX[code] * grow
        x = x.to(torch.float16)
        check_append(x, x, [16 + 4, 16 + 5, 16 + 6], kc, ks, kc.clone(), ks.clone(), bs, code)


def test_append_rows_of_a_wider_buffer():
    bs, heads, D = 32, 4, 64
    buf = torch.randn(50, 3 * heads * D + 8, device=DEV).to(torch.float16)
    k = buf[:, 8:8 + heads * D].unflatten(1, (heads, D))
    v = buf[:, 8 + 2 * heads * D:].unflatten(1, (heads, D))
    kc, ks = random_cache(6, heads, bs, D, "e4m3", 5)
    vc, vs = random_cache(6, heads, bs, D, "e4m3", 6)
    check_append(k, v, [32 + i for i in range(50)], kc, ks, vc, vs, bs, "e4m3")


def test_append_beyond_32_bit_offsets():
    bs, heads, D = 128, 8, 128
    nb = (1 << 32) // (bs * heads * D) + 40  # the last blocks lie past 2^32 bytes
    kc, vc = (torch.zeros(nb, heads, bs, D, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(nb, heads, device=DEV) for _ in range(2))
    x = torch.randn(200, heads, D, device=DEV).to(torch.bfloat16)
    ndq.kv_append(ndq.KvCache(kc, vc, ks, vs), x, x, torch.arange(200, device=DEV) + (nb - 2) * bs)
    torch.cuda.synchronize()
    small_c, small_s = append_ref(torch.zeros(2, heads, bs, D, dtype=torch.int8), torch.zeros(2, heads), x.cpu(),
                                  list(range(200)), bs, "int8")
    for c, s in ((kc, ks), (vc, vs)):
        assert torch.equal(c[-2:].cpu(), small_c) and torch.equal(s[-2:].cpu(), small_s)
        assert int(c[:-2].count_nonzero()) == 0 and int(s[:-2].count_nonzero()) == 0


# ---- attention -------------------------------------------------------------------


def attend_ref(q, kc, ks, vc, vs, table, kv, start, bs, scale, window, dtype):
    """(out, bound, lse) in 64 bits."""
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    bound = torch.full_like(out, 1e-30)
    lse = torch.full((T, Hq), -float("inf"), dtype=torch.float64, device=DEV)
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    for r in range(len(kv)):
        n, L = start[r + 1] - start[r], kv[r]
        if n == 0 or L == 0:
            continue
        ids = torch.from_numpy(table[r, :-(-L // bs)].astype(np.int64)).to(DEV)
        there = ((ids >= 0) & (ids < kc.shape[0])).repeat_interleave(bs)[:L]
        ids = ids.clamp(0, kc.shape[0] - 1)
        pos = torch.arange(L - n, L, device=DEV)[:, None]
        col = torch.arange(L, device=DEV)[None, :]
        see = (col <= pos) & there[None, :]
        if window:
            see &= col > pos - window
        for h in range(Hkv):
            k = (kc[ids, h].double() * ks[ids, h].double()[:, None, None]).flatten(0, 1)[:L]
            v = (vc[ids, h].double() * vs[ids, h].double()[:, None, None]).flatten(0, 1)[:L]
            seen_any = see.any(0)
            k, v = torch.where(seen_any[:, None], k, 0.0), torch.where(seen_any[:, None], v, 0.0)
            for g in range(G):
                qq = q[start[r]:start[r + 1], h * G + g].double()
                e = torch.where(see, qq @ k.T * scale, -float("inf"))
                m = e.amax(1, keepdim=True).clamp(min=-1e300)
                p = torch.where(see, torch.exp(e - m), 0.0)
                z = p.sum(1, keepdim=True)
                some = z[:, 0] > 0
                p = torch.where(z > 0, p / z, 0.0)
                eps = 2.0 ** -20 * abs(scale) * torch.where(see, qq.abs() @ k.abs().T, 0.0).amax(1) + \
                    2.0 ** -21 * torch.where(see, e.abs(), 0.0).amax(1)
                o = p @ v
                spread = p @ v.abs()
                b = (2.0 ** -11 + 2.0 ** -13 + 4 * eps[:, None]) * spread + L * 2.0 ** -24 * v.abs().amax()
                out[start[r]:start[r + 1], h * G + g] = o
                bound[start[r]:start[r + 1], h * G + g] += b + unit * (o.abs() + b)
                lse[start[r]:start[r + 1], h * G + g] = torch.where(some, (m + z.log())[:, 0], -float("inf"))
    return out, bound, lse


def attend_case(kv, n, Hq, Hkv, D, bs, code, dtype, seed=0, extra=3, size=1.0):
    """Inputs with garbage wherever nothing may be read into the result: the
    unwritten ends of blocks hold NaN codes, unused table entries bad ids."""
    R = len(kv)
    rng = np.random.default_rng(seed + R)
    blocks = [-(-max(x, 0) // bs) for x in kv]
    nb = sum(blocks) + extra
    ids = rng.permutation(nb)
    width = max(blocks + [1]) + 1
    table = np.full((R, width), -1, dtype=np.int32)
    table[:, -1] = 1 << 30
    kc, ks = random_cache(nb, Hkv, bs, D, code, seed + 1)
    vc, vs = random_cache(nb, Hkv, bs, D, code, seed + 2, 0.3)
    at = 0
    for r, c in enumerate(blocks):
        table[r, :c] = ids[at:at + c]
        if kv[r] % bs:
            for x in (kc, vc):
                x.view(torch.int8)[int(ids[at + c - 1]), :, kv[r] % bs:] = 0x7f
        at += c
    for b in ids[at:]:
        kc.view(torch.int8)[int(b)] = 0x7f
        vc.view(torch.int8)[int(b)] = 0x7f
        ks[int(b)] = float("nan")
        vs[int(b)] = float("inf")
    start = np.concatenate([[0], np.cumsum(n)]).tolist()
    g = torch.Generator(device=DEV).manual_seed(seed + 7)
    q = (torch.randn(start[-1], Hq, D, device=DEV, generator=g) * size).to(dtype)
    return q, kc, ks, vc, vs, table, start


def check_attend(kv, n, Hq, Hkv, D, bs, code, dtype, window=0, seed=0, scale=None, size=1.0, with_start=True, stream=None):
    q, kc, ks, vc, vs, table, start = attend_case(kv, n, Hq, Hkv, D, bs, code, dtype, seed, size=size)
    scale = D ** -0.5 if scale is None else scale
    want, bound, lse_want = attend_ref(q, kc, ks, vc, vs, table, [max(x, 0) for x in kv], start, bs, scale, window, dtype)
    cache = ndq.KvCache(kc, vc, ks, vs)
    lse = torch.full(q.shape[:2], 99.0, device=DEV)
    ws = ndq.attention_workspace(len(kv), q.shape[0], Hq, cache)
    kw = dict(q_start=dev32(start) if with_start else None, max_q=max(n), scale=scale, window=window, workspace=ws)
    tt, kl = torch.from_numpy(table).to(DEV), dev32(kv)
    out = ndq.attention_kv8(q, cache, tt, kl, lse=lse, **kw)
    again = ndq.attention_kv8(q, cache, tt, kl, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits, with and without lse
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= bound).all(), (float((err / bound).max()), (err / bound).argmax())
    empty = torch.isinf(lse_want)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    tol = 2.0 ** -18 * (1 + lse_want[~empty].abs()) + 2.0 ** -18 * size * 40
    assert ((lse.double() - lse_want)[~empty].abs() <= tol).all()


HEADS = [(8, 8), (32, 8), (8, 1), (10, 2), (14, 2)]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", HEADS)
def test_attend_step(code, dtype, D, bs, heads):
    kv = [1, 0, 15, 16, 17, 127, 128, 129, 300, 1025, 5]
    check_attend(kv, [1] * len(kv), *heads, D, bs, code, dtype, with_start=False)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,n", [([7], [1]), ([1], [1]), ([9000], [1]), ([40000, 3], [1, 1]), ([300] * 200, [1] * 200),
                                  ([0] * 300 + [77] + [0] * 5, [1] * 306), ([5, 900, 33], [0, 1, 0])])
def test_attend_step_lengths(code, D, kv, n):
    check_attend(kv, n, 8, 2, D, 16, code, torch.bfloat16)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(32, 8), (4, 4), (16, 1), (10, 2), (40, 1)])
@pytest.mark.parametrize("kv,n", [([100, 7, 3000, 16], [2, 3, 4, 1]), ([5, 64, 130], [5, 8, 2]), ([3, 20, 0], [5, 20, 2]),
                                  ([700, 33], [17, 33]), ([513, 256, 1], [200, 256, 1])])
def test_attend_several_queries(code, D, heads, kv, n):
    # (a request with more queries than tokens: its first queries see nothing)
    check_attend(kv, n, *heads, D, 32, code, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window", [1, 5, 16, 100, 1000])
@pytest.mark.parametrize("kv,n", [([1000, 17, 3], [1, 1, 1]), ([1000, 70, 40], [4, 3, 2]), ([1100, 300], [130, 300])])
def test_attend_window(dtype, window, kv, n):
    check_attend(kv, n, 8, 2, 128, 16, "e4m3", dtype, window=window)


@pytest.mark.parametrize("n", [1, 6, 150])
def test_attend_large_and_small_magnitudes(n):
    # queries of 1000 and of 1e-6, sharp softmax, negative and zero scale
    check_attend([600, 200], [n, n], 8, 2, 128, 16, "e4m3", torch.bfloat16, size=1000.0, scale=1e-4)
    check_attend([600, 200], [n, n], 8, 2, 128, 16, "int8", torch.float16, size=1e-6)
    check_attend([600, 200], [n, n], 8, 2, 128, 16, "e4m3", torch.bfloat16, scale=3.0)
    check_attend([600, 200], [n, n], 8, 2, 64, 16, "e4m3", torch.bfloat16, scale=-0.2)
    check_attend([600, 200], [n, n], 8, 2, 64, 16, "int8", torch.bfloat16, scale=0.0)


@pytest.mark.parametrize("n", [1, 4, 140])
def test_attend_scales_of_blocks_far_apart(n):
    bs, D = 16, 128
    kv = [400, 1200]
    q, kc, ks, vc, vs, table, start = attend_case(kv, [n, n], 8, 2, D, bs, "e4m3", torch.bfloat16, 11)
    g = torch.Generator(device=DEV).manual_seed(5)
    vs *= torch.exp2(torch.randint(-40, 41, vs.shape, device=DEV, generator=g).float())
    vs[::7] = 0.0
    want, bound, _ = attend_ref(q, kc, ks, vc, vs, table, kv, start, bs, D ** -0.5, 0, torch.bfloat16)
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start))
    err = (out.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("n", [1, 3, 90])
def test_attend_missing_blocks_and_short_tables(n):
    bs, D = 16, 64
    kv = [500, 333]
    q, kc, ks, vc, vs, table, start = attend_case(kv, [n, n], 4, 2, D, bs, "int8", torch.bfloat16, 21)
    table[0, 3:9] = -1
    table[1, 0] = 1 << 29
    want, bound, _ = attend_ref(q, kc, ks, vc, vs, table, kv, start, bs, D ** -0.5, 0, torch.bfloat16)
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start))
    assert ((out.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("n", [4, 200])
def test_attend_nan_reaches_only_the_rows_that_see_it(n):
    bs, D, kv = 16, 128, [600]
    for where in ("k", "v"):
        q, kc, ks, vc, vs, table, start = attend_case(kv, [n], 8, 2, D, bs, "e4m3", torch.bfloat16, 31)
        tok = 600 - n + n // 2  # seen by the queries from n // 2 on
        x = kc if where == "k" else vc
        x.view(torch.int8)[int(table[0, tok // bs]), 1, tok % bs, 17] = 0x7f
        out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv),
                                q_start=dev32(start))
        nan = out.isnan()
        expect = torch.zeros_like(nan)
        if where == "k":
            expect[n // 2:, 4:] = True
        else:
            expect[n // 2:, 4:, 17] = True
        assert torch.equal(nan, expect)


@pytest.mark.parametrize("n", [1, 120])
def test_attend_beyond_32_bit_offsets(n):
    bs, heads, D, kv = 128, 8, 128, [900]
    nb = (1 << 32) // (bs * heads * D) + 40
    small = attend_case(kv, [n], 8, heads, D, bs, "int8", torch.bfloat16, 41, extra=0)
    q, kc, ks, vc, vs, table, start = small
    big = [torch.zeros(nb, heads, bs, D, dtype=torch.int8, device=DEV) for _ in range(2)]
    scale = [torch.zeros(nb, heads, device=DEV) for _ in range(2)]
    m = kc.shape[0]
    for dst, src in zip(big + scale, (kc, vc, ks, vs)):
        dst[nb - m:] = src
    far = np.where((table >= 0) & (table < m), table + nb - m, table).astype(np.int32)
    a = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start))
    b = ndq.attention_kv8(q, ndq.KvCache(big[0], big[1], *scale), torch.from_numpy(far).to(DEV), dev32(kv), q_start=dev32(start))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_attend_strided_queries_on_another_stream():
    kv, n, D, bs = [300, 41], [2, 60], 128, 32
    q, kc, ks, vc, vs, table, start = attend_case(kv, n, 8, 2, D, bs, "e4m3", torch.bfloat16, 51)
    cache, tt, kl, qs = ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), dev32(start)
    want = ndq.attention_kv8(q, cache, tt, kl, q_start=qs)
    wide = torch.full((q.shape[0], 12 * D + 8), 9.0, dtype=q.dtype, device=DEV)
    wide[:, 8:8 + 8 * D] = q.flatten(1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.empty_like(q)
    ws = ndq.attention_workspace(2, q.shape[0], 8, cache)
    torch.cuda.synchronize()
    ndq.attention_kv8(wide[:, 8:8 + 8 * D].unflatten(1, (8, D)), cache, tt, kl, q_start=qs, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_attend_lengths_outside_the_buffers_are_cut():
    # (device-side lengths are not checked by the host: they must not lead out of the buffers)
    kv, n, D, bs = [300, 41], [2, 3], 128, 16
    q, kc, ks, vc, vs, table, start = attend_case(kv, n, 8, 2, D, bs, "e4m3", torch.bfloat16, 61)
    cache, tt = ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV)
    guard = torch.full((q.shape[0] + 4, 8, D), 5.0, dtype=q.dtype, device=DEV)
    out = guard[2:-2]
    for lens, starts in (([1 << 30, -4], [0, 2, 5]), ([300, 41], [-3, 2, 900]), ([300, 41], [4, 1, 2]), ([300, 41], [0, 5, 5])):
        ndq.attention_kv8(q, cache, tt, dev32(lens), q_start=dev32(starts), out=out)
    torch.cuda.synchronize()
    assert (guard[:2] == 5).all() and (guard[-2:] == 5).all()


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("n", [1, 4, 140])
def test_attend_zero_blocks_beside_small_values(code, n):
    # blocks of values 0 (scale 0) take nothing from the weights of small values
    bs, D = 16, 128
    kv = [400, 1200]
    q, kc, ks, vc, vs, table, start = attend_case(kv, [n, n], 8, 2, D, bs, code, torch.bfloat16, 12)
    vs *= 2.0 ** -14
    vs[::5] = 0.0
    want, bound, _ = attend_ref(q, kc, ks, vc, vs, table, kv, start, bs, D ** -0.5, 0, torch.bfloat16)
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), q_start=dev32(start))
    err = (out.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("scale", [1e6, -1e6, 1e9])
@pytest.mark.parametrize("n", [1, 6, 150])
def test_attend_scores_whose_roundings_pass_the_exponents(n, scale):
    # scores 1e7 and more apart: the largest takes all, in every kernel, and
    # its value (7 bits) is exact
    bs, D, kv, H = 16, 128, 250, 2
    nb = -(-kv // bs)
    key = torch.from_numpy(np.random.default_rng(3).permutation(kv) - 125)
    kc, vc = (torch.zeros(nb, H, bs, D, dtype=torch.int8) for _ in range(2))
    g = torch.Generator().manual_seed(3)
    v = torch.randint(-127, 128, (kv, H, D), generator=g)
    for j in range(kv):
        kc[j // bs, :, j % bs] = key[j]
        vc[j // bs, :, j % bs] = v[j].to(torch.int8)
    cache = ndq.KvCache(kc.to(DEV), vc.to(DEV), torch.ones(nb, H, device=DEV), torch.full((nb, H), 2.0 ** -6, device=DEV))
    q = torch.ones(n, 4 * H, D, dtype=torch.bfloat16, device=DEV)
    table = torch.arange(nb, dtype=torch.int32, device=DEV)[None]
    out = ndq.attention_kv8(q, cache, table, dev32([kv]), q_start=dev32([0, n]), scale=scale).cpu()
    for i in range(n):
        seen = key[:kv - n + i + 1] * (1 if scale > 0 else -1)
        want = v[int(seen.argmax())].to(torch.float32).repeat_interleave(4, 0) * 2.0 ** -6
        assert torch.equal(out[i].float(), want), i


@pytest.mark.parametrize("n", [1, 5, 150])
def test_attend_nan_queries_that_see_nothing(n):
    q, kc, ks, vc, vs, table, start = attend_case([400, 300], [n, n], 8, 2, 128, 16, "e4m3", torch.bfloat16, 13)
    q[n:] = float("nan")
    table[1] = -1
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = ndq.attention_kv8(q, ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32([400, 300]),
                            q_start=dev32(start), lse=lse)
    assert torch.isfinite(out).all() and int(out[n:].count_nonzero()) == 0
    assert torch.isfinite(lse[:n]).all() and (lse[n:] == -float("inf")).all()


# ---- adapters ----------------------------------------------------------------------


def check_lora(M, K, N, nA, rank, dtype, index, ranks=None, seed=0, inplace=False, garbage=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, device=DEV, generator=g).to(torch.bfloat16)
    a = (torch.randn(nA, rank, K, device=DEV, generator=g) / max(K, 1) ** 0.5).to(torch.bfloat16)
    b = torch.randn(nA, N, rank, device=DEV, generator=g).to(torch.bfloat16)
    ranks = [rank if i % 2 else max(0, rank - 3) for i in range(nA)] if ranks is None else ranks
    scales = torch.rand(nA, device=DEV, generator=g) + 0.5
    base = torch.randn(M, N, device=DEV, generator=g).to(dtype)
    if garbage:  # beyond an adapter's rank
        for i, r in enumerate(ranks):
            a[i, r:] = float("nan")
            b[i, :, r:] = float("inf")
    want, bound = base.double(), torch.zeros(M, N, dtype=torch.float64, device=DEV)
    ix = torch.tensor(index, dtype=torch.int64, device=DEV)
    for i, r in enumerate(ranks):
        rows = (ix == i).nonzero()[:, 0]
        xa, aa, bb = x[rows].double(), a[i, :r].double(), b[i, :, :r].double()
        s = float(scales[i])
        t = xa @ aa.T * s
        want[rows] += t @ bb.T
        bound[rows] += (K + 16) * 2.0 ** -23 * (xa.abs() @ aa.abs().T * s) @ bb.abs().T + (rank + 16) * 2.0 ** -23 * t.abs() @ bb.abs().T
    bound += (2.0 ** -23 if dtype == torch.float32 else 2.0 ** -8) * (want.abs() + bound) + 1e-30
    out = base if inplace else None
    ws = ndq.lora_workspace(M, nA, rank, K)
    ws.fill_(255)
    y = ndq.lora_add(x, a, b, dev32(ranks), scales, dev32(index), base, out=out, workspace=ws)
    torch.cuda.synchronize()
    err = (y.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())
    if not inplace:
        again = ndq.lora_add(x, a, b, dev32(ranks), scales, dev32(index), base, workspace=ws)
        assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,N,nA,rank", [(1, 4096, 1024, 1, 8), (1, 64, 7, 2, 1), (3, 1000, 1032, 2, 16), (17, 520, 300, 5, 24),
                                           (61, 4096, 512, 48, 16), (130, 1024, 4099, 3, 64), (300, 333, 129, 4, 5),
                                           (700, 2048, 640, 7, 128), (64, 14336, 256, 64, 8), (1025, 256, 512, 2, 33)])
def test_lora(dtype, M, K, N, nA, rank):
    rng = np.random.default_rng(M + K)
    runs = np.sort(rng.integers(-1, nA, M)).tolist()       # adjacent rows
    check_lora(M, K, N, nA, rank, dtype, runs)
    check_lora(M, K, N, nA, rank, dtype, rng.permutation(runs).tolist(), seed=1)


def test_lora_edges():
    f32 = torch.float32
    check_lora(5, 256, 64, 2, 8, f32, [-1, 2, 99, -5, 0])             # indexes outside the adapters
    check_lora(40, 256, 64, 2, 8, f32, [-1] * 40)                      # nothing to add
    check_lora(40, 256, 64, 2, 8, f32, [1] * 40, ranks=[8, 0])         # an adapter of rank 0
    check_lora(9, 0, 64, 2, 8, f32, [1] * 9, garbage=False)            # empty sums
    check_lora(200, 512, 512, 3, 16, f32, [i % 3 for i in range(200)], inplace=True)
    check_lora(200, 512, 512, 3, 16, torch.bfloat16, [i // 70 for i in range(200)], inplace=True)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, 8, device=DEV)
    y = ndq.lora_add(x, torch.empty(1, 4, 64, dtype=torch.bfloat16, device=DEV), torch.empty(1, 8, 4, dtype=torch.bfloat16, device=DEV),
                     dev32([4]), torch.ones(1, device=DEV), dev32([]), none)
    assert y.shape == (0, 8)


def test_lora_unaligned_buffers():
    M, K, N, nA, rank = 33, 264, 130, 3, 12
    g = torch.Generator(device=DEV).manual_seed(3)

    def off(shape, dtype, scale=1.0):
        n = int(np.prod(shape))
        buf = torch.zeros(n + 3, dtype=dtype, device=DEV)
        buf[1:1 + n] = (torch.randn(n, device=DEV, generator=g) * scale).to(dtype)
        return buf[1:1 + n].view(shape)

    bf = torch.bfloat16
    x, a, b, base = off((M, K), bf), off((nA, rank, K), bf, 0.1), off((nA, N, rank), bf), off((M, N), torch.float32)
    index = dev32([i % 4 - 1 for i in range(M)])
    ranks, scales = dev32([12, 7, 12]), torch.tensor([1.0, 2.0, 0.5], device=DEV)
    y = ndq.lora_add(x, a, b, ranks, scales, index, base)
    z = ndq.lora_add(*(t.clone() for t in (x, a, b)), ranks, scales, index, base.clone())
    assert (y - z).abs().max() <= 2.0 ** -14 * z.abs().max()
    want = base.double()
    for i, r in enumerate([12, 7, 12]):
        rows = (index == i).nonzero()[:, 0]
        want[rows] += (x[rows].double() @ a[i, :r].double().T * float(scales[i])) @ b[i, :, :r].double().T
    assert ((y.double() - want).abs() <= 2.0 ** -14 * want.abs().max()).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [3, 200])
def test_lora_infinite_inputs(M, dtype):
    # of rank 1, so that no two infinities meet: y is infinite with the sign of the product, NaN for NaN
    g = torch.Generator(device=DEV).manual_seed(9)
    K, N = 256, 512
    x = torch.randn(M, K, device=DEV, generator=g).to(torch.bfloat16)
    x[0, 5], x[1, 7], x[2, 9] = float("inf"), -float("inf"), float("nan")
    a = torch.randn(1, 8, K, device=DEV, generator=g).to(torch.bfloat16)
    b = torch.randn(1, N, 8, device=DEV, generator=g).to(torch.bfloat16)
    a[a == 0], b[b == 0] = 1.0, 1.0
    base = torch.randn(M, N, device=DEV, generator=g).to(dtype)
    y = ndq.lora_add(x, a, b, dev32([1]), torch.ones(1, device=DEV), dev32([0] * M), base)
    want = base.double() + (x.double() @ a[0, :1].double().T) @ b[0, :, :1].double().T
    odd = ~torch.isfinite(want)
    assert odd[:3].all() and not odd[3:].any()
    assert torch.equal(y[:2].double(), want[:2]) and y[2].isnan().all()
    assert torch.isfinite(y[3:]).all()
