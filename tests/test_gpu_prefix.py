"""GPU tests of attention behind shared prefixes: against the definition in 64
bits, which knows of no groups, within the bound of attention over the cache
(its derivation stands there).  Joining the two parts adds one binary32 product
and sum a part and row to numerator and denominator, below 2^-20 of either,
which the bound's 2^-13 holds.

The tables are wide enough that every case with a group of two and requests of
few rows on average takes the kernels of shared prefixes (see the call's
documentation); test_narrow_tables_and_many_rows has those that do not."""
import numpy as np
import pytest
import torch

from test_gpu_serving import DEV, attend_ref, dev32, random_cache

pytestmark = pytest.mark.gpu

import quantized_weight_block_gb300 as ndq  # noqa: E402

BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _no_device_fault():
    yield
    assert ndq.get_device_fault() == 0


class Case:
    """Requests in groups (sizes), a shared prefix each (0: none), tokens of
    their own and new ones; requests after the last group share nothing.
    Garbage lies wherever nothing may be read into the result."""

    def __init__(self, sizes, prefix, own, fresh, Hq, Hkv, D, bs, code="e4m3", dtype=BF, seed=0, size=1.0, first=0, vscale=0.3, wide=True):
        R = len(own)
        rng = np.random.default_rng(seed + R)
        self.bs, self.dtype, self.D, self.Hq, self.fresh, self.prefix, self.code = bs, dtype, D, Hq, fresh, prefix, code
        self.groups = first + np.concatenate([[0], np.cumsum(sizes)])
        shared = [0] * R  # blocks
        of = [-1] * R
        for g, p in enumerate(prefix):
            for r in range(self.groups[g], self.groups[g + 1]):
                shared[r], of[r] = p // bs, g
        base = [prefix[of[r]] if of[r] >= 0 else 0 for r in range(R)]
        self.kv = [base[r] + own[r] + fresh[r] for r in range(R)]
        blocks = [-(-n // bs) for n in self.kv]
        nb = sum(p // bs for p in prefix) + sum(b - s for b, s in zip(blocks, shared)) + 4
        ids = rng.permutation(nb)
        width = max(blocks + [1]) + 1
        if wide and R > len(sizes):
            width = max(width, int(1.3e8) // ((R - len(sizes)) * bs * 2 * D * Hkv) + 1)
        self.table = np.full((R, width), -1, dtype=np.int32)
        self.table[:, -1] = 1 << 30
        self.kc, self.ks = random_cache(nb, Hkv, bs, D, code, seed + 1)
        self.vc, self.vs = random_cache(nb, Hkv, bs, D, code, seed + 2, vscale)
        self.width = max(blocks + [1])  # columns in use
        at, common = 0, []
        for p in prefix:
            common.append(ids[at:at + p // bs])
            at += p // bs
        for r in range(R):
            if of[r] >= 0:
                self.table[r, :shared[r]] = common[of[r]]
            n = blocks[r] - shared[r]
            self.table[r, shared[r]:blocks[r]] = ids[at:at + n]
            at += n
            if self.kv[r] % bs:
                for x in (self.kc, self.vc):
                    x.view(torch.int8)[int(self.table[r, blocks[r] - 1]), :, self.kv[r] % bs:] = 0x7f
        for b in ids[at:]:
            for x in (self.kc, self.vc):
                x.view(torch.int8)[int(b)] = 0x7f
            self.ks[int(b)], self.vs[int(b)] = float("nan"), float("inf")
        self.start = np.concatenate([[0], np.cumsum(fresh)]).tolist()
        g = torch.Generator(device=DEV).manual_seed(seed + 7)
        self.q = (torch.randn(self.start[-1], Hq, D, device=DEV, generator=g) * size).to(dtype)

    def cache(self):
        return ndq.KvCache(self.kc, self.vc, self.ks, self.vs)

    def args(self):
        return dict(block_table=torch.from_numpy(self.table).to(DEV), kv_len=dev32(self.kv), group_start=dev32(self.groups),
                    prefix_len=dev32(self.prefix))

    def reference(self, scale=None, window=0):
        return attend_ref(self.q, self.kc, self.ks, self.vc, self.vs, self.table, self.kv, self.start, self.bs,
                          self.D ** -0.5 if scale is None else scale, window, self.dtype)

    def check(self, scale=None, window=0, with_start=True, size=1.0):
        want, bound, lse_want = self.reference(scale, window)
        cache = self.cache()
        lse = torch.full(self.q.shape[:2], 99.0, device=DEV)
        ws = ndq.attention_prefix_workspace(cache, self.q.shape[0], self.Hq)
        kw = dict(q_start=dev32(self.start) if with_start else None, max_q=max(self.fresh), scale=scale, window=window, workspace=ws)
        args = self.args()
        out = ndq.attention_prefix_kv8(self.q, cache, lse=lse, **args, **kw)
        again = ndq.attention_prefix_kv8(self.q, cache, **args, **kw)
        torch.cuda.synchronize()
        assert int(ws[:4096].count_nonzero()) == 0
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits, with and without lse
        assert torch.isfinite(out).all()
        err = (out.double() - want).abs()
        assert (err <= bound).all(), (float((err / bound).max()), (err > bound).nonzero()[:4].tolist())
        empty = torch.isinf(lse_want)
        assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
        tol = 2.0 ** -18 * (1 + lse_want[~empty].abs()) + 2.0 ** -18 * size * 40
        assert ((lse.double() - lse_want)[~empty].abs() <= tol).all()
        return out


def own_lengths(R, most, seed=0):
    return np.random.default_rng(seed).integers(0, most + 1, R).tolist()


HEADS = [(8, 8), (32, 8), (8, 1), (10, 2), (14, 2)]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", HEADS)
def test_step(code, dtype, D, bs, heads):
    # groups of 5, 1 and 3 behind 700, 130 and 1000 tokens, two requests of their own
    Case([5, 1, 3], [700, 130, 1000], [0, 1, 15, 16, 300, 2, 127, 128, 129, 50, 400], [1] * 11, *heads, D, bs, code, dtype).check(with_start=False)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sizes,prefix,own", [
    ([1], [16], [0]), ([1], [5000], [3]), ([2], [15], [3, 4]), ([2], [0], [3, 400]), ([3], [40000], [1, 0, 900]),
    ([70], [2500], own_lengths(70, 300)), ([300], [1000], own_lengths(300, 40)), ([1] * 40, list(range(3, 1603, 40)), own_lengths(40, 60)),
    ([64, 64, 2], [300, 3000, 12000], own_lengths(130, 90)), ([0, 5, 0, 2], [100, 700, 900, 50], own_lengths(7, 100))])
def test_step_groups_and_lengths(D, sizes, prefix, own):
    Case(sizes, prefix, own, [1] * len(own), 8, 2, D, 16).check()


@pytest.mark.parametrize("groups,each,prefix", [(33, 2, 300), (40, 5, 700), (600, 3, 150)])
@pytest.mark.parametrize("prompts", [False, True])
def test_many_groups(groups, each, prefix, prompts):
    # (more than 32 groups are planned by the whole block, more than 512 several to a thread; prefixes of 0 among them)
    R = groups * each
    lengths = [(37 * g) % prefix for g in range(groups)]
    fresh = [40 if prompts and r % 50 == 7 else 1 for r in range(R)]
    Case([each] * groups, lengths, own_lengths(R, 60), fresh, 8, 2, 64, 16, "int8").check()


@pytest.mark.parametrize("heads", [(32, 8), (4, 4), (16, 1), (10, 2), (40, 1)])
@pytest.mark.parametrize("code,D", [("e4m3", 128), ("int8", 64)])
@pytest.mark.parametrize("sizes,prefix,own,fresh", [
    ([4], [500], [9, 0, 100, 33], [2, 3, 4, 1]), ([2, 2], [300, 1111], [0, 5, 64, 700], [5, 0, 8, 1]),
    ([3], [2000], [5, 300, 0], [17, 40, 33]), ([6, 1], [640, 90], [0, 0, 1000, 3, 20, 400, 77], [60, 1, 2, 1, 1, 0, 3]),
    ([9], [1500], own_lengths(9, 500, 9), [1, 1, 130, 2, 1, 1, 1, 3, 1])])
def test_several_queries(heads, code, D, sizes, prefix, own, fresh):
    Case(sizes, prefix, own, fresh, *heads, D, 32, code).check()


@pytest.mark.parametrize("wide,fresh", [(False, [1, 1, 1, 1]), (False, [5, 1, 40, 2]), (True, [300, 1, 500, 40]), (True, [130] * 4)])
@pytest.mark.parametrize("window", [0, 100])
def test_narrow_tables_and_many_rows(wide, fresh, window):
    Case([3], [640], [0, 70, 300, 5], fresh, 32, 8, 128, 16, wide=wide).check(window=window)


@pytest.mark.parametrize("window", [1, 16, 100, 700, 5000])
@pytest.mark.parametrize("fresh", [1, 5, 30])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_window(window, fresh, dtype):
    # (windows that end in the prefix, in the own tokens, and behind nothing of either)
    Case([4, 2], [1000, 333], [0, 300, 7, 900, 64, 1], [fresh] * 6, 8, 2, 128, 16, "e4m3", dtype).check(window=window)


@pytest.mark.parametrize("fresh", [1, 3, 30])
def test_queries_inside_the_prefix(fresh):
    # a prefix said to be longer than some requests' tokens: every query sees up to itself
    c = Case([3], [1000], [100, 60, 0], [fresh] * 3, 8, 2, 128, 16)
    c.kv[1], c.kv[2] = 517 + fresh, max(fresh, 20)
    c.check()
    c.prefix = [1 << 30]  # beyond the table: what is there is shared
    c.table[:, -1] = -1
    c.kv = [c.kv[0]] * 3
    c.table[:] = c.table[0]
    c.check()


@pytest.mark.parametrize("first", [1, 2])
def test_requests_before_the_first_group(first):
    c = Case([3], [600], own_lengths(5, 200, 3), [2] * 5, 8, 2, 64, 16, first=first)
    c.check()


@pytest.mark.parametrize("n", [1, 6, 30])
def test_large_and_small_magnitudes(n):
    for kw, chk in ((dict(size=1000.0), dict(scale=1e-4, size=1000.0)), (dict(size=1e-6, code="int8", dtype=F16), dict(size=1e-6)), (dict(), dict(scale=3.0)),
                    (dict(D=64), dict(scale=-0.2)), (dict(D=64, code="int8"), dict(scale=0.0))):
        c = dict(Hq=8, Hkv=2, D=128, bs=16) | kw
        Case([2, 1], [600, 200], [40, 0, 200], [n] * 3, **c).check(**chk)


@pytest.mark.parametrize("n", [1, 4, 31])
def test_scales_of_blocks_far_apart(n):
    c = Case([3], [900], [400, 10, 700], [n] * 3, 8, 2, 128, 16, seed=11)
    g = torch.Generator(device=DEV).manual_seed(5)
    c.vs *= torch.exp2(torch.randint(-40, 41, c.vs.shape, device=DEV, generator=g).float())
    c.vs[::7] = 0.0
    want, bound, _ = c.reference()
    out = ndq.attention_prefix_kv8(c.q, c.cache(), q_start=dev32(c.start), **c.args())
    err = (out.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("spread", [90, -90])
@pytest.mark.parametrize("n", [1, 4, 31])
def test_a_part_of_far_larger_values(n, spread):
    # V of the prefix 2^90 above or below V of the own tokens
    c = Case([3], [640], [100, 10, 300], [n] * 3, 8, 2, 128, 16, seed=12)
    own = torch.ones(c.vs.shape[0], dtype=torch.bool)
    own[c.table[0, :40].astype(np.int64)] = False
    c.vs[own.to(DEV)] *= 2.0 ** spread
    want, bound, _ = c.reference()
    out = ndq.attention_prefix_kv8(c.q, c.cache(), q_start=dev32(c.start), **c.args())
    if spread > 0:
        ok = torch.isfinite(want.to(BF))
        assert ((out.double() - want).abs() <= bound)[ok].all()
    else:
        err = (out.double() - want).abs()
        assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("n", [1, 3, 60])
def test_missing_blocks_and_short_tables(n):
    c = Case([2], [500], [333, 4], [n] * 2, 4, 2, 64, 16, "int8", seed=21)
    c.table[:, 3:9] = -1
    c.table[:, 20] = 1 << 29
    c.table[0, 35] = -1
    want, bound, _ = c.reference()
    out = ndq.attention_prefix_kv8(c.q, c.cache(), q_start=dev32(c.start), **c.args())
    assert ((out.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("n", [1, 4, 30])
@pytest.mark.parametrize("where", ["k", "v"])
def test_nan_reaches_the_rows_that_see_it(n, where):
    c = Case([3, 1], [320, 100], [50, 0, 200, 7], [n] * 4, 8, 2, 128, 16, seed=31)
    c.kv[1] = 200 + n  # this request's queries sit inside the prefix, after its token 200
    x = c.kc if where == "k" else c.vc
    tok = 210
    x.view(torch.int8)[int(c.table[0, tok // 16]), 1, tok % 16, 17] = 0x7f
    out = ndq.attention_prefix_kv8(c.q, c.cache(), q_start=dev32(c.start), **c.args())
    expect = torch.zeros_like(out, dtype=torch.bool)
    heads, pos = slice(4, 8), slice(None) if where == "k" else slice(17, 18)
    expect[:n, heads, pos] = True
    expect[2 * n:3 * n, heads, pos] = True
    if n > 10:
        expect[n + 10:2 * n, heads, pos] = True  # (query i of request 1 sits at 200 + i)
    assert torch.equal(out.isnan(), expect)


def test_unseen_rows_of_the_other_requests_have_no_influence():
    # NaN queries of one request stay there, and what a request does not see is not read into it
    c = Case([4], [512], [30, 0, 90, 5], [1] * 4, 8, 2, 128, 16, seed=41)
    args = c.args()
    want = ndq.attention_prefix_kv8(c.q, c.cache(), **args)
    c.q[2] = float("nan")
    got = ndq.attention_prefix_kv8(c.q, c.cache(), **args)
    keep = torch.tensor([0, 1, 3], device=DEV)
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16)) and got[2].isnan().all()


@pytest.mark.parametrize("n", [1, 30])
def test_a_table_without_blocks(n):
    c = Case([2], [64], [20, 4], [n] * 2, 8, 2, 64, 16, seed=42)
    c.table[:] = -1
    lse = torch.zeros(c.q.shape[:2], device=DEV)
    out = ndq.attention_prefix_kv8(c.q, c.cache(), q_start=dev32(c.start), lse=lse, **c.args())
    assert not out.any() and (lse == -float("inf")).all()


@pytest.mark.parametrize("n", [1, 100])
def test_beyond_32_bit_offsets(n):
    bs, heads, D = 128, 8, 128
    c = Case([2], [600], [300, 9], [n] * 2, 8, heads, D, bs, "int8", seed=51)
    nb, m = (1 << 32) // (bs * heads * D) + 40, c.kc.shape[0]
    big = [torch.zeros(nb, heads, bs, D, dtype=torch.int8, device=DEV) for _ in range(2)]
    scale = [torch.zeros(nb, heads, device=DEV) for _ in range(2)]
    for dst, src in zip(big + scale, (c.kc, c.vc, c.ks, c.vs)):
        dst[nb - m:] = src
    args = c.args()
    a = ndq.attention_prefix_kv8(c.q, c.cache(), q_start=dev32(c.start), **args)
    args["block_table"] = torch.from_numpy(np.where((c.table >= 0) & (c.table < m), c.table + nb - m, c.table).astype(np.int32)).to(DEV)
    b = ndq.attention_prefix_kv8(c.q, ndq.KvCache(*big, *scale), q_start=dev32(c.start), **args)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_queries_beyond_max_q_are_left_out():
    c = Case([3], [400], [10, 0, 50], [6, 2, 40], 8, 2, 128, 16, seed=61)
    want, bound, _ = c.reference()
    guard = torch.full_like(c.q, 5.0)
    out = ndq.attention_prefix_kv8(c.q, c.cache(), q_start=dev32(c.start), max_q=3, out=guard, **c.args())
    done = torch.zeros(c.q.shape[0], dtype=torch.bool, device=DEV)
    for a, b in zip(c.start, c.start[1:]):
        done[a:min(b, a + 3)] = True
    assert (out[~done] == 5).all()
    assert ((out.double() - want).abs() <= bound)[done].all()


def test_device_arrays_outside_the_buffers_lead_nowhere():
    # (device-side lengths and groups are not checked by the host: they must not lead out of the buffers)
    c = Case([2], [200], [300, 41], [2, 3], 8, 2, 128, 16, seed=62)
    cache, table = c.cache(), torch.from_numpy(c.table).to(DEV)
    guard = torch.full((c.q.shape[0] + 4, 8, 128), 5.0, dtype=c.q.dtype, device=DEV)
    out = guard[2:-2]
    ws = ndq.attention_prefix_workspace(cache, 5, 8)
    ws[4096:] = 0xff
    for lens in (c.kv, [1 << 30, -4]):
        for starts in (c.start, [-3, 2, 900], [4, 1, 2], [0, 5, 5]):
            for groups, prefix in (([0, 2], [200]), ([-5, 900], [1 << 30]), ([2, 0], [64]), ([1, 1, 0, 2], [64, -3, 128]), ([0, 1, 1, 9], [16, 0, 300])):
                ndq.attention_prefix_kv8(c.q, cache, table, dev32(lens), dev32(groups), dev32(prefix), q_start=dev32(starts), out=out, workspace=ws)
    torch.cuda.synchronize()
    assert (guard[:2] == 5).all() and (guard[-2:] == 5).all()
    assert int(ws[:4096].count_nonzero()) == 0


@pytest.mark.parametrize("fresh", [1, 30])
def test_captured_and_replayed_with_other_lengths(fresh):
    # one graph, its arrays rewritten between replays: other groups, lengths and queries
    T = 6 * fresh
    cases = [Case(s, p, own_lengths(6, 150, i), [fresh] * 6, 8, 2, 128, 16, seed=70 + i)
             for i, (s, p) in enumerate((([6, 0], [900, 0]), ([2, 4], [100, 640]), ([1, 3], [2000, 33])))]
    nb, width = max(c.kc.shape[0] for c in cases), max(c.table.shape[1] for c in cases)
    kc, vc = (torch.zeros(nb, 2, 16, 128, dtype=cases[0].kc.dtype, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(nb, 2, device=DEV) for _ in range(2))
    cache = ndq.KvCache(kc, vc, ks, vs)
    i32 = dict(dtype=torch.int32, device=DEV)
    table, kv, gs, pl = torch.full((6, width), -1, **i32), torch.zeros(6, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32)
    q, out, ws = torch.zeros_like(cases[0].q), torch.zeros_like(cases[0].q), ndq.attention_prefix_workspace(cache, T, 8)
    start = dev32(np.arange(7) * fresh)

    def call():
        ndq.attention_prefix_kv8(q, cache, table, kv, gs, pl, q_start=start, max_q=fresh, out=out, workspace=ws)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in cases + cases[:1]:
        m = c.kc.shape[0]
        for dst, src in ((kc.view(torch.int8), c.kc.view(torch.int8)), (vc.view(torch.int8), c.vc.view(torch.int8)), (ks, c.ks), (vs, c.vs)):
            dst[:m] = src
        table.fill_(-1)
        table[:, :c.table.shape[1]] = torch.from_numpy(c.table).to(DEV)
        kv.copy_(dev32(c.kv))
        gs.copy_(dev32(c.groups))
        pl.copy_(dev32(c.prefix))
        q.copy_(c.q)
        graph.replay()
        torch.cuda.synchronize()
        want, bound, _ = c.reference()
        assert ((out.double() - want).abs() <= bound).all()


def test_strided_queries_on_another_stream():
    c = Case([2], [300], [0, 41], [2, 60], 8, 2, 128, 32, seed=81)
    cache, args, qs = c.cache(), c.args(), dev32(c.start)
    want = ndq.attention_prefix_kv8(c.q, cache, q_start=qs, **args)
    wide = torch.full((c.q.shape[0], 12 * 128 + 8), 9.0, dtype=c.q.dtype, device=DEV)
    wide[:, 8:8 + 8 * 128] = c.q.flatten(1)
    side = torch.cuda.Stream()
    out, ws = torch.empty_like(c.q), ndq.attention_prefix_workspace(cache, c.q.shape[0], 8)
    torch.cuda.synchronize()
    ndq.attention_prefix_kv8(wide[:, 8:8 + 8 * 128].unflatten(1, (8, 128)), cache, q_start=qs, out=out, workspace=ws, stream=side, **args)
    side.synchronize()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    got = ndq.attention_prefix_kv8(c.q, cache, q_start=qs, stream=side, **args)  # what it makes itself
    side.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_without_groups_it_is_attention_over_the_cache():
    c = Case([], [], [300, 41, 7], [1, 20, 3], 8, 2, 128, 16, seed=82)
    args = c.args()
    a = ndq.attention_prefix_kv8(c.q, c.cache(), q_start=dev32(c.start), **args)
    b = ndq.attention_kv8(c.q, c.cache(), args["block_table"], args["kv_len"], q_start=dev32(c.start))
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_calls_of_different_shapes_take_turns_on_one_workspace():
    # other tokens, heads and head sizes lay the workspace out anew: nothing that an earlier call left may be read
    cases = [Case([4], [700], [300, 40, 0, 500], [1] * 4, 32, 8, 128, 16, seed=91),
             Case([5, 2], [2000, 333], own_lengths(7, 400, 2), [3, 1, 4, 1, 30, 2, 6], 8, 2, 64, 32, "int8", F16, seed=92),
             Case([40], [900], own_lengths(40, 200, 3), [1] * 40, 16, 1, 128, 64, seed=93),
             Case([3], [1500], [5, 300, 0], [17, 40, 33], 10, 2, 128, 16, seed=94),
             Case([1] * 35 + [3], [200 + 7 * g for g in range(36)], own_lengths(38, 50, 4), [1] * 38, 4, 4, 64, 16, seed=95)]
    need = [ndq.ndq_attention_prefix_workspace_bytes(c.D, c.q.shape[0], c.Hq, c.kc.shape[1]) for c in cases]
    ws = torch.full((max(need),), 0xff, dtype=torch.uint8, device=DEV)
    ws[:4096] = 0
    want = [c.reference() for c in cases]
    caches, args = [c.cache() for c in cases], [c.args() for c in cases]
    for i in (0, 1, 2, 3, 4, 3, 0, 4, 2, 1, 0, 0, 2):
        c = cases[i]
        lse = torch.zeros(c.q.shape[:2], device=DEV)
        out = ndq.attention_prefix_kv8(c.q, caches[i], q_start=dev32(c.start), max_q=max(c.fresh), lse=lse, workspace=ws, **args[i])
        assert ((out.double() - want[i][0]).abs() <= want[i][1]).all(), i
        assert ((lse.double() - want[i][2]).abs() <= 2.0 ** -18 * (1 + want[i][2].abs()) + 2.0 ** -18 * 40).all(), i
        assert int(ws[:4096].count_nonzero()) == 0
