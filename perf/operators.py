"""The cases by which the serving operators are measured.

Four operators of a generation step: ``kv_plan`` (block tables and slot maps
from request lengths), ``kv_append`` (new keys and values into the 8-bit
cache), ``attention_kv8`` (attention over that cache) and ``lora_add``
(low-rank adapters of many requests beside a shared projection).  ``run``
computes them in plain torch operations, or calls the package when ``own`` is
set.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
S_MIN, S_MAX = 2.0 ** -100, 2.0 ** 100  # the range of a cache scale


def listed():
    return [
        # the bookkeeping of one generation step of a medium batch: pure latency
        dict(name="plan step 64", op="plan", R=64, bs=16, longest=8192, prefill=0.0, chunk=1),
        # a large mixed step: most requests generate one token, some bring a prompt chunk
        dict(name="plan mixed 2000", op="plan", R=2000, bs=32, longest=16384, prefill=0.06, chunk=4096),
        # one new token for each of 64 requests: blocks half full, scales that grow
        dict(name="append step 64", op="append", R=64, fresh=1, Hkv=8, D=128, bs=16, code="e4m3", dtype="bf16"),
        # prompt chunks of nine requests into blocks of 64 tokens
        dict(name="append prompt int8", op="append", R=9, fresh=1789, Hkv=8, D=128, bs=64, code="int8", dtype="f16"),
        # one user, a short context: latency
        dict(name="attend step 1x777", op="attend", R=1, fresh=1, context=776, ragged=False, Hq=32, Hkv=8, D=128, bs=16,
             code="e4m3", dtype="bf16", window=0),
        # an ordinary batch of 64 users with contexts of every length
        dict(name="attend step 64 ragged", op="attend", R=64, fresh=1, context=8191, ragged=True, Hq=32, Hkv=8, D=128,
             bs=16, code="int8", dtype="bf16", window=0),
        # few users with very long contexts, eight query heads for each cache head
        dict(name="attend step 8 long", op="attend", R=8, fresh=1, context=131000, ragged=True, Hq=64, Hkv=8, D=128,
             bs=64, code="e4m3", dtype="bf16", window=0),
        # verification of four drafted tokens, heads of 64, a sliding window
        dict(name="attend draft 33x4 window", op="attend", R=33, fresh=4, context=6000, ragged=True, Hq=32, Hkv=8, D=64,
             bs=32, code="e4m3", dtype="f16", window=2048),
        # prompt chunks over their own and earlier tokens: arithmetic
        dict(name="attend prompt 4 chunks", op="attend", R=4, fresh=4000, context=8192, ragged=True, Hq=32, Hkv=8, D=128,
             bs=16, code="e4m3", dtype="bf16", window=0),
        # one row beside a key projection of 1024
        dict(name="lora step 1", op="lora", M=1, runs=1, nA=4, rank=8, K=4096, N=1024, dtype="f32", idle=0.0),
        # a batch of 61 users with up to 48 adapters beside a 4096 x 4096 projection
        dict(name="lora step 61", op="lora", M=61, runs=61, nA=48, rank=16, K=4096, N=4096, dtype="f32", idle=0.1),
        # prompts of six requests beside an FFN projection
        dict(name="lora prompt 5003", op="lora", M=5003, runs=6, nA=6, rank=64, K=4096, N=14336, dtype="bf16", idle=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "lora"])
    bs = rng.choice([16, 32, 64, 128])
    if op == "plan":
        step = rng.random() < 0.5
        return dict(op=op, R=_log(rng, 1, 3000), bs=bs, longest=_log(rng, 100, 16000),
                    prefill=0.0 if step else rng.uniform(0, 0.05),
                    chunk=1 if step else _log(rng, 2, 4096))
    code, dtype, D = rng.choice(["e4m3", "int8"]), rng.choice(["bf16", "f16"]), rng.choice([64, 128, 128])
    if op == "append":
        R = _log(rng, 1, 256)
        return dict(op=op, R=R, fresh=1 if rng.random() < 0.4 else _log(rng, 2, max(2, 16000 // R)),
                    Hkv=rng.choice([1, 2, 4, 8]), D=D, bs=bs, code=code, dtype=dtype)
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 7, 8])
        kind = rng.random()
        if kind < 0.6:  # steps of one or a few tokens
            R = _log(rng, 1, 200)
            fresh, context = rng.choice([1, 1, 1, 2, 4, 5]), _log(rng, 1, min(131000, 600000 // R))
        else:  # prompt chunks
            R = rng.randint(1, 4)
            fresh, context = _log(rng, 17, 4000), _log(rng, 1, 8000)
        return dict(op=op, R=R, fresh=fresh, context=context, ragged=rng.random() < 0.7,
                    Hq=Hkv * (G if kind < 0.6 else min(G, 4)), Hkv=Hkv, D=D, bs=bs, code=code, dtype=dtype, window=rng.choice([0, 0, _log(rng, 16, 4096)]))
    M = _log(rng, 1, 4096)
    K, N = rng.choice([(4096, 4096), (4096, 1024), (4096, 14336), (14336, 4096), (2048, 512), (1000, 1032)])
    return dict(op=op, M=M, runs=min(M, _log(rng, 1, 256)), nA=_log(rng, 1, 64),
                rank=rng.choice([4, 8, 16, 24, 32, 64]), K=K, N=N, dtype=rng.choice(["f32", "bf16"]), idle=rng.choice([0.0, 0.2]))


# ---- inputs ------------------------------------------------------------------


def _lengths(case):
    """(cached, fresh) of each request, as lists: the same set for every seed, which only deals them out."""
    R = case["R"]
    u = torch.rand(3, R, generator=torch.Generator().manual_seed(R)).tolist()
    if case["op"] == "plan":
        return ([int(a * case["longest"]) for a in u[0]],
                [1 + int(b * case["chunk"]) if a < case["prefill"] else 1 for a, b in zip(u[1], u[2])])
    if case["op"] == "append":
        even = case["fresh"] == 1 or R == 1
        return [int(3000 * a) for a in u[0]], [case["fresh"] if even else 1 + int(a * case["fresh"]) for a in u[1]]
    if not case["ragged"]:
        return [case["context"]] * R, [case["fresh"]] * R
    spread = [(i + 1) / R for i in range(R)] if R <= 8 else u[0]  # few requests: lengths spread evenly
    cached = [int((0.02 + 0.98 * a) * case["context"]) for a in spread]
    if case["fresh"] <= 16:
        return cached, [case["fresh"]] * R
    return cached, [max(1, int((0.3 + 0.7 * a) * case["fresh"])) for a in reversed(spread)]


def _dealt(case, gen):
    cached, fresh = _lengths(case)
    order = torch.randperm(case["R"], generator=gen).tolist()
    return [cached[i] for i in order], [fresh[i] for i in order]


def _quantize(x, code):
    """Random cache contents: codes and scales of x [blocks, heads, bs, D]."""
    s = x.abs().amax(dim=(2, 3)) / QMAX[code]
    c = x / s[:, :, None, None]
    return (c.clamp(-448, 448).to(torch.float8_e4m3fn) if code == "e4m3" else c.round().clamp(-127, 127).to(torch.int8)), s


def _cache(case, nblocks, dev_gen):
    Hkv, bs, D, code = case["Hkv"], case["bs"], case["D"], case["code"]
    out = []
    for spread in (1.0, 0.5):
        c = torch.empty(nblocks, Hkv, bs, D, dtype=CODE[code], device=DEV)
        s = torch.empty(nblocks, Hkv, dtype=torch.float32, device=DEV)
        channel = torch.exp(0.4 * torch.randn(1, Hkv, 1, D, device=DEV, generator=dev_gen)) * spread
        step = max(1, (1 << 26) // (Hkv * bs * D))
        for b in range(0, nblocks, step):
            n = min(step, nblocks - b)
            x = torch.randn(n, Hkv, bs, D, device=DEV, generator=dev_gen) * channel
            c[b:b + n], s[b:b + n] = _quantize(x, code)
        out += [c, s]
    return out


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dgen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "plan":
        R, bs = case["R"], case["bs"]
        cached, fresh = (torch.tensor(x, dtype=torch.int32) for x in _dealt(case, gen))
        width = (case["longest"] + case["chunk"]) // bs + 2
        had = (cached + bs - 1) // bs
        pool = torch.randperm(R * width, generator=gen).to(torch.int32)
        table = pool[:R * width].reshape(R, width).clone()
        table[torch.arange(width)[None, :] >= had[:, None]] = -1
        need = int(((cached + fresh + bs - 1) // bs - had).sum())
        free = R * width + torch.randperm(need + 100, generator=gen).to(torch.int32)
        s |= dict(cached=cached.to(DEV), fresh=fresh.to(DEV), table=table.to(DEV), free=free.to(DEV),
                  count=torch.tensor([need + 50], **i32), T=int(fresh.sum()))
        return s
    if case["op"] in ("append", "attend"):
        R, bs, Hkv, D = case["R"], case["bs"], case["Hkv"], case["D"]
        dt = DTYPES[case["dtype"]]
        cached, fresh = _dealt(case, gen)
        kv = [a + b for a, b in zip(cached, fresh)]
        blocks = [-(-n // bs) for n in kv]
        total = sum(blocks)
        nblocks = total + total // 16 + 2
        ids = torch.randperm(nblocks, generator=gen)[:total].to(torch.int32)
        width = max(blocks)
        table = torch.full((R, width), -1, dtype=torch.int32)
        at = torch.arange(width)[None, :] < torch.tensor(blocks)[:, None]
        table[at] = ids
        kc, ks, vc, vs = _cache(case, nblocks, dgen)
        T = sum(fresh)
        s |= dict(kc=kc, ks=ks, vc=vc, vs=vs, T=T)
        if case["op"] == "append":
            r = torch.repeat_interleave(torch.arange(R), torch.tensor(fresh))
            start = torch.tensor([0] + fresh).cumsum(0)
            pos = torch.tensor(cached)[r] + torch.arange(T) - start[r]
            slots = table[r, pos // bs].long() * bs + pos % bs
            # keys and values as slices of one row of the fused projection, now and then larger than what the block holds
            size = torch.exp(0.5 * torch.randn(T, 1, 1, 1, device=DEV, generator=dgen))
            kvrow = (torch.randn(T, 2, Hkv, D, device=DEV, generator=dgen) * size).to(dt)
            s |= dict(k=kvrow[:, 0], v=kvrow[:, 1], slots=slots.to(DEV))
            return s
        s |= dict(q=(torch.randn(T, case["Hq"], D, device=DEV, generator=dgen) * 1.2).to(dt), table=table.to(DEV),
                  kv_len=torch.tensor(kv, **i32), q_start=torch.tensor([0] + fresh).cumsum(0).to(torch.int32).to(DEV),
                  max_q=max(fresh), scale=1.0 / math.sqrt(D), out=torch.empty(T, case["Hq"], D, dtype=dt, device=DEV))
        return s
    M, nA, rank, K, N = case["M"], case["nA"], case["rank"], case["K"], case["N"]
    dt = DTYPES[case["dtype"]]
    edges = [0] + sorted(torch.randperm(M - 1, generator=gen)[:case["runs"] - 1].add(1).tolist()) + [M]
    which = torch.randint(0, nA, (case["runs"],), generator=gen).to(torch.int32)
    which[torch.rand(case["runs"], generator=gen) < case["idle"]] = -1  # requests without an adapter
    index = torch.repeat_interleave(which, torch.tensor([b - a for a, b in zip(edges, edges[1:])]))
    ranks = torch.tensor([rank if i % 3 else max(1, rank // 2) for i in range(nA)], dtype=torch.int32)
    a = (torch.randn(nA, rank, K, device=DEV, generator=dgen) / math.sqrt(K)).to(torch.bfloat16)
    b = (torch.randn(nA, N, rank, device=DEV, generator=dgen) * 0.3).to(torch.bfloat16)
    s |= dict(x=torch.randn(M, K, device=DEV, generator=dgen).to(torch.bfloat16), a=a, b=b, ranks=ranks.to(DEV),
              scales=(0.5 + torch.rand(nA, generator=gen)).to(DEV), index=index.to(DEV),
              base=torch.randn(M, N, device=DEV, generator=dgen).to(dt),
              out=torch.empty(M, N, dtype=dt, device=DEV))
    return s


# ---- plain forms -------------------------------------------------------------


def _plan(s):
    bs, T, R = s["bs"], s["T"], s["R"]
    cached, fresh, table, free = s["cached"].clamp(min=0), s["fresh"].clamp(min=0), s["table"], s["free"]
    width = table.shape[1]
    kv_len = cached + fresh
    q_start = torch.zeros(R + 1, dtype=torch.int32, device=DEV)
    q_start[1:] = fresh.cumsum(0)
    had = (cached + bs - 1) // bs
    need = (kv_len + bs - 1) // bs - had
    first = need.cumsum(0) - need
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(q_start[1:], t, right=True)
    pos = cached[r] + t - q_start[r]
    blk = pos // bs
    taken = s["count"] - 1 - (first[r] + blk - had[r])
    got = torch.where(taken >= 0, free[taken.clamp(min=0)], -1)
    new = blk >= had[r]
    inside = blk < width
    ident = torch.where(new, got, table[r, blk.clamp(max=width - 1)])
    ident = torch.where(inside, ident, -1)
    wide = torch.cat([table, table[:, :1]], dim=1)  # the last column takes what is not written
    wide[r, torch.where(new & inside, blk, width)] = torch.where(new & inside, got, 0).to(torch.int32)
    table.copy_(wide[:, :width])
    slots = torch.where(ident >= 0, ident.long() * bs + pos % bs, -1)
    return [q_start, kv_len, pos.to(torch.int32), slots, s["count"] - need.sum().to(torch.int32), table]


def _code(x, code):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn) if code == "e4m3" else x.round().clamp(-127, 127).to(torch.int8)


def _append(s):
    bs, code, slots, T = s["bs"], s["code"], s["slots"], s["T"]
    blk, off = slots // bs, slots % bs
    lead = torch.ones(T, dtype=torch.bool, device=DEV)
    lead[1:] = blk[1:] != blk[:-1]
    run = lead.cumsum(0) - 1
    ublk, uoff = blk[lead], off[lead]
    for x, c, sc in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        x = x.float()
        amax = torch.zeros(ublk.numel(), s["Hkv"], device=DEV)
        amax.scatter_reduce_(0, run[:, None].expand(-1, s["Hkv"]), x.abs().amax(2), "amax")
        fresh = amax / torch.full_like(amax, QMAX[code])
        fresh = torch.where(amax > 0, fresh.clamp(S_MIN, S_MAX), 0.0)
        old = torch.where(uoff[:, None] > 0, sc[ublk], 0.0)
        new = torch.maximum(old, fresh)
        div = torch.where(new > 0, new, 1.0)
        grown = (uoff > 0) & ((new > old) & (old > 0)).any(1)
        gb = ublk[grown]
        before = c[gb].float() * old[grown][:, :, None, None] / div[grown][:, :, None, None]
        keep = (torch.arange(bs, device=DEV)[None, None, :, None] < uoff[grown][:, None, None, None]) & \
            ((new > old) & (old > 0))[grown][:, :, None, None]
        c.view(torch.int8)[gb] = torch.where(keep, _code(before, code).view(torch.int8), c.view(torch.int8)[gb])
        c.view(torch.int8)[blk, :, off] = _code(x / div[run][:, :, None], code).view(torch.int8)
        sc[ublk] = new
    return [s["kc"], s["ks"], s["vc"], s["vs"]]


def _attend(s):
    R, Hq, Hkv, D, bs = s["R"], s["Hq"], s["Hkv"], s["D"], s["bs"]
    G, mq, T = Hq // Hkv, s["max_q"], s["T"]
    table, kv_len, q_start = s["table"].long().clamp(min=0), s["kv_len"].long(), s["q_start"].long()
    L = table.shape[1] * bs
    k = s["kc"][table].float() * s["ks"][table][..., None, None]  # [R, W, Hkv, bs, D]
    k = k.permute(0, 2, 4, 1, 3).reshape(R, Hkv, D, L)
    n = q_start[1:] - q_start[:-1]
    i = torch.arange(mq, device=DEV)
    row = (q_start[:-1, None] + i).clamp(max=T - 1)  # [R, mq]
    q = s["q"].float()[row].reshape(R, mq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * mq, D)
    p = torch.matmul(q * s["scale"], k).reshape(R, Hkv, G, mq, L)
    del k
    at = (kv_len - n)[:, None] + i  # position of each query
    j = torch.arange(L, device=DEV)
    seen = (j <= at[..., None]) & (j < kv_len[:, None, None])
    if s["window"]:
        seen = seen & (j > at[..., None] - s["window"])
    p.masked_fill_(~seen[:, None, None], -math.inf)
    p -= p.amax(-1, keepdim=True).clamp(min=-3e38)
    p.exp_()
    total = p.sum(-1, keepdim=True)
    v = s["vc"][table].float() * s["vs"][table][..., None, None]
    v = v.permute(0, 2, 1, 3, 4).reshape(R, Hkv, L, D)
    o = torch.matmul(p.reshape(R, Hkv, G * mq, L), v).reshape(R, Hkv, G, mq, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(R, mq, Hq, D)
    r = torch.searchsorted(q_start[1:], torch.arange(T, device=DEV), right=True)
    return o[r, torch.arange(T, device=DEV) - q_start[r]].to(s["q"].dtype)


def _lora(s):
    nA, rank = s["nA"], s["rank"]
    t = torch.matmul(s["x"].float(), s["a"].float().reshape(nA * rank, -1).T).reshape(-1, nA, rank)
    mine = (torch.arange(nA, device=DEV) == s["index"][:, None])[..., None]
    mine = mine & (torch.arange(rank, device=DEV) < s["ranks"][:, None])
    t = torch.where(mine, t * s["scales"][:, None], 0.0)
    d = torch.matmul(t.reshape(-1, nA * rank), s["b"].float().permute(0, 2, 1).reshape(nA * rank, -1))
    return (s["base"].float() + d).to(s["base"].dtype)


# ---- one pass ------------------------------------------------------------------


def _handle(s, ndq):
    if "handle" not in s:  # what a program keeps from one call to the next
        if s["op"] == "plan":
            s["handle"] = ndq.kv_plan_buffers(s["R"], s["T"], DEV)
        elif s["op"] == "append":
            s["handle"] = ndq.KvCache(s["kc"], s["vc"], s["ks"], s["vs"])
        elif s["op"] == "attend":
            s["handle"] = ndq.KvCache(s["kc"], s["vc"], s["ks"], s["vs"])
            s["ws"] = ndq.attention_workspace(s["R"], s["T"], s["Hq"], s["handle"], max_q=s["max_q"])
        else:
            s["handle"] = ndq.lora_workspace(s["M"], s["nA"], s["rank"], s["K"], DEV)
    return s["handle"]


def run(s):
    if not own:
        return {"plan": _plan, "append": _append, "attend": _attend, "lora": _lora}[s["op"]](s)
    import quantized_weight_block_gb300 as ndq

    h = _handle(s, ndq)
    if s["op"] == "plan":
        p = ndq.kv_plan(s["cached"], s["fresh"], s["bs"], s["free"], s["count"], s["table"], out=h)
        return [p.q_start, p.kv_len, p.positions, p.slots, p.free_left, s["table"]]
    if s["op"] == "append":
        ndq.kv_append(h, s["k"], s["v"], s["slots"])
        return [s["kc"], s["ks"], s["vc"], s["vs"]]
    if s["op"] == "attend":
        return ndq.attention_kv8(s["q"], h, s["table"], s["kv_len"], q_start=s["q_start"], max_q=s["max_q"],
                                 scale=s["scale"], window=s["window"], out=s["out"], workspace=s["ws"])
    return ndq.lora_add(s["x"], s["a"], s["b"], s["ranks"], s["scales"], s["index"], s["base"], out=s["out"], workspace=h)


# ---- what a pass cannot do without -------------------------------------------


def _seen(case, cached, fresh):
    """Sum over queries of visible keys, and the keys that some query sees."""
    w = case["window"]
    pairs = keys = 0
    for c, f in zip(cached, fresh):
        if not w:
            pairs += f * c + f * (f + 1) // 2
            keys += c + f
        else:
            pairs += sum(min(w, c + i + 1) for i in range(f))
            keys += min(c + f, w + f - 1)
    return pairs, keys


def work(case):
    if case["op"] == "plan":
        T = sum(_lengths(case)[1])
        return dict(bytes=16 * case["R"] + 12 * T + 12 * T / case["bs"], flops=10 * T)
    if case["op"] == "append":
        cached, fresh = _lengths(case)
        n = 2 * sum(fresh) * case["Hkv"] * case["D"]
        touched = 2 * sum((c + f - 1) // case["bs"] - c // case["bs"] + 1 for c, f in zip(cached, fresh)) * case["Hkv"]
        return dict(bytes=3 * n + 8 * touched + 8 * sum(fresh), flops=3 * n)
    if case["op"] == "attend":
        cached, fresh = _lengths(case)
        pairs, keys = _seen(case, cached, fresh)
        cache = 2 * keys * case["Hkv"] * case["D"] + 8 * (keys // case["bs"]) * case["Hkv"]
        return dict(bytes=cache + 4 * sum(fresh) * case["Hq"] * case["D"],
                    flops=4 * pairs * case["Hq"] * case["D"])
    # the expected number of adapters in use
    used = case["nA"] * (1 - (1 - 1 / case["nA"]) ** (case["runs"] * (1 - case["idle"])))
    r = case["rank"] * 5 / 6
    out = case["M"] * case["N"] * (4 if case["dtype"] == "f32" else 2)
    return dict(bytes=2 * case["M"] * case["K"] + 2 * used * r * (case["K"] + case["N"]) + 2 * out,
                flops=2 * case["M"] * r * (case["K"] + case["N"]))


# ---- the definitions in 64 bits ----------------------------------------------


def _exact_attend(s):
    G = s["Hq"] // s["Hkv"]
    start, kv = s["q_start"].tolist(), s["kv_len"].tolist()
    out = torch.zeros(s["T"], s["Hq"], s["D"], dtype=torch.float64, device=DEV)
    for r in range(s["R"]):
        ids = s["table"][r, :-(-kv[r] // s["bs"])].long()
        n = start[r + 1] - start[r]
        pos = torch.arange(kv[r] - n, kv[r], device=DEV)[:, None]
        col = torch.arange(kv[r], device=DEV)[None, :]
        hide = col > pos
        if s["window"]:
            hide |= col <= pos - s["window"]
        for h in range(s["Hkv"]):
            k = (s["kc"][ids, h].double() * s["ks"][ids, h].double()[:, None, None]).flatten(0, 1)[:kv[r]]
            v = (s["vc"][ids, h].double() * s["vs"][ids, h].double()[:, None, None]).flatten(0, 1)[:kv[r]]
            for g in range(G):
                e = s["q"][start[r]:start[r + 1], h * G + g].double() @ k.T * s["scale"]
                e[hide] = -math.inf
                out[start[r]:start[r + 1], h * G + g] = torch.softmax(e, -1) @ v
    return out


def _exact_append(s):
    """Scales alone: a code next to a rounding boundary may go either way in 64 bits."""
    out = []
    slots, bs = s["slots"].tolist(), s["bs"]
    first, last = {}, {}
    for t, x in enumerate(slots):
        first.setdefault(x // bs, t)
        last[x // bs] = t
    for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        new = sc.double().cpu()
        a = x.double().abs().amax(2).cpu()
        for b, t in first.items():
            m = a[t:last[b] + 1].amax(0) / QMAX[s["code"]]
            new[b] = torch.maximum(new[b], m) if slots[t] % bs else m
        out.append(new.to(DEV))
    return [None, out[0], None, out[1]]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None  # whole numbers
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    y = s["base"].double()
    index, ranks = s["index"], s["ranks"].tolist()
    for a in range(s["nA"]):
        rows = (index == a).nonzero()[:, 0]
        low = s["x"][rows].double() @ s["a"][a, :ranks[a]].double().T
        y[rows] += float(s["scales"][a]) * (low @ s["b"][a, :, :ranks[a]].double().T)
    return y
