"""The cases by which the step's other operators are measured.

Three operators that stand around the cache of a generation step:
``embed_packed`` (rows of a packed embedding table, decoded and scaled),
``qk_norm_rope`` (the norms of query and key heads and their rotation by
position, in one pass) and ``attention_prefix_kv8`` (attention over the 8-bit
cache for requests that share a long prefix, which is read once for all of
them).  ``run`` computes them in plain torch operations, or calls the package
when ``own`` is set.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FORMATS = {"gguf:q8_0": (32, 34), "gguf:q4_0": (32, 18), "gguf:q4_k": (256, 144), "gguf:q6_k": (256, 210)}


def listed():
    return [
        # the token of one user: latency
        dict(name="embed step 1", op="embed", fmt="gguf:q6_k", V=128256, K=4096, T=1, scale=1.0, dtype="bf16"),
        # the tokens of a batch, scaled by the root of the row's length, to binary32
        dict(name="embed step 61", op="embed", fmt="gguf:q8_0", V=128256, K=4096, T=61, scale=64.0, dtype="f32"),
        # prompts of a large step
        dict(name="embed prompt 16001", op="embed", fmt="gguf:q4_k", V=128256, K=4096, T=16001, scale=1.0, dtype="bf16"),
        # one generation step of 61 users in a batch of 64, far positions: latency
        dict(name="rope step 64", op="rope", T=64, pad=3, Hq=32, Hkv=8, D=128, rot=128, far=131000, norm=True,
             interleaved=False, din="bf16", dtype="bf16"),
        # drafted tokens, heads of 64 rotated in part, neighbouring pairs, no norm
        dict(name="rope draft 132 interleaved", op="rope", T=132, pad=0, Hq=32, Hkv=8, D=64, rot=32, far=8000, norm=False,
             interleaved=True, din="f16", dtype="f16"),
        # prompt chunks, projections in bfloat16
        dict(name="rope prompt 16001", op="rope", T=16001, pad=0, Hq=32, Hkv=8, D=128, rot=128, far=32000, norm=True,
             interleaved=False, din="bf16", dtype="bf16"),
        # prompt chunks, projections in binary32 as the packed product leaves them
        dict(name="rope prompt 5003 f32", op="rope", T=5003, pad=0, Hq=64, Hkv=8, D=128, rot=128, far=32000, norm=True,
             interleaved=False, din="f32", dtype="bf16"),
        # a few users behind one system prompt: latency
        dict(name="prefix step 5x2000", op="prefix", R=5, groups=1, fresh=1, prefix=2000, private=300, ragged=True, Hq=32, Hkv=8,
             D=128, bs=16, code="e4m3", dtype="bf16", window=0),
        # a batch of 64 users behind one long document
        dict(name="prefix step 64x32000", op="prefix", R=64, groups=1, fresh=1, prefix=32000, private=2000, ragged=True,
             Hq=32, Hkv=8, D=128, bs=64, code="e4m3", dtype="bf16", window=0),
        # sampled answers to several prompts: seven groups of every size and length
        dict(name="prefix step 96 in 7 groups", op="prefix", R=96, groups=7, fresh=1, prefix=12000, private=1500, ragged=True,
             Hq=32, Hkv=8, D=64, bs=16, code="int8", dtype="f16", window=0),
        # verification of four drafted tokens, eight query heads for each cache head
        dict(name="prefix draft 33x4", op="prefix", R=33, groups=2, fresh=4, prefix=16000, private=1000, ragged=True, Hq=64,
             Hkv=8, D=128, bs=32, code="e4m3", dtype="bf16", window=0),
        # prompts of eight requests behind one system prompt: arithmetic
        dict(name="prefix prompt 8 chunks", op="prefix", R=8, groups=1, fresh=1000, prefix=8000, private=600, ragged=True,
             Hq=32, Hkv=8, D=128, bs=16, code="e4m3", dtype="bf16", window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "rope", "prefix", "prefix"])
    if op == "embed":
        K = rng.choice([512, 1024, 2048, 4096])
        return dict(op=op, fmt=rng.choice(sorted(FORMATS)), V=_log(rng, 1000, 130000), K=K, T=_log(rng, 1, 16000),
                    scale=rng.choice([1.0, math.sqrt(K)]), dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        T = _log(rng, 1, 8000)
        return dict(op=op, T=T, pad=rng.choice([0, min(5, T - 1)]), Hq=_log(rng, 1, 40), Hkv=rng.choice([1, 2, 4, 5, 8]), D=D,
                    rot=rng.choice([D, D, D // 32 * 16]), far=_log(rng, 100, 1000000), norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.4, din=rng.choice(["bf16", "f16", "f32"]), dtype=rng.choice(["bf16", "f16"]))
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
    if rng.random() < 0.7:  # steps of one or a few tokens
        R, fresh = _log(rng, 1, 100), rng.choice([1, 1, 1, 2, 3, 5])
        prefix = _log(rng, 20, min(32000, 2000000 // R))
    else:  # prompt chunks
        R, fresh, G = rng.randint(1, 6), _log(rng, 17, 1000), min(G, 4)
        prefix = _log(rng, 20, 8000)
    return dict(op=op, R=R, groups=rng.randint(1, max(1, min(8, R // 2))), fresh=fresh, prefix=prefix,
                private=_log(rng, 1, 2000), ragged=rng.random() < 0.7, Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128, 128]),
                bs=rng.choice([16, 32, 64, 128]), code=rng.choice(["e4m3", "int8"]), dtype=rng.choice(["bf16", "f16"]),
                window=rng.choice([0, 0, 0, _log(rng, 64, 16000)]))


# ---- inputs ------------------------------------------------------------------


def _lengths(case):
    """Group starts, prefix lengths, tokens and new tokens of each request: the same for every seed."""
    R, n = case["R"], case["groups"]
    u = torch.rand(3, max(R, 8), generator=torch.Generator().manual_seed(R * 31 + n)).tolist()
    if n == 1 or not case["ragged"]:
        starts = [R * g // n for g in range(n + 1)]
        prefix = [case["prefix"]] * n
    else:  # groups of unlike sizes and lengths
        w = [0.3 + x for x in u[2][:n]]
        starts = [0]
        for g in range(n):
            starts.append(R if g == n - 1 else min(R, max(starts[-1] + 1, round(R * sum(w[:g + 1]) / sum(w)))))
        prefix = [max(1, int((g + 1) / n * case["prefix"])) for g in range(n)]
    fresh = [case["fresh"]] * R
    own_tokens = [case["private"]] * R
    if case["ragged"]:
        own_tokens = [int(x * case["private"]) for x in u[0][:R]]
        if case["fresh"] > 16:
            fresh = [max(1, int((0.3 + 0.7 * x) * case["fresh"])) for x in u[1][:R]]
    which = [next(g for g in range(n) if starts[g] <= r < starts[g + 1]) for r in range(R)]
    kv = [prefix[which[r]] + own_tokens[r] + fresh[r] for r in range(R)]
    return starts, prefix, which, kv, fresh


def _payload(case, gen):
    """Random packed rows with scales of the size that real ones have."""
    B, S = FORMATS[case["fmt"]]
    n = case["V"] * case["K"] // B
    x = torch.randint(0, 256, (n, S), dtype=torch.uint8, device=DEV, generator=gen)

    def half(lo, hi):
        return (lo + (hi - lo) * torch.rand(n, device=DEV, generator=gen)).to(torch.float16).view(torch.uint8).reshape(n, 2)

    if case["fmt"] == "gguf:q8_0":
        x[:, :2] = half(1e-4, 8e-4)
    elif case["fmt"] == "gguf:q4_0":
        x[:, :2] = half(2e-3, 8e-3)
    elif case["fmt"] == "gguf:q4_k":
        x[:, :2], x[:, 2:4] = half(5e-5, 2e-4), half(2e-4, 8e-4)
    else:
        x[:, 208:] = half(1e-5, 4e-5)
    return x.reshape(-1)


def _cache(case, nblocks, gen):
    Hkv, bs, D, code = case["Hkv"], case["bs"], case["D"], case["code"]
    out = []
    for spread in (1.0, 0.5):
        c = torch.empty(nblocks, Hkv, bs, D, dtype=CODE[code], device=DEV)
        s = torch.empty(nblocks, Hkv, dtype=torch.float32, device=DEV)
        channel = torch.exp(0.4 * torch.randn(1, Hkv, 1, D, device=DEV, generator=gen)) * spread
        step = max(1, (1 << 26) // (Hkv * bs * D))
        for b in range(0, nblocks, step):
            n = min(step, nblocks - b)
            x = torch.randn(n, Hkv, bs, D, device=DEV, generator=gen) * channel
            s[b:b + n] = x.abs().amax(dim=(2, 3)) / QMAX[code]
            x = x / s[b:b + n, :, None, None]
            c[b:b + n] = x.clamp(-448, 448).to(torch.float8_e4m3fn) if code == "e4m3" else x.round().clamp(-127, 127).to(torch.int8)
        out += [c, s]
    return out


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dgen = torch.Generator(device=DEV).manual_seed(seed)
    s, i32 = dict(case), torch.int32
    if case["op"] == "embed":
        ids = torch.randint(0, case["V"], (case["T"],), generator=gen).to(i32)
        s |= dict(w=_payload(case, dgen), ids=ids.to(DEV), out=torch.empty(case["T"], case["K"], dtype=DTYPES[case["dtype"]], device=DEV))
        return s
    if case["op"] == "rope":
        T, Hq, Hkv, D, rot = (case[k] for k in ("T", "Hq", "Hkv", "D", "rot"))
        real = T - case["pad"]
        if T <= 256:  # a step: every token of another request
            pos = torch.randint(0, case["far"], (T,), generator=gen)
        else:  # chunks of up to 4096 tokens
            chunk = torch.randint(0, case["far"], ((T + 4095) // 4096,), generator=gen)
            pos = chunk.repeat_interleave(4096)[:T] + torch.arange(T) % 4096
        pos[real:] = -1
        # queries and keys as slices of one row of the fused projection
        row = (torch.randn(T, Hq + 2 * Hkv, D, device=DEV, generator=dgen) * 1.5).to(DTYPES[case["din"]])
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
        s |= dict(q=row[:, :Hq], k=row[:, Hq:Hq + Hkv], pos=pos.to(i32).to(DEV), freq=freq.float().to(DEV), eps=1e-6,
                  qw=None, kw=None)
        if case["norm"]:
            s |= dict(qw=1 + 0.2 * torch.randn(D, device=DEV, generator=dgen), kw=1 + 0.2 * torch.randn(D, device=DEV, generator=dgen))
        for name, H in (("qo", Hq), ("ko", Hkv)):
            s[name] = torch.zeros(T, H, D, dtype=DTYPES[case["dtype"]], device=DEV)
        return s
    R, bs = case["R"], case["bs"]
    starts, prefix, which, kv, fresh = _lengths(case)
    shared = [n // bs for n in prefix]  # whole blocks alone can be shared
    blocks = [-(-n // bs) for n in kv]
    total = sum(shared) + sum(b - shared[g] for b, g in zip(blocks, which))
    nblocks = total + total // 16 + 2
    ids = torch.randperm(nblocks, generator=gen)[:total].to(i32)
    table = torch.full((R, max(blocks)), -1, dtype=i32)
    at = sum(shared)
    first = [sum(shared[:g]) for g in range(len(shared))]
    for r in range(R):
        g = which[r]
        own_blocks = blocks[r] - shared[g]
        table[r, :shared[g]] = ids[first[g]:first[g] + shared[g]]
        table[r, shared[g]:blocks[r]] = ids[at:at + own_blocks]
        at += own_blocks
    kc, ks, vc, vs = _cache(case, nblocks, dgen)
    T, dt = sum(fresh), DTYPES[case["dtype"]]
    s |= dict(kc=kc, ks=ks, vc=vc, vs=vs, T=T, table=table.to(DEV), kv_len=torch.tensor(kv, dtype=i32, device=DEV),
              q_start=torch.tensor([0] + fresh).cumsum(0).to(i32).to(DEV), max_q=max(fresh), scale=1.0 / math.sqrt(case["D"]),
              group_start=torch.tensor(starts, dtype=i32, device=DEV), prefix_len=torch.tensor(prefix, dtype=i32, device=DEV),
              q=(torch.randn(T, case["Hq"], case["D"], device=DEV, generator=dgen) * 1.2).to(dt),
              out=torch.empty(T, case["Hq"], case["D"], dtype=dt, device=DEV))
    return s


# ---- plain forms -------------------------------------------------------------


def _half(b):
    return b.contiguous().view(torch.float16).float()


def _decode(fmt, x):
    """Packed blocks [n, S] to binary32 [n, B], each product and sum rounded by itself."""
    if fmt == "gguf:q8_0":
        return _half(x[:, :2]) * x[:, 2:].contiguous().view(torch.int8).float()
    if fmt == "gguf:q4_0":
        return _half(x[:, :2]) * (torch.cat([x[:, 2:] & 15, x[:, 2:] >> 4], 1).float() - 8)
    if fmt == "gguf:q4_k":
        d, dmin, c, q = _half(x[:, :2]), _half(x[:, 2:4]), x[:, 4:16], x[:, 16:]
        sc = torch.cat([c[:, :4] & 63, (c[:, 8:] & 15) | ((c[:, :4] >> 6) << 4)], 1).float()
        mn = torch.cat([c[:, 4:8] & 63, (c[:, 8:] >> 4) | ((c[:, 4:8] >> 6) << 4)], 1).float()
        q = q.reshape(-1, 4, 1, 32)
        codes = torch.cat([q & 15, q >> 4], 2).reshape(-1, 8, 32).float()
        return ((d * sc)[..., None] * codes - (dmin * mn)[..., None]).flatten(1)
    ql, qh, sc, d = x[:, :128], x[:, 128:192], x[:, 192:208].contiguous().view(torch.int8).float(), _half(x[:, 208:])
    ql, qh = ql.reshape(-1, 2, 2, 32), qh.reshape(-1, 2, 1, 32)
    low = torch.cat([ql & 15, ql >> 4], 2)  # [n, half, quarter, 32]
    high = torch.cat([(qh >> s) & 3 for s in (0, 2, 4, 6)], 2)
    codes = (low | (high << 4)).float() - 32
    return ((d * sc)[..., None] * codes.reshape(-1, 16, 16)).flatten(1)


def _embed(s):
    B, S = FORMATS[s["fmt"]]
    rows = s["w"].reshape(s["V"], -1)[s["ids"].long()]
    return (_decode(s["fmt"], rows.reshape(-1, S)).reshape(s["T"], s["K"]) * s["scale"]).to(DTYPES[s["dtype"]])


def _rope(s):
    rot, dt = s["rot"], DTYPES[s["dtype"]]
    angle = s["pos"].double()[:, None] * s["freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, w, y in ((s["q"], s["qw"], s["qo"]), (s["k"], s["kw"], s["ko"])):
        z = x.float()
        if w is not None:
            z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + s["eps"]) * w
        r, rest = z[..., :rot], z[..., rot:]
        if s["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        out.append(torch.where(s["pos"][:, None, None] >= 0, torch.cat([r, rest], -1).to(dt), y))
    return out


def _prefix(s):
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


# ---- one pass ------------------------------------------------------------------


def run(s):
    if not own:
        return {"embed": _embed, "rope": _rope, "prefix": _prefix}[s["op"]](s)
    import quantized_weight_block_gb300 as ndq

    if s["op"] == "embed":
        return ndq.embed_packed(s["fmt"], s["w"], s["V"], s["K"], s["ids"], scale=s["scale"], out=s["out"])
    if s["op"] == "rope":
        return list(ndq.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"],
                                     interleaved=s["interleaved"], q_out=s["qo"], k_out=s["ko"]))
    if "cache" not in s:  # what a program keeps from one call to the next
        s["cache"] = ndq.KvCache(s["kc"], s["vc"], s["ks"], s["vs"])
        s["ws"] = ndq.attention_prefix_workspace(s["cache"], s["T"], s["Hq"])
    return ndq.attention_prefix_kv8(s["q"], s["cache"], s["table"], s["kv_len"], s["group_start"], s["prefix_len"],
                                    q_start=s["q_start"], max_q=s["max_q"], scale=s["scale"], window=s["window"],
                                    out=s["out"], workspace=s["ws"])


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "embed":
        B, S = FORMATS[case["fmt"]]
        rows = case["V"] * (1 - (1 - 1 / case["V"]) ** case["T"])  # different ones, as expected
        return dict(bytes=rows * case["K"] // B * S + case["T"] * (4 + case["K"] * size[case["dtype"]]), flops=2 * case["T"] * case["K"])
    if case["op"] == "rope":
        n = (case["T"] - case["pad"]) * (case["Hq"] + case["Hkv"]) * case["D"]
        return dict(bytes=n * (size[case["din"]] + size[case["dtype"]]) + 4 * case["T"], flops=n * (8 if case["norm"] else 3))
    starts, prefix, which, kv, fresh = _lengths(case)
    w, pairs, keys = case["window"], 0, 0
    lowest = [None] * len(prefix)  # the first token of each prefix that some query sees
    for g, n, f in zip(which, kv, fresh):
        end = [n - f + i + 1 for i in range(f)]
        begin = [max(0, e - w) if w else 0 for e in end]
        pairs += sum(e - b for b, e in zip(begin, end))
        keys += n - max(prefix[g], begin[0])
        lowest[g] = min(begin[0], prefix[g]) if lowest[g] is None else min(lowest[g], begin[0])
    keys += sum(p - x for p, x in zip(prefix, lowest) if x is not None)
    cache = 2 * keys * case["Hkv"] * case["D"] + 8 * (keys // case["bs"]) * case["Hkv"]
    return dict(bytes=cache + 4 * sum(fresh) * case["Hq"] * case["D"], flops=4 * pairs * case["Hq"] * case["D"])


# ---- the definitions in 64 bits ----------------------------------------------


def _exact_embed(s):
    """Block by block from the fields of each format, in 64 bits."""
    B, S = FORMATS[s["fmt"]]
    bpr = s["K"] // B
    blocks = s["w"].reshape(s["V"], bpr, S)[s["ids"].long()]
    byte = blocks.to(torch.int64)

    def f16(i):
        return blocks[..., i:i + 2].contiguous().view(torch.float16).double()

    e = torch.arange(B, device=DEV)
    if s["fmt"] == "gguf:q8_0":
        c = byte[..., 2:]
        y = torch.where(c > 127, c - 256, c) * f16(0)
    elif s["fmt"] == "gguf:q4_0":
        y = (((byte[..., 2 + e % 16] >> (4 * (e // 16))) & 15) - 8) * f16(0)
    elif s["fmt"] == "gguf:q4_k":
        j = e // 32  # sub-block
        code = (byte[..., 16 + 32 * (j // 2) + e % 32] >> (4 * (j % 2))) & 15
        lo = j < 4
        jj = j % 4
        sc = torch.where(lo, byte[..., 4 + jj] & 63, (byte[..., 12 + jj] & 15) + (byte[..., 4 + jj] >> 6) * 16)
        mn = torch.where(lo, byte[..., 8 + jj] & 63, (byte[..., 12 + jj] >> 4) + (byte[..., 8 + jj] >> 6) * 16)
        y = f16(0) * sc * code - f16(2) * mn
    else:
        h, r, x = e // 128, e // 32 % 4, e % 32
        low = (byte[..., 64 * h + 32 * (r % 2) + x] >> (4 * (r // 2))) & 15
        high = (byte[..., 128 + 32 * h + x] >> (2 * r)) & 3
        sc = byte[..., 192 + e // 16]
        y = f16(208) * torch.where(sc > 127, sc - 256, sc) * (low + 16 * high - 32)
    return y.reshape(s["T"], s["K"]) * s["scale"]


def _exact_rope(s):
    rot = s["rot"]
    out = []
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"].double()[:, None] * s["freq"].double())[:, None]
    for x, w, y in ((s["q"], s["qw"], s["qo"]), (s["k"], s["kw"], s["ko"])):
        z = x.double()
        if w is not None:
            z = z / (z.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * w.double()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        c = torch.complex(z[..., first].contiguous(), z[..., second].contiguous()) * turn
        z = z.clone()
        z[..., first], z[..., second] = c.real, c.imag
        out.append(torch.where(s["pos"][:, None, None] >= 0, z, y.double()))
    return out


def _exact_prefix(s):
    G, bs = s["Hq"] // s["Hkv"], s["bs"]
    start, kv = s["q_start"].tolist(), s["kv_len"].tolist()
    out = torch.zeros(s["T"], s["Hq"], s["D"], dtype=torch.float64, device=DEV)
    for r in range(s["R"]):
        ids = s["table"][r, :-(-kv[r] // bs)].long()
        n = start[r + 1] - start[r]
        pos = torch.arange(kv[r] - n, kv[r], device=DEV)[:, None]
        col = torch.arange(kv[r], device=DEV)[None, :]
        hide = col > pos
        if s["window"]:
            hide |= col <= pos - s["window"]
        for h in range(s["Hkv"]):
            k = (s["kc"][ids, h].double() * s["ks"][ids, h].double()[:, None, None]).flatten(0, 1)[:kv[r]]
            v = (s["vc"][ids, h].double() * s["vs"][ids, h].double()[:, None, None]).flatten(0, 1)[:kv[r]]
            q = s["q"][start[r]:start[r + 1], h * G:(h + 1) * G].double().transpose(0, 1)  # [G, n, D]
            e = (q @ k.T) * s["scale"]
            e.masked_fill_(hide, -math.inf)
            out[start[r]:start[r + 1], h * G:(h + 1) * G] = (torch.softmax(e, -1) @ v).transpose(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "rope": _exact_rope, "prefix": _exact_prefix}[case["op"]](s)
