"""GPU tests of the norm and rotation of heads against the formulas in 64 bits.

The bound.  A norm's sum of squares (16 terms a lane, then up to 4 additions),
its root and the three products are off by at most 32 roundings of 2^-24; a
cosine or sine by 2^-21 (an angle of half a turn at most, rounded to 2^-24 of
itself and to 2^-32 of a turn, and two units of the function); the two products
of a rotation and their sum add less than 2^-22.  Hence
    |out - ref| <= (2^-19 + 2^-21 + 2^-22) (|a| + |b|)  <=  2^-18 (|a| + |b|)
with a, b the exact pair, plus one rounding of the output (2^-8 bfloat16, 2^-11
or 2^-25 binary16).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

import quantized_weight_block_gb300 as ndq  # noqa: E402

DEV = "cuda"
F32, BF, F16 = torch.float32, torch.bfloat16, torch.float16


def reference(x, pos, freq, w, eps, interleaved):
    """(result, size of each value's pair) in 64 bits."""
    z, rot = x.double(), 2 * freq.numel()
    if w is not None:
        z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    f = pos.double()[:, None, None] * freq.double()
    c, s = f.cos(), f.sin()
    size = z.abs()
    out = z.clone()
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = z[..., at[0]], z[..., at[1]]
    out[..., at[0]], out[..., at[1]] = a * c - b * s, a * s + b * c
    size[..., at[0]] = size[..., at[1]] = a.abs() + b.abs()
    return out, size


def compare(got, x, pos, freq, w, eps, interleaved, before):
    want, size = reference(x, pos, freq, w, eps, interleaved)
    bound = 2.0 ** -18 * size
    bound += want.abs().clamp(max=1e300) * (2.0 ** -8 if got.dtype is BF else 2.0 ** -11) + (0 if got.dtype is BF else 2.0 ** -25)
    live = (pos >= 0)[:, None, None].expand_as(want)
    assert torch.equal(got[~live], before[~live])
    err = (got.double() - want).abs()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got)[live], nan[live])
    bad = live & ~nan & ~(err <= bound + 1e-300)
    assert not bad.any(), (bad.nonzero()[:4].tolist(), err[bad][:4].tolist(), bound[bad][:4].tolist())


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEV)


def check(T, Hq, Hk, D, rot, din=BF, dout=BF, norm=True, interleaved=False, far=100000, eps=1e-6, inplace=False, pad=0, seed=0, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    row = (torch.randn(T, Hq + 2 * Hk, D, device=DEV, generator=g) * size).to(din)
    q, k = row[:, :Hq], row[:, Hq:Hq + Hk]
    pos = torch.randint(0, far, (T,), device=DEV, generator=g, dtype=torch.int32)
    if pad:
        pos[-pad:] = -1
    qw, kw = ((1 + 0.3 * torch.randn(D, device=DEV, generator=g)) if norm else None for _ in range(2))
    f = freqs(rot)
    qi, ki, rest = q.clone(), k.clone(), row[:, Hq + Hk:].clone()
    if inplace:
        before = (q.clone(), k.clone())
        out = ndq.qk_norm_rope(q, k, pos, f, qw, kw, eps, interleaved, q_out=q, k_out=k)
    else:
        qo, ko = (torch.randn(T, H, D, device=DEV, generator=g).to(dout) for H in (Hq, Hk))
        before = (qo.clone(), ko.clone())
        out = ndq.qk_norm_rope(q, k, pos, f, qw, kw, eps, interleaved, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    compare(out[0], qi, pos, f, qw, eps, interleaved, before[0])
    compare(out[1], ki, pos, f, kw, eps, interleaved, before[1])
    assert torch.equal(row[:, Hq + Hk:], rest)
    if not inplace:
        assert torch.equal(q, qi) and torch.equal(k, ki)


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 192, 208, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("din", [F32, BF, F16])
def test_head_sizes(D, interleaved, din):
    for rot in {0, 16, D // 32 * 16, D}:
        for norm in (True, False):
            check(5, 7, 3, D, rot, din=din, dout=F16 if din is F16 else BF, norm=norm, interleaved=interleaved, seed=D + rot)


@pytest.mark.parametrize("T,pad", [(1, 0), (2, 1), (64, 3), (133, 0), (2431, 7), (5003, 0)])
@pytest.mark.parametrize("Hq,Hk", [(32, 8), (5, 1), (1, 1), (40, 40)])
def test_token_counts(T, pad, Hq, Hk):
    check(T, Hq, Hk, 128, 128, pad=pad)
    check(T, Hq, Hk, 64, 32, din=F16, dout=F16, interleaved=True, norm=False, pad=pad)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("din", [BF, F16])
def test_in_place(din, interleaved):
    check(77, 8, 2, 128, 64, din=din, dout=din, inplace=True, interleaved=interleaved, pad=4)


def test_every_position_keeps_its_angle():
    # positions to 2^31 - 1: a rotation of (1, 0) is the cosine and sine itself
    pos = torch.tensor([0, 1, 2, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1], dtype=torch.int32, device=DEV)
    for f in (freqs(128), -freqs(128), torch.linspace(0, 1, 64, device=DEV), torch.full((64,), 2.0 ** -140, device=DEV)):
        q = torch.zeros(pos.numel(), 1, 128, device=DEV)
        q[..., :64] = 1.0
        out, _ = ndq.qk_norm_rope(q, None, pos, f, out_dtype=F16)
        a = pos.double()[:, None] * f.double()
        want = torch.cat([a.cos(), a.sin()], 1)
        assert ((out[:, 0].double() - want).abs() <= want.abs() * 2.0 ** -11 + 2.0 ** -21 + 2.0 ** -25).all()


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e18, 1e30])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_large_and_small_magnitudes(size, eps):
    if eps > 0 and size < 1e-20:
        return check(9, 6, 2, 128, 128, din=F32, size=size, eps=1e-30)  # (an eps beside values of that size)
    check(9, 6, 2, 128, 128, din=F32, size=size, eps=eps)
    check(9, 6, 2, 64, 64, din=BF, size=size, eps=eps, interleaved=True)


def test_zeros_infinities_and_nan_stay_in_their_heads():
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(6, 4, 128, device=DEV, generator=g).to(BF)
    clean = q.clone()
    q[0, 0] = 0.0
    q[1, 1, 5] = float("nan")
    q[2, 2, 70] = float("inf")
    pos = torch.arange(6, dtype=torch.int32, device=DEV) * 1000
    f, w = freqs(128), torch.ones(128, device=DEV)
    for weight in (w, None):
        got, _ = ndq.qk_norm_rope(q, None, pos, f, weight)
        other, _ = ndq.qk_norm_rope(clean, None, pos, f, weight)
        touched = torch.zeros(6, 4, dtype=torch.bool, device=DEV)
        touched[0, 0] = touched[1, 1] = touched[2, 2] = True
        assert torch.equal(got[~touched], other[~touched])
        assert not got[0, 0].any()
        if weight is not None:
            assert torch.isnan(got[1, 1]).all()
            assert torch.isnan(got[2, 2, [6, 70]]).all() and not got[2, 2, [5, 7, 69, 71]].any()  # x / inf is 0, inf / inf NaN
        else:
            assert torch.isnan(got[1, 1, [5, 69]]).all() and torch.isfinite(got[1, 1, [4, 6, 68, 70]]).all()


def test_one_side_alone_and_mixed_norms():
    g = torch.Generator(device=DEV).manual_seed(2)
    q, k = (torch.randn(11, H, 64, device=DEV, generator=g).to(BF) for H in (6, 2))
    pos, f = torch.arange(11, dtype=torch.int32, device=DEV), freqs(64)
    w = 1 + 0.1 * torch.randn(64, device=DEV, generator=g)
    both = ndq.qk_norm_rope(q, k, pos, f, w, None)
    qo, none = ndq.qk_norm_rope(q, None, pos, f, w)
    assert none is None and torch.equal(qo, both[0])
    none, ko = ndq.qk_norm_rope(None, k, pos, f)
    assert none is None and torch.equal(ko, both[1])
    compare(both[0], q, pos, f, w, 1e-6, False, both[0])
    compare(both[1], k, pos, f, None, 1e-6, False, both[1])


def test_captured_and_replayed_with_other_positions():
    T = 16
    q, k = torch.randn(T, 8, 128, device=DEV).to(BF), torch.randn(T, 2, 128, device=DEV).to(BF)
    pos, f, w = torch.zeros(T, dtype=torch.int32, device=DEV), freqs(128), torch.ones(128, device=DEV)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    ndq.qk_norm_rope(q, k, pos, f, w, w, q_out=qo, k_out=ko)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ndq.qk_norm_rope(q, k, pos, f, w, w, q_out=qo, k_out=ko)
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        pos.copy_(torch.randint(-1, 100000, (T,), generator=g))
        q.copy_(torch.randn(q.shape, generator=g))
        before = qo.clone(), ko.clone()
        graph.replay()
        torch.cuda.synchronize()
        compare(qo, q, pos, f, w, 1e-6, False, before[0])
        compare(ko, k, pos, f, w, 1e-6, False, before[1])


def test_on_another_stream():
    q = torch.randn(300, 8, 128, device=DEV)
    pos, f = torch.arange(300, dtype=torch.int32, device=DEV), freqs(128)
    want, _ = ndq.qk_norm_rope(q, None, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = ndq.qk_norm_rope(q, None, pos, f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.parametrize("size", [1e-30, 1e-36, 2.0 ** -100])
@pytest.mark.parametrize("eps", [1e-19, 1e-20, 1e-24, 1e-40])
def test_an_eps_far_above_the_squares(size, eps):
    # (the squares vanish in binary32, the eps does not: it is the norm)
    eps = torch.tensor(eps).item()
    check(9, 6, 2, 128, 128, din=F32, size=size, eps=eps)
    check(9, 6, 2, 64, 64, din=BF, size=size, eps=eps, interleaved=True)


@pytest.mark.parametrize("size", [1e18, 1e30])
def test_an_eps_beside_squares_that_overflow(size):
    for eps in (1e-20, 1e30, 3e38):
        check(9, 6, 2, 128, 128, din=F32, size=size, eps=torch.tensor(eps).item())


def turns(pos, freq):
    """pos * freq / (2 pi) modulo 1, in [-1/2, 1/2], rounded once to 64 bits (freq: a binary32 value)."""
    one = 1 << 300

    def atan_of_inverse(n):
        term, total, i = one // n, 0, 0
        while term:
            total += (-1) ** i * (term // (2 * i + 1))
            term //= n * n
            i += 1
        return total

    pi = 4 * (4 * atan_of_inverse(5) - atan_of_inverse(239))
    num, den = float(freq).as_integer_ratio()
    t = pos * num * one * one // (den * 2 * pi) % one
    return (t if t < one // 2 else t - one) / one


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_next_to_multiples_of_a_quarter_turn(interleaved):
    # Sines and cosines near 0 show the angle itself: with bfloat16 outputs they
    # keep 2^-8 of themselves, the angle 2^-31 of a turn, and the functions,
    # their correction and the rotation 2^-20 of the result.  The positions are numerators of
    # convergents of pi (odd and even multiples of half a turn) and their multiples.
    pos = [n * k for n in (355, 103993, 104348, 208341, 312689, 833719, 1146408, 4272943, 5419351, 80143857, 165707065, 245850922, 411557987) for k in (1, 2, 4)
           if n * k < 1 << 31]
    f = torch.tensor([s * 2.0 ** -i for i in range(16) for s in (1, -1)], device=DEV)
    q = torch.zeros(len(pos), 1, 64, device=DEV)
    q[..., 0:64:2] = 1.0
    if not interleaved:
        q = torch.cat([q[..., 0::2], q[..., 1::2]], -1).contiguous()
    out, _ = ndq.qk_norm_rope(q, None, torch.tensor(pos, dtype=torch.int32, device=DEV), f, interleaved=interleaved, out_dtype=BF)
    out = out[:, 0].double()
    got_c, got_s = (out[:, 0::2], out[:, 1::2]) if interleaved else (out[:, :32], out[:, 32:])
    t = torch.tensor([[turns(n, x) for x in f.tolist()] for n in pos], dtype=torch.float64, device=DEV)

    def quarter(t):  # the sine of t turns, of the distance to the nearest half turn where that is small
        n = (2 * t).round()
        return torch.where(n % 2 == 0, 1.0, -1.0) * ((t - n / 2) * 2 * torch.pi).sin()

    for got, want in ((got_s, quarter(t)), (got_c, quarter(t + 0.25))):
        err = (got - want).abs()
        bound = want.abs() * (2.0 ** -8 + 2.0 ** -20) + 2 * torch.pi * 2.0 ** -31
        assert (err <= bound).all(), (float((err / bound).max()), (err > bound).nonzero()[:4].tolist())


def test_inputs_and_outputs_between_one_another_in_one_buffer():
    g = torch.Generator(device=DEV).manual_seed(3)
    row = torch.randn(33, 20, 64, device=DEV, generator=g).to(BF)
    q, k, qo, ko = row[:, :6], row[:, 8:10], row[:, 10:16], row[:, 17:19]
    pos, f, w = torch.arange(33, dtype=torch.int32, device=DEV), freqs(64), torch.ones(64, device=DEV)
    want = ndq.qk_norm_rope(q.clone(), k.clone(), pos, f, w, w)
    rest = row[:, [6, 7, 16, 19]].clone()
    ndq.qk_norm_rope(q, k, pos, f, w, w, q_out=qo, k_out=ko)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]) and torch.equal(row[:, [6, 7, 16, 19]], rest)
    with pytest.raises(ndq.NdqError):
        ndq.qk_norm_rope(q, k, pos, f, w, w, q_out=row[:, 4:10], k_out=ko)


def test_a_head_of_zeros_without_eps():
    q = torch.randn(3, 4, 128, device=DEV).to(BF)
    q[1, 2] = 0.0
    pos, f, w = torch.arange(3, dtype=torch.int32, device=DEV), freqs(128), torch.ones(128, device=DEV)
    none, _ = ndq.qk_norm_rope(q, None, pos, f, w, eps=0.0)  # 0 / 0
    nan = torch.zeros(3, 4, dtype=torch.bool, device=DEV)
    nan[1, 2] = True
    assert none[nan].isnan().all() and torch.isfinite(none[~nan]).all()
    for eps in (1e-6, 1e-20, 1e-44):
        some, _ = ndq.qk_norm_rope(q, None, pos, f, w, eps=eps)
        assert not some[1, 2].any() and torch.isfinite(some).all()
