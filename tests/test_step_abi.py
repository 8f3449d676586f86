"""Refusals of the packed embedding lookup, of the norm and rotation of heads
and of attention behind shared prefixes: what the host checks before any launch,
so these run without a GPU."""
import pytest
import torch

import quantized_weight_block_gb300 as ndq
from test_serving_abi import BAD_CACHES, cache
from test_serving_binding import On, attend_args, on_gpu

OK, NULL, UNKNOWN, NEGATIVE, BLOCKS, LENGTH, BAD_DTYPE, WORKSPACE, BAD_ARG, MISALIGNED = 0, 1, 2, 5, 6, 7, 9, 10, 15, 16
F32, F16, BF16, DOUBLE = ndq.NDQ_FLOAT, ndq.NDQ_FLOAT16, ndq.NDQ_BFLOAT16, ndq.NDQ_DOUBLE
P = 4096  # a pointer that is never followed
Q8, FP8 = ndq.format_id("gguf:q8_0"), ndq.format_id("fp8_e4m3fn_row_bf16")


def embed(**kw):
    a = dict(format_id=Q8, V=10, K=64, w=P, w_len=10 * 2 * 34, ids=P, ids_dtype=ndq.NDQ_INT32, n_tokens=3, scale=1.0,
             out_dtype=BF16, y=P, y_stride=64) | kw
    return ndq.ndq_embed_packed(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(format_id=99), UNKNOWN), (dict(format_id=-1), UNKNOWN), (dict(V=-1), NEGATIVE), (dict(K=-32), NEGATIVE),
    (dict(n_tokens=-1), NEGATIVE), (dict(K=48), BLOCKS), (dict(w_len=679), LENGTH), (dict(V=11), LENGTH),
    (dict(format_id=FP8, K=24, w_len=10 * 26), BLOCKS), (dict(out_dtype=DOUBLE), BAD_DTYPE), (dict(out_dtype=0), BAD_DTYPE),
    (dict(ids_dtype=F32), BAD_DTYPE), (dict(w=0), NULL), (dict(ids=0), NULL), (dict(y=0), NULL), (dict(y_stride=63), BAD_ARG),
    (dict(y_stride=-64), BAD_ARG), (dict(y_stride=1 << 41), BAD_ARG), (dict(scale=float("nan")), BAD_ARG),
    (dict(scale=float("inf")), BAD_ARG), (dict(n_tokens=1 << 31), BAD_ARG), (dict(y=P + 1), MISALIGNED),
    (dict(out_dtype=F32, y=P + 2), MISALIGNED), (dict(ids=P + 2), MISALIGNED), (dict(ids_dtype=ndq.NDQ_INT64, ids=P + 4), MISALIGNED),
    (dict(n_tokens=0), OK), (dict(K=0, w_len=0, y_stride=0), OK), (dict(n_tokens=0, ids=0, y=0), OK)])
def test_embed_refusals(kw, want):
    assert embed(**kw) == want


def rope(**kw):
    a = dict(q=P, q_heads=8, q_stride=1024, k=P, k_heads=2, k_stride=256, in_dtype=BF16, n_tokens=3, head_dim=128, rot_dim=128,
             interleaved=0, positions=P, inv_freq=P, q_weight=P, k_weight=P, eps=1e-6, q_out=2 * P, q_out_stride=1024,
             k_out=2 * P, k_out_stride=256, out_dtype=BF16) | kw
    return ndq.ndq_qk_norm_rope(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(n_tokens=-1), NEGATIVE), (dict(q_heads=-1), NEGATIVE), (dict(k_heads=-1), NEGATIVE), (dict(in_dtype=DOUBLE), BAD_DTYPE),
    (dict(out_dtype=F32), BAD_DTYPE), (dict(head_dim=0), BAD_ARG), (dict(head_dim=120), BAD_ARG), (dict(head_dim=272), BAD_ARG),
    (dict(rot_dim=-16), BAD_ARG), (dict(rot_dim=144), BAD_ARG), (dict(rot_dim=24), BAD_ARG), (dict(interleaved=2), BAD_ARG),
    (dict(eps=-1e-6), BAD_ARG), (dict(eps=float("nan")), BAD_ARG), (dict(n_tokens=1 << 31), BAD_ARG), (dict(q_heads=4097), BAD_ARG),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(q_out=0), NULL), (dict(k_out=0), NULL), (dict(positions=0), NULL),
    (dict(inv_freq=0), NULL), (dict(q_stride=1016), BAD_ARG), (dict(k_out_stride=255), BAD_ARG), (dict(q_stride=1028), MISALIGNED),
    (dict(k=P + 8), MISALIGNED), (dict(q_out=P + 2), MISALIGNED), (dict(positions=P + 2), MISALIGNED),
    (dict(k_weight=P + 1), MISALIGNED), (dict(in_dtype=F32, q_out=P), BAD_ARG), (dict(k_out=P, k_out_stride=512), BAD_ARG),
    (dict(n_tokens=0), OK), (dict(q_heads=0, k_heads=0, q=0, k=0), OK)])
def test_rope_refusals(kw, want):
    assert rope(**kw) == want


def bytes_for(n=3, heads=8, kv=2, D=128):
    return ndq.ndq_attention_prefix_workspace_bytes(D, n, heads, kv)


def prefix(c=None, **kw):
    a = dict(q=P, dtype=BF16, n_tokens=3, q_heads=8, q_stride=1024, block_table=P, table_width=4, kv_len=P, q_start=P, n_req=2, max_q=3,
             group_start=P, prefix_len=P, n_groups=1, scale=1.0, window=0, out=P, lse=0, workspace=P, ws_bytes=bytes_for()) | kw
    return ndq.ndq_attention_prefix_kv8(c or cache(), **a)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), NULL), (dict(out=0), NULL), (dict(kv_len=0), NULL), (dict(block_table=0), NULL), (dict(group_start=0), NULL),
    (dict(prefix_len=0), NULL), (dict(n_groups=-1), NEGATIVE), (dict(n_groups=1 << 31), BAD_ARG), (dict(dtype=F32), BAD_DTYPE),
    (dict(n_tokens=-1), NEGATIVE), (dict(n_req=-1), NEGATIVE), (dict(max_q=-1), NEGATIVE), (dict(window=-1), NEGATIVE),
    (dict(table_width=-1), NEGATIVE), (dict(q_heads=0), BAD_ARG), (dict(q_heads=7), BAD_ARG), (dict(table_width=1 << 27), BAD_ARG),
    (dict(n_tokens=1 << 29), BAD_ARG), (dict(scale=float("nan")), BAD_ARG), (dict(q_start=0), BAD_ARG), (dict(q_stride=1016), BAD_ARG),
    (dict(q_stride=1028), MISALIGNED), (dict(q=P + 2), MISALIGNED), (dict(out=P + 8), MISALIGNED), (dict(lse=P + 2), MISALIGNED),
    (dict(group_start=P + 2), MISALIGNED), (dict(prefix_len=P + 1), MISALIGNED), (dict(workspace=0), WORKSPACE),
    (dict(workspace=P + 128), WORKSPACE), (dict(ws_bytes=bytes_for() - 1), WORKSPACE), (dict(n_tokens=0), OK), (dict(n_req=0), OK),
    (dict(max_q=0), OK)])
def test_prefix_refusals(kw, want):
    assert prefix(**kw) == want


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_prefix_cache_refusals(kw, want):
    assert prefix(cache(**kw)) == want


def test_prefix_workspace_sizes():
    assert bytes_for(D=96) == bytes_for(n=-1) == bytes_for(heads=0) == bytes_for(kv=0) == bytes_for(heads=7) == bytes_for(n=1 << 29) == 0
    assert ndq.ndq_attention_workspace_bytes(128) < bytes_for(n=0) < bytes_for(n=1) < bytes_for(n=2)
    # records and parts of every row, and of 192 units more
    assert bytes_for(n=1000) >= 1000 * 8 * (16 + 130 * 4) + 192 * 256 * 130 * 4


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,heads,kv", [(1, 1, 1), (7, 8, 2), (64, 32, 8), (1000, 40, 8), (16001, 64, 8)])
def test_prefix_workspace_holds_every_part(D, n, heads, kv):
    # a part: D values, maximum, sum and two words to make rows of 16 bytes; a
    # record of 16 and one of 8 bytes a row.  Parts: two a row of the prefix (units of 128 rows and
    # fewer), 256 rows for each of 192 CTAs beyond one a unit; one a row of the
    # own tokens, 16 rows for each of 8 warps of 512 CTAs beyond one a row tile.
    rows, part = n * heads, 4 * (D + 4)
    need = rows * (16 + 8) + part * (2 * rows + 192 * 256) + part * (rows + 512 * 8 * 16)
    got = ndq.ndq_attention_prefix_workspace_bytes(D, n, heads, kv)
    assert 0 <= got - ndq.ndq_attention_workspace_bytes(D) - need <= 4 * 256  # (and each region on 256 bytes)


# ---- the tensor calls -----------------------------------------------------------

BF, I32 = torch.bfloat16, torch.int32


def embed_args():
    return dict(fmt="gguf:q8_0", w=torch.zeros(680, dtype=torch.uint8), V=10, K=64, ids=torch.zeros(3, dtype=I32), out=torch.zeros(3, 64))


def rope_args():
    return dict(q=torch.zeros(3, 4, 64, dtype=BF), k=torch.zeros(3, 2, 64, dtype=BF), positions=torch.zeros(3, dtype=I32),
                inv_freq=torch.zeros(32), q_weight=torch.ones(64), k_weight=torch.ones(64), q_out=torch.zeros(3, 4, 64, dtype=BF),
                k_out=torch.zeros(3, 2, 64, dtype=BF))


def prefix_args():
    return attend_args() | dict(group_start=torch.tensor([0, 2], dtype=I32), prefix_len=torch.tensor([16], dtype=I32))


CALLS = {"embed_packed": embed_args, "qk_norm_rope": rope_args, "attention_prefix_kv8": prefix_args}


@pytest.fixture
def launches(monkeypatch):
    """The library's calls, which must not come."""
    seen = []
    for name in CALLS:
        monkeypatch.setattr(ndq._lib, "ndq_" + name, lambda *a, name=name: (seen.append(name), 0)[1])
    monkeypatch.setattr(ndq, "_raw_stream", lambda stream, device: 0)
    return seen


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_the_device_are_taken(name, launches):
    getattr(ndq, name)(**on_gpu(CALLS[name]()))
    assert launches == [name]


@pytest.mark.parametrize("elsewhere", [-1, 1])
@pytest.mark.parametrize("name,arg", [(n, a) for n, f in CALLS.items() for a, v in f().items() if isinstance(v, torch.Tensor)])
def test_a_tensor_elsewhere_is_refused(name, arg, elsewhere, launches):
    args = on_gpu(CALLS[name]())
    args[arg] = On.at(args[arg], elsewhere)
    with pytest.raises(ValueError):
        getattr(ndq, name)(**args)
    assert launches == []


@pytest.mark.parametrize("name,change", [
    ("embed_packed", dict(ids=torch.zeros(3, 1, dtype=I32))), ("embed_packed", dict(ids=torch.zeros(3))),
    ("embed_packed", dict(ids=torch.zeros(6, dtype=I32)[::2])), ("embed_packed", dict(out=torch.zeros(2, 64))),
    ("embed_packed", dict(out=torch.zeros(64, 3).t())), ("embed_packed", dict(out=torch.zeros(3, 64, dtype=torch.float64))),
    ("embed_packed", dict(w=torch.zeros(680, dtype=torch.int8))), ("embed_packed", dict(out_dtype=BF)),
    ("qk_norm_rope", dict(q=torch.zeros(3, 4, 64))), ("qk_norm_rope", dict(k=torch.zeros(4, 2, 64, dtype=BF))),
    ("qk_norm_rope", dict(k=torch.zeros(3, 2, 128, dtype=BF))), ("qk_norm_rope", dict(q=torch.zeros(3, 64, 4, dtype=BF).transpose(1, 2))),
    ("qk_norm_rope", dict(positions=torch.zeros(3, dtype=torch.int64))), ("qk_norm_rope", dict(positions=torch.zeros(2, dtype=I32))),
    ("qk_norm_rope", dict(inv_freq=torch.zeros(32, dtype=torch.float64))), ("qk_norm_rope", dict(q_weight=torch.ones(64, dtype=BF))),
    ("qk_norm_rope", dict(k_weight=torch.ones(32))), ("qk_norm_rope", dict(q_out=torch.zeros(3, 4, 64))),
    ("qk_norm_rope", dict(k_out=torch.zeros(3, 2, 32, dtype=BF))), ("qk_norm_rope", dict(k=None)),
    ("qk_norm_rope", dict(q=None, k=None)), ("attention_prefix_kv8", dict(group_start=torch.zeros(3, dtype=I32))),
    ("attention_prefix_kv8", dict(group_start=torch.zeros(2, dtype=torch.int64))), ("attention_prefix_kv8", dict(prefix_len=torch.tensor(16, dtype=I32))),
    ("attention_prefix_kv8", dict(prefix_len=torch.zeros(1, 1, dtype=I32))), ("attention_prefix_kv8", dict(prefix_len=torch.zeros(1))),
    ("attention_prefix_kv8", dict(group_start=torch.zeros(4, dtype=I32)[::2])), ("attention_prefix_kv8", dict(lse=torch.zeros(3, 5))),
    ("attention_prefix_kv8", dict(workspace=torch.zeros(64, dtype=torch.uint8)[::2]))])
def test_other_tensors_are_refused(name, change, launches):
    args = on_gpu(CALLS[name]() | change)
    with pytest.raises(ValueError):
        getattr(ndq, name)(**args)
    assert launches == []


# ---- outputs over inputs: refused before any launch ------------------------------

Q, K_, Q_OUT, K_OUT, POS, FREQ, QW, KW = (i << 20 for i in range(1, 9))  # far apart


def apart(**kw):
    return rope(**dict(q=Q, k=K_, q_out=Q_OUT, k_out=K_OUT, positions=POS, inv_freq=FREQ, q_weight=QW, k_weight=KW) | kw)


ROW, KROW = 8 * 128 * 2, 2 * 128 * 2  # bytes of a token's heads


@pytest.mark.parametrize("kw", [
    dict(q_out=Q + 16), dict(q_out=Q + 3 * ROW - 16), dict(q_out=Q - 3 * ROW + 16), dict(q_out=K_), dict(q_out=K_ + 3 * KROW - 16),
    dict(k_out=Q), dict(k_out=K_ + KROW), dict(k_out=Q_OUT), dict(k_out=Q_OUT + 3 * ROW - 16), dict(k_out=Q_OUT - 3 * KROW + 16),
    dict(q_out=POS), dict(k_out=POS - 3 * KROW + 16), dict(q_out=FREQ + 240), dict(k_out=FREQ), dict(q_out=QW + 496), dict(k_out=QW), dict(q_out=KW),
    dict(k_out=KW), dict(q_out=Q, in_dtype=F32, q_stride=2048), dict(q=Q, q_out=Q, k=Q + 16, k_out=K_OUT),
    # rows of one buffer: the same stride and heads that meet, other strides
    dict(q_stride=1536, k=Q + ROW - 16, k_stride=1536, q_out=Q, q_out_stride=1536), dict(q_stride=1536, q_out=Q + ROW, q_out_stride=1536),
    dict(q_stride=4096, q_out=Q + ROW, q_out_stride=1536), dict(q_stride=4096, q_out=Q + ROW, q_out_stride=3584),
    dict(in_dtype=F32, q_stride=2048, q_out=Q + 4096, q_out_stride=2048)])
def test_rope_outputs_over_inputs_are_refused(kw):
    assert apart(**kw) == BAD_ARG


W, IDS, Y = 1 << 20, 2 << 20, 3 << 20


@pytest.mark.parametrize("kw", [
    dict(y=W), dict(y=W + 678), dict(y=W - 3 * 128 + 2), dict(y=IDS), dict(y=IDS - 126), dict(y=IDS + 8), dict(y=IDS - 256, y_stride=128, n_tokens=3),
    dict(y=IDS - 2 * 65536 - 64, y_stride=32768), dict(y=IDS + 20, ids_dtype=ndq.NDQ_INT64), dict(out_dtype=F32, y=IDS - 764)])
def test_embed_outputs_over_inputs_are_refused(kw):
    assert embed(**dict(w=W, ids=IDS, y=Y) | kw) == BAD_ARG
