"""Refusals of the serving operators: what the host checks before any launch,
so these run without a GPU."""
import ctypes

import pytest

import quantized_weight_block_gb300 as ndq

OK, NULL, NEGATIVE, BAD_DTYPE, WORKSPACE, BAD_ARG, MISALIGNED = 0, 1, 5, 9, 10, 15, 16
F32, F16, BF16, DOUBLE = ndq.NDQ_FLOAT, ndq.NDQ_FLOAT16, ndq.NDQ_BFLOAT16, ndq.NDQ_DOUBLE
P = 4096  # a pointer that is never followed


def cache(**kw):
    a = dict(k=P, v=P, k_scale=P, v_scale=P, num_blocks=10, kv_heads=2, block_size=16, head_dim=128,
             code_type=ndq.NDQ_FLOAT8E4M3FN) | kw
    return ndq.ndq_kv_cache(*(a[f] for f, _ in ndq.ndq_kv_cache._fields_))


BAD_CACHES = [(dict(k=0), NULL), (dict(v=0), NULL), (dict(k_scale=0), NULL), (dict(v_scale=0), NULL),
              (dict(code_type=F16), BAD_DTYPE), (dict(block_size=8), BAD_ARG), (dict(block_size=48), BAD_ARG),
              (dict(block_size=256), BAD_ARG), (dict(head_dim=96), BAD_ARG), (dict(kv_heads=0), BAD_ARG),
              (dict(num_blocks=0), BAD_ARG), (dict(num_blocks=1 << 31), BAD_ARG), (dict(k=P + 8), MISALIGNED),
              (dict(v=P + 1), MISALIGNED), (dict(k_scale=P + 2), MISALIGNED)]


def plan(**kw):
    a = dict(cached=P, fresh=P, n_req=3, block_size=16, free_blocks=P, free_count=P, block_table=P, table_width=4,
             q_start=P, kv_len=P, positions=P, slots=P, n_tokens=3, free_left=P + 4) | kw
    return ndq.ndq_kv_plan(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(n_req=-1), NEGATIVE), (dict(n_tokens=-1), NEGATIVE), (dict(table_width=-1), NEGATIVE),
    (dict(block_size=24), BAD_ARG), (dict(block_size=0), BAD_ARG), (dict(n_req=1 << 31), BAD_ARG),
    (dict(cached=0), NULL), (dict(fresh=0), NULL), (dict(free_blocks=0), NULL), (dict(free_count=0), NULL),
    (dict(block_table=0), NULL), (dict(q_start=0), NULL), (dict(kv_len=0), NULL), (dict(positions=0), NULL),
    (dict(slots=0), NULL), (dict(free_left=0), NULL), (dict(free_left=P), BAD_ARG), (dict(slots=P + 4), MISALIGNED),
    (dict(cached=P + 2), MISALIGNED)])
def test_plan_refusals(kw, want):
    assert plan(**kw) == want


def append(c=None, **kw):
    a = dict(k=P, v=P, in_dtype=BF16, k_stride=256, v_stride=256, slots=P, n_tokens=3) | kw
    return ndq.ndq_kv_append(c or cache(), **a)


@pytest.mark.parametrize("kw,want", [
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(slots=0), NULL), (dict(in_dtype=F32), BAD_DTYPE),
    (dict(n_tokens=-1), NEGATIVE), (dict(k_stride=255), BAD_ARG), (dict(v_stride=-256), BAD_ARG),
    (dict(k_stride=260), MISALIGNED), (dict(k=P + 2), MISALIGNED), (dict(v=P + 8), MISALIGNED), (dict(slots=P + 4), MISALIGNED),
    (dict(n_tokens=0, k=0, v=0, slots=0), OK)])
def test_append_refusals(kw, want):
    assert append(**kw) == want


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_refusals(kw, want):
    assert append(cache(**kw)) == want
    assert attend(cache(**kw)) == want


def attend(c=None, **kw):
    a = dict(q=P, dtype=BF16, n_tokens=3, q_heads=8, q_stride=1024, block_table=P, table_width=4, kv_len=P, q_start=P,
             n_req=2, max_q=3, scale=1.0, window=0, out=P, lse=0, workspace=P,
             ws_bytes=ndq.ndq_attention_workspace_bytes(128)) | kw
    return ndq.ndq_attention_kv8(c or cache(), **a)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), NULL), (dict(out=0), NULL), (dict(kv_len=0), NULL), (dict(block_table=0), NULL),
    (dict(dtype=F32), BAD_DTYPE), (dict(n_tokens=-1), NEGATIVE), (dict(n_req=-1), NEGATIVE), (dict(max_q=-1), NEGATIVE),
    (dict(window=-1), NEGATIVE), (dict(table_width=-1), NEGATIVE), (dict(q_heads=0), BAD_ARG), (dict(q_heads=7), BAD_ARG),
    (dict(table_width=1 << 27), BAD_ARG), (dict(n_tokens=1 << 29), BAD_ARG), (dict(scale=float("nan")), BAD_ARG),
    (dict(scale=float("inf")), BAD_ARG), (dict(q_start=0), BAD_ARG), (dict(q_stride=1016), BAD_ARG),
    (dict(q_stride=1028), MISALIGNED), (dict(q=P + 2), MISALIGNED), (dict(out=P + 8), MISALIGNED),
    (dict(lse=P + 2), MISALIGNED), (dict(workspace=0), WORKSPACE), (dict(workspace=P + 8), WORKSPACE),
    (dict(ws_bytes=ndq.ndq_attention_workspace_bytes(128) - 1), WORKSPACE), (dict(n_tokens=0), OK), (dict(n_req=0), OK),
    (dict(max_q=0), OK)])
def test_attention_refusals(kw, want):
    assert attend(**kw) == want


def test_workspace_sizes():
    assert ndq.ndq_attention_workspace_bytes(96) == 0
    assert 0 < ndq.ndq_attention_workspace_bytes(64) < ndq.ndq_attention_workspace_bytes(128)
    assert ndq.ndq_lora_workspace_bytes(-1, 8, 64) == 0
    assert ndq.ndq_lora_workspace_bytes(4, 0, 64) == 0 and ndq.ndq_lora_workspace_bytes(4, 129, 64) == 0
    assert ndq.ndq_lora_workspace_bytes(4, 8, 64) >= 4 * 8 * 4


def lora(**kw):
    a = dict(x=P, M=3, K=64, lora_a=P, lora_b=P, n_adapters=2, max_rank=8, N=32, ranks=P, scales=P, index=P, base=P,
             dtype=F32, y=P, workspace=P, ws_bytes=1 << 30) | kw
    return ndq.ndq_lora_add(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(x=0), NULL), (dict(lora_a=0), NULL), (dict(lora_b=0), NULL), (dict(ranks=0), NULL), (dict(scales=0), NULL),
    (dict(index=0), NULL), (dict(base=0), NULL), (dict(y=0), NULL), (dict(dtype=DOUBLE), BAD_DTYPE),
    (dict(dtype=F16), BAD_DTYPE), (dict(M=-1), NEGATIVE), (dict(K=-1), NEGATIVE), (dict(N=-1), NEGATIVE),
    (dict(n_adapters=-1), NEGATIVE), (dict(max_rank=0), BAD_ARG), (dict(max_rank=129), BAD_ARG), (dict(N=1 << 31), BAD_ARG),
    (dict(x=P + 1), MISALIGNED), (dict(y=P + 2), MISALIGNED), (dict(ranks=P + 2), MISALIGNED), (dict(workspace=0), WORKSPACE),
    (dict(workspace=P + 4), WORKSPACE), (dict(ws_bytes=8), WORKSPACE), (dict(M=0), OK), (dict(N=0), OK)])
def test_lora_refusals(kw, want):
    assert lora(**kw) == want


def test_descriptor_layout_matches_the_header():
    assert ctypes.sizeof(ndq.ndq_kv_cache) == 4 * 8 + 8 + 4 * 4


def test_append_launch_limit():
    rows = dict(k_stride=4096 * 128, v_stride=4096 * 128)
    assert append(cache(kv_heads=4096), n_tokens=(1 << 21) + 1, **rows) == BAD_ARG


PLAN_PARTS = {"cached": 12, "fresh": 12, "free_blocks": 4, "free_count": 4, "block_table": 48, "q_start": 16, "kv_len": 12, "positions": 20,
              "slots": 40, "free_left": 4}  # bytes, for 3 requests, a table of width 4 and 5 tokens
PLAN_OUTPUTS = ("block_table", "q_start", "kv_len", "positions", "slots", "free_left")


@pytest.mark.parametrize("out", PLAN_OUTPUTS)
@pytest.mark.parametrize("other", PLAN_PARTS)
def test_plan_outputs_over_other_arrays_are_refused(out, other):
    if out == other:
        return
    apart = {n: P * (i + 1) for i, n in enumerate(PLAN_PARTS)}
    step = 8 if "slots" in (out, other) else 4
    # the same place, the output's last element on the other's first, its first on the other's last
    for shift in (0, -(PLAN_PARTS[out] - step) // step * step, (PLAN_PARTS[other] - 1) // step * step):
        assert plan(n_req=3, table_width=4, n_tokens=5, **(apart | {out: apart[other] + shift})) == BAD_ARG


def test_failure_path_requests():
    for limit in (1, 999, 2000001):
        assert ndq.ndq_test_lose_copies(limit) == 13
    assert ndq.ndq_test_lose_copies(1000) == OK and ndq.ndq_test_lose_copies(0) == OK  # (cancelled)
