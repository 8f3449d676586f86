"""GPU tests of the packed embedding lookup: every format's rows bit for bit
against the oracle's decode, times the scale in binary32, rounded once."""
import zlib

import numpy as np
import pytest
import torch

import synth
from conftest import assert_bit_exact

pytestmark = pytest.mark.gpu

import quantized_weight_block_gb300 as ndq  # noqa: E402

FORMATS = ["gguf:q8_0", "q8_g32_fp16", "gguf:q4_0", "gguf:iq4_nl", "gguf:q4_k", "gguf:q6_k",
           "gguf:mxfp4", "gguf:nvfp4", "nvfp4", "q4_g64_fp16"] + synth.NEXT_FORMATS
OUT = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
DEV = "cuda"


@pytest.fixture(autouse=True)
def _no_device_fault():
    yield
    assert ndq.get_device_fault() == 0


def expected(orc, fmt, shape, x, ids, scale, out):
    w = torch.from_numpy(orc.decode(fmt, shape, x, "float32").reshape(shape).copy())
    ok = (ids >= 0) & (ids < shape[0])
    y = w[torch.where(ok, ids, 0).long()] * torch.tensor(scale, dtype=torch.float32)
    return torch.where(ok[:, None], y, 0.0).to(OUT[out])


def words(x):
    return x.contiguous().cpu().view(torch.uint16 if x.element_size() == 2 else torch.float32).numpy()


def check(orc, fmt, V, K, T, scale=1.0, out="bfloat16", ids_dtype=torch.int32, x_off=0, y_off=0, gap=0, dist="workload", ndiv=1, seed=None):
    seed = zlib.crc32(f"{fmt}{V}{K}{T}".encode()) % 1000 if seed is None else seed
    x = synth.payload(fmt, (V, K), seed=seed, dist=dist, ndiv=ndiv)
    buf = torch.zeros(x.size + x_off + 16, dtype=torch.uint8, device=DEV)
    buf[x_off:x_off + x.size] = torch.from_numpy(x).to(DEV)
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (T,), generator=g).to(ids_dtype)
    if T > 4:
        ids[1], ids[2], ids[3], ids[4] = -1, V, ids[0], V - 1
    whole = torch.full((T * (K + gap) + y_off + 8,), float("nan"), dtype=OUT[out], device=DEV)
    y = whole[y_off:y_off + T * (K + gap)].view(T, K + gap)[:, :K]
    got = ndq.embed_packed(fmt, buf[x_off:x_off + x.size], V, K, ids.to(DEV), scale=scale, out=y)
    torch.cuda.synchronize()
    assert got is y
    assert_bit_exact(words(y), words(expected(orc, fmt, (V, K), x, ids, scale, out)), out, f"{fmt} {V}x{K} {T}")
    rest = torch.ones_like(whole, dtype=torch.bool)
    rest[y_off:y_off + T * (K + gap)].view(T, K + gap)[:, :K] = False
    assert torch.isnan(whole[rest].float()).all()  # what lies around the rows is as it was


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("out", OUT)
def test_rows(orc, fmt, out):
    B, _ = synth.GEOMETRY[fmt]
    for K in (B if B > 16 else 16, 512 + max(B, 16), 4096):  # one block, a short last segment, whole segments
        check(orc, fmt, 24, K, 37, out=out, dist="bytes", ndiv=3 if fmt == "nvfp4" else 1)
    check(orc, fmt, 24, 2048, 37, scale=45.254833, out=out)


@pytest.mark.parametrize("fmt", FORMATS)
def test_unaligned_payloads_and_outputs(orc, fmt):
    K = 768
    for x_off, y_off, gap, out in ((1, 0, 0, "bfloat16"), (2, 1, 0, "float16"), (7, 0, 8, "float32"), (0, 0, 3, "bfloat16"), (0, 5, 0, "float32")):
        check(orc, fmt, 11, K, 9, out=out, x_off=x_off, y_off=y_off, gap=gap, dist="bytes")


@pytest.mark.parametrize("T", [1, 2, 61, 1000, 5003])
@pytest.mark.parametrize("ids_dtype", [torch.int32, torch.int64])
def test_token_counts(orc, T, ids_dtype):
    check(orc, "gguf:q6_k", 301, 1024, T, ids_dtype=ids_dtype, scale=32.0)
    check(orc, "gguf:q8_0", 301, 96, T, ids_dtype=ids_dtype)


def test_far_ids_and_offsets_beyond_32_bits(orc):
    fmt, K, V = "gguf:q8_0", 4096, 520000  # 2.26 GB of payload
    block = synth.payload(fmt, (4, K), seed=3)
    x = torch.zeros(V * K // 32 * 34, dtype=torch.uint8, device=DEV)
    x.view(V, -1)[V - 4:] = torch.from_numpy(block).view(4, -1).to(DEV)
    ids = torch.tensor([V - 1, 0, V - 3, V - 4, 1 << 40, -(1 << 40)], device=DEV)
    y = ndq.embed_packed(fmt, x, V, K, ids, out_dtype=torch.float32)
    want = expected(orc, fmt, (4, K), block, torch.tensor([3, -1, 1, 0, -1, -1]), 1.0, "float32")
    assert_bit_exact(words(y), words(want), "float32")
    # (zero codes of zero scales are zeros, as the rows of ids outside the table)


def test_empty_calls():
    w = torch.zeros(34, dtype=torch.uint8, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert ndq.embed_packed("gguf:q8_0", w, 1, 32, none).shape == (0, 32)
    y = ndq.embed_packed("gguf:q8_0", w[:0], 0, 64, torch.zeros(3, dtype=torch.int32, device=DEV))  # no row at all
    assert y.shape == (3, 64) and not y.any()


def test_captured_and_replayed_with_other_ids(orc):
    fmt, V, K, T = "gguf:q4_k", 50, 1024, 8
    x = synth.payload(fmt, (V, K), seed=1)
    w, ids = torch.from_numpy(x).to(DEV), torch.zeros(T, dtype=torch.int64, device=DEV)
    y = torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
    ndq.embed_packed(fmt, w, V, K, ids, out=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ndq.embed_packed(fmt, w, V, K, ids, out=y)
    for seed in range(3):
        now = torch.randint(-1, V + 1, (T,), generator=torch.Generator().manual_seed(seed))
        ids.copy_(now)
        graph.replay()
        torch.cuda.synchronize()
        assert_bit_exact(words(y), words(expected(orc, fmt, (V, K), x, now, 1.0, "bfloat16")), "bfloat16")


def test_on_another_stream(orc):
    fmt, V, K, T = "gguf:q8_0", 64, 512, 33
    x = synth.payload(fmt, (V, K), seed=2)
    w, ids = torch.from_numpy(x).to(DEV), torch.arange(T, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = ndq.embed_packed(fmt, w, V, K, ids, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert_bit_exact(words(y), words(expected(orc, fmt, (V, K), x, ids.cpu(), 1.0, "bfloat16")), "bfloat16")


FIRST_CALLS = """
import sys, threading
sys.path[:0] = [{root!r}, {tests!r}]
import torch, synth
import quantized_weight_block_gb300 as ndq
from test_gpu_embed import FORMATS
K, T, V = 4096, 300, 24
work = []
for fmt in FORMATS:
    w = torch.from_numpy(synth.payload(fmt, (V, K), seed=1)).cuda()
    work.append((fmt, w, torch.arange(T, device="cuda") % V))
torch.cuda.synchronize()
got, gate = [[None] * len(work) for _ in range(8)], threading.Barrier(8)

def run(i):
    for j, (fmt, w, ids) in enumerate(work):
        gate.wait()
        try:
            got[i][j] = ndq.embed_packed(fmt, w, V, K, ids)
        except Exception as e:
            got[i][j] = e

threads = [threading.Thread(target=run, args=(i,)) for i in range(8)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
for j, (fmt, w, ids) in enumerate(work):
    want = ndq.embed_packed(fmt, w, V, K, ids)
    for i in range(8):
        assert isinstance(got[i][j], torch.Tensor), (fmt, got[i][j])
        assert torch.equal(got[i][j].view(torch.int16), want.view(torch.int16)), fmt
print("ok")
"""


def test_first_calls_of_several_threads_at_once():
    # (in a process of its own, where no format has been asked for yet)
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=os.path.dirname(tests), tests=tests)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-500:] + r.stderr[-1500:]
