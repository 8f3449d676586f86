"""GPU test of the serving kernels' device-side failure path, without a GPU
fault: the host asks for one call whose waits for staged copies expect more
bytes than come (ndq_test_lose_copies), as if the copies had been lost.  The
copies do land, the waits run out after a millisecond, the kernels set their
bits in the fault word and end, and the next call on the same workspace is
complete again.
"""
import numpy as np
import pytest
import torch

from test_gpu_serving import DEV, attend_case, dev32

pytestmark = pytest.mark.gpu

import quantized_weight_block_gb300 as ndq  # noqa: E402

PROMPT, TILES, ROWS = 8, 16, 32  # bits of the fault word
LIMIT_US = 2000


@pytest.fixture(autouse=True)
def _clean_fault_word():
    torch.cuda.synchronize()
    ndq.get_device_fault()
    yield
    ndq.ndq_test_lose_copies(0)
    torch.cuda.synchronize()
    ndq.get_device_fault()


def expire_and_recover(call, bits):
    want = call()
    torch.cuda.synchronize()
    assert ndq.get_device_fault() == 0
    assert ndq.ndq_test_lose_copies(LIMIT_US) == 0
    call()
    torch.cuda.synchronize()
    assert ndq.get_device_fault() == bits
    for _ in range(2):  # the request was for one call
        got = call()
        torch.cuda.synchronize()
        assert ndq.get_device_fault() == 0
        assert torch.equal(got, want)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,n,bits", [([700, 9000, 30], [1, 1, 1], ROWS), ([5000, 300], [4, 3], ROWS), ([2000, 500], [300, 200], PROMPT),
                                       ([3000], [64], PROMPT), ([2000, 1500, 4000], [300, 1, 2], PROMPT | ROWS)])
def test_attention_copies_that_never_land(code, D, kv, n, bits):
    q, kc, ks, vc, vs, table, start = attend_case(kv, n, 8, 2, D, 16, code, torch.bfloat16, 191)
    cache, tt, kl, qs = ndq.KvCache(kc, vc, ks, vs), torch.from_numpy(table).to(DEV), dev32(kv), dev32(start)
    ws = ndq.attention_workspace(len(kv), q.shape[0], 8, cache)

    def call():
        out = ndq.attention_kv8(q, cache, tt, kl, q_start=qs, max_q=max(n), workspace=ws)
        assert int(ws[:4096].count_nonzero()) == 0
        return out

    expire_and_recover(call, bits)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,bits", [(200, 512, TILES), (1500, 8192, TILES), (20, 512, 0)])
def test_adapter_copies_that_never_land(dtype, M, N, bits):
    K, nA, rank = 256, 3, 16
    g = torch.Generator(device=DEV).manual_seed(201)
    x, a, b = (torch.randn(s, device=DEV, generator=g).to(torch.bfloat16) for s in ((M, K), (nA, rank, K), (nA, N, rank)))
    base, index = torch.randn(M, N, device=DEV, generator=g).to(dtype), dev32(np.arange(M) * 7 // M % 4 - 1)
    ranks, scales, ws = dev32([16, 9, 16]), torch.ones(nA, device=DEV), ndq.lora_workspace(M, nA, rank, K)
    expire_and_recover(lambda: ndq.lora_add(x, a, b, ranks, scales, index, base, workspace=ws), bits)
