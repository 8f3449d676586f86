"""GPU test of the serving operators together: in the example's attention layer
(prompts, then generation steps, with adapters) every stage's output is
recorded and checked against its definition on the inputs that the stage got,
with the bounds of the stages' own tests; and the requests' bookkeeping.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from conftest import ROOT
from test_gpu_serving import append_ref, attend_ref, same_codes

pytestmark = pytest.mark.gpu

import quantized_weight_block_gb300 as ndq  # noqa: E402


def _example():
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_layer_stage_by_stage(monkeypatch):
    ex = _example()
    layer = ex.AttentionLayer(num_blocks=40, hidden=512, q_heads=4, kv_heads=2)
    prompts = [37, 5, 100]
    reqs = ex.Requests(3, 40, 12)
    seen = {}

    def record(name):
        fn = getattr(ndq, name)

        def call(*a, **kw):
            before = [x.clone() if isinstance(x, torch.Tensor) else x for x in a]
            if name == "kv_append":
                before += [t.cpu().clone() for t in (layer.cache.k, layer.cache.k_scale, layer.cache.v, layer.cache.v_scale)]
            y = fn(*a, **kw)
            seen.setdefault(name, []).append((before, kw, y.clone() if isinstance(y, torch.Tensor) else y))
            return y

        monkeypatch.setattr(ndq, name, call)

    for name in ("lora_add", "kv_append", "attention_kv8"):
        record(name)
    g = torch.Generator(device="cuda").manual_seed(1)
    for step in range(4):
        fresh = prompts if step == 0 else [1, 1, 1]
        seen.clear()
        plan = reqs.plan(fresh, layer.cache.block_size)
        x = torch.randn(sum(fresh), layer.hidden, device="cuda", generator=g).to(torch.bfloat16)
        adapter = torch.repeat_interleave(torch.tensor([1, -1, 2], dtype=torch.int32, device="cuda"), torch.tensor(fresh, device="cuda"))
        y = layer(x, adapter, plan, reqs.table, max(fresh))
        assert y.shape == (sum(fresh), layer.hidden)
        assert reqs.cached.tolist() == [p + step for p in prompts]
        assert plan.q_start.tolist() == np.concatenate([[0], np.cumsum(fresh)]).tolist()
        # adapters: q, k, v and the output projection
        assert len(seen["lora_add"]) == 4
        for (xs, a, b, ranks, scales, index, base), kw, got in seen["lora_add"]:
            want, bound = base.double(), torch.zeros_like(base, dtype=torch.float64)
            for i, r in enumerate(ranks.tolist()):
                rows = (index == i).nonzero()[:, 0]
                aa, bb, xx = a[i, :r].double(), b[i, :, :r].double(), xs[rows].double()
                want[rows] += float(scales[i]) * (xx @ aa.T) @ bb.T
                bound[rows] += float(scales[i]) * (xs.shape[1] + a.shape[1] + 32) * 2.0 ** -23 * (xx.abs() @ aa.abs().T) @ bb.abs().T
            bound += (2.0 ** -23 if base.dtype == torch.float32 else 2.0 ** -8) * (want.abs() + bound) + 1e-30
            assert ((got.double() - want).abs() <= bound).all()
        # the append: codes and scales bit for bit
        (_, k, v, slots, kc, ks, vc, vs), _, _ = seen["kv_append"][0]
        for x0, c0, s0, c1, s1 in ((k, kc, ks, layer.cache.k, layer.cache.k_scale), (v, vc, vs, layer.cache.v, layer.cache.v_scale)):
            want_c, want_s = append_ref(c0, s0, x0.cpu(), slots.tolist(), 16, "e4m3")
            used = torch.zeros(c0.shape[0], 16, dtype=torch.bool)  # (other places hold whatever was in memory)
            for r, n in enumerate(reqs.cached.tolist()):
                for p in range(n):
                    used[int(reqs.table[r, p // 16]), p % 16] = True
            mask = used[:, None, :, None].expand_as(c0)
            assert same_codes(torch.where(mask, c1.cpu().view(torch.int8), 0).view(torch.float8_e4m3fn),
                              torch.where(mask, want_c.view(torch.int8), 0).view(torch.float8_e4m3fn))
            assert torch.equal(s1.cpu()[used.any(1)], want_s[used.any(1)])
        # attention over what the cache holds
        (q, _, table, kv_len), _, got = seen["attention_kv8"][0]
        c = layer.cache
        want, bound, _ = attend_ref(q, c.k, c.k_scale, c.v, c.v_scale, table.cpu().numpy(), kv_len.tolist(), plan.q_start.tolist(), 16,
                                    128 ** -0.5, 0, torch.bfloat16)
        assert ((got.double() - want).abs() <= bound).all()
    assert ndq.get_device_fault() == 0


def test_example_runs(capsys):
    _example().main()
    assert "free blocks" in capsys.readouterr().out
