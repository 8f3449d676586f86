"""Refusals of the serving operators' tensor calls that need no GPU: tensors on
the host, on different devices, or of other dimensions never reach the library.
"""
import pytest
import torch

import quantized_weight_block_gb300 as ndq

BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64
GPU = 0


class On(torch.Tensor):
    """A host tensor that says it lies on another device."""

    @staticmethod
    def at(x, gpu=GPU):
        y = x.as_subclass(On)
        y.gpu = gpu
        return y

    def get_device(self):
        return self.gpu

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        with torch._C.DisableTorchFunctionSubclass():
            return func(*args, **(kwargs or {}))


def cache():
    c = ndq.KvCache.__new__(ndq.KvCache)
    c.num_blocks, c.kv_heads, c.block_size, c.head_dim, c.device, c.gpu = 4, 2, 16, 64, torch.device("cuda", GPU), GPU
    c.desc = ndq.ndq_kv_cache(4096, 4096, 4096, 4096, 4, 2, 16, 64, ndq.NDQ_INT8)
    return c


def plan_args():
    return dict(cached=torch.zeros(3, dtype=I32), fresh=torch.ones(3, dtype=I32), block_size=16, free_blocks=torch.arange(5, dtype=I32),
                free_count=torch.tensor([5], dtype=I32), block_table=torch.full((3, 4), -1, dtype=I32), n_tokens=3)


def append_args():
    return dict(cache=cache(), k=torch.zeros(3, 2, 64, dtype=BF), v=torch.zeros(3, 2, 64, dtype=BF), slots=torch.zeros(3, dtype=I64))


def attend_args():
    return dict(q=torch.zeros(3, 4, 64, dtype=BF), cache=cache(), block_table=torch.zeros(2, 4, dtype=I32), kv_len=torch.ones(2, dtype=I32),
                q_start=torch.tensor([0, 1, 3], dtype=I32), out=torch.zeros(3, 4, 64, dtype=BF), lse=torch.zeros(3, 4),
                workspace=torch.zeros(64, dtype=torch.uint8))


def lora_args():
    return dict(x=torch.zeros(3, 64, dtype=BF), lora_a=torch.zeros(2, 8, 64, dtype=BF), lora_b=torch.zeros(2, 32, 8, dtype=BF),
                ranks=torch.ones(2, dtype=I32), scales=torch.ones(2), index=torch.zeros(3, dtype=I32), base=torch.zeros(3, 32),
                out=torch.zeros(3, 32), workspace=torch.zeros(64, dtype=torch.uint8))


CALLS = {"kv_plan": plan_args, "kv_append": append_args, "attention_kv8": attend_args, "lora_add": lora_args}


@pytest.fixture
def launches(monkeypatch):
    """The library's calls, which must not come."""
    seen = []
    for name in ("ndq_kv_plan", "ndq_kv_append", "ndq_attention_kv8", "ndq_lora_add"):
        monkeypatch.setattr(ndq._lib, name, lambda *a, name=name: (seen.append(name), 0)[1])
    monkeypatch.setattr(ndq, "_raw_stream", lambda stream, device: 0)
    monkeypatch.setattr(ndq, "kv_plan_buffers", lambda R, T, device: ndq.KvPlan(
        *(On.at(torch.zeros(n, dtype=d)) for n, d in ((R + 1, I32), (R, I32), (T, I32), (T, I64), (1, I32)))))
    return seen


def on_gpu(args):
    return {k: On.at(v) if isinstance(v, torch.Tensor) else v for k, v in args.items()}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_the_device_are_taken(name, launches):
    getattr(ndq, name)(**on_gpu(CALLS[name]()))
    assert launches == ["ndq_" + name]


@pytest.mark.parametrize("name", CALLS)
def test_host_tensors_are_refused(name, launches):
    with pytest.raises(ValueError):
        getattr(ndq, name)(**CALLS[name]())
    assert launches == []


@pytest.mark.parametrize("elsewhere", [-1, GPU + 1])
@pytest.mark.parametrize("name,arg", [(n, a) for n, f in CALLS.items() for a, v in f().items() if isinstance(v, torch.Tensor)])
def test_a_tensor_elsewhere_is_refused(name, arg, elsewhere, launches):
    args = on_gpu(CALLS[name]())
    args[arg] = On.at(args[arg], elsewhere)
    with pytest.raises(ValueError):
        getattr(ndq, name)(**args)
    assert launches == []


def test_plan_outputs_elsewhere_are_refused(launches):
    args = on_gpu(plan_args())
    args["out"] = ndq.KvPlan(*(torch.zeros(n, dtype=d) for n, d in ((4, I32), (3, I32), (3, I32), (3, I64), (1, I32))))
    with pytest.raises(ValueError):
        ndq.kv_plan(**args)
    assert launches == []


@pytest.mark.parametrize("name,arg,shape", [
    ("kv_plan", "cached", (3, 2)), ("kv_plan", "fresh", (3, 1)), ("kv_plan", "free_blocks", (5, 1)), ("kv_append", "slots", (3, 1)),
    ("kv_append", "v", (3, 2, 32)), ("kv_append", "k", (2, 2, 64)), ("attention_kv8", "kv_len", (2, 5)), ("attention_kv8", "q_start", (3, 2)),
    ("lora_add", "ranks", (2, 2)), ("lora_add", "scales", (2, 1)), ("lora_add", "index", (3, 7))])
def test_other_dimensions_are_refused(name, arg, shape, launches):
    args = on_gpu(CALLS[name]())
    args[arg] = On.at(torch.zeros(shape, dtype=args[arg].dtype))
    with pytest.raises(ValueError):
        getattr(ndq, name)(**args)
    assert launches == []


def test_a_workspace_with_gaps_is_refused(launches):
    for name in ("attention_kv8", "lora_add"):
        args = on_gpu(CALLS[name]())
        args["workspace"] = On.at(torch.zeros(64, dtype=torch.uint8)[::2])
        with pytest.raises(ValueError):
            getattr(ndq, name)(**args)
    assert launches == []
