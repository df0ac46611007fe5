"""Refusals of the decode-step binding that need no GPU: tensors that say they are on one
device or another, which are never followed."""
import pytest
import torch


class Placed(torch.Tensor):
    """A CPU tensor that says it is on a CUDA device."""

    is_cuda = True
    where = 0

    def get_device(self):
        return self.where


def on(device, *shape, dtype=torch.float32):
    t = torch.Tensor._make_subclass(Placed, torch.zeros(shape, dtype=dtype))
    t.where = device
    return t


def tensors(op, device):
    half, i32 = torch.float16, torch.int32
    new = lambda *s, dtype=torch.float32: on(device, *s, dtype=dtype)  # noqa: E731
    cache = (4, 16, 2, 64)
    return {
        "qmv_lora_add": lambda: dict(x=new(3, 64), a=new(2, 8, 64, dtype=half), b=new(2, 32, 8, dtype=half),
                                     adapter=new(3, dtype=i32), scale=new(2), base=new(3, 32), out=new(3, 32),
                                     workspace=new(1 << 20, dtype=torch.uint8)),
        "qmv_rope_append": lambda: dict(qkv=new(3, 6 * 64), positions=new(1, 3, dtype=i32), table=new(9, 32, 2),
                                        axis_of_pair=bytes(32), slots=new(3, dtype=torch.int64),
                                        k_cache=new(*cache, dtype=half), v_cache=new(*cache, dtype=half),
                                        out=new(3, 2, 64, dtype=half)),
        "qmv_prefix_attention": lambda: dict(q=new(2, 1, 4, 64, dtype=half), k_cache=new(*cache, dtype=half),
                                             v_cache=new(*cache, dtype=half), prefix_table=new(2, dtype=i32),
                                             prefix_len=20, own_table=new(2, 1, dtype=i32), own_len=new(2, dtype=i32),
                                             out=new(2, 1, 4, 64, dtype=half), workspace=new(1 << 20, dtype=torch.uint8)),
        "qmv_penalize_logits": lambda: dict(logits=new(2, 100), tokens=new(2, 5, dtype=i32), prompt_len=new(2, dtype=i32),
                                            total_len=new(2, dtype=i32), repetition=new(2), presence=new(2),
                                            frequency=new(2), bias_tokens=new(2, 3, dtype=i32), bias_values=new(2, 3),
                                            mask=new(2, 4, dtype=i32), mask_row=new(2, dtype=i32), out=new(2, 100)),
    }[op]()


OPERATORS = ["qmv_lora_add", "qmv_rope_append", "qmv_prefix_attention", "qmv_penalize_logits"]


@pytest.fixture(autouse=True)
def device_zero(monkeypatch):
    from gemm_qmv_quantize_gb300 import _decode
    monkeypatch.setattr(_decode, "_current_device", lambda: 0)
    monkeypatch.setattr(_decode, "_fn", lambda name: pytest.fail(f"{name} is called"))


@pytest.mark.parametrize("op", OPERATORS)
def test_tensors_on_different_devices(op):
    import gemm_qmv_quantize_gb300 as q
    elsewhere = tensors(op, 1)
    for name, t in elsewhere.items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError, match="cuda:1"):
                getattr(q, op)(**{**tensors(op, 0), name: t})


@pytest.mark.parametrize("op", OPERATORS)
def test_tensors_that_are_not_on_the_current_device(op):
    import gemm_qmv_quantize_gb300 as q
    with pytest.raises(ValueError, match="current device is cuda:0"):
        getattr(q, op)(**tensors(op, 1))


@pytest.mark.parametrize("op", OPERATORS)
def test_tensors_on_the_cpu(op):
    import gemm_qmv_quantize_gb300 as q
    for name, t in tensors(op, 0).items():
        if isinstance(t, torch.Tensor):
            with pytest.raises(ValueError, match="must be a CUDA tensor"):
                getattr(q, op)(**{**tensors(op, 0), name: torch.zeros(t.shape, dtype=t.dtype)})
