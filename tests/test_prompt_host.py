"""What the binding hands to the library for kvq_norm_rope and
kvq_prompt_attention (no GPU is needed: nothing is launched)."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def kvq():
    from sub_byte_quantized_kvq_gb300 import build
    build.build()
    from sub_byte_quantized_kvq_gb300 import kvq as mod
    return mod


@pytest.fixture
def calls(kvq, monkeypatch):
    """A list of (name, arguments): what would have gone to the library (the tensors lie on the host)."""
    seen = []
    monkeypatch.setattr(kvq, "_check_on", lambda *a: None)
    monkeypatch.setattr(kvq, "_call", lambda what, index, stream, *args: seen.append((what, args)))
    return seen


def rows(n, heads, D=64):
    return torch.zeros((n, heads, D), dtype=torch.bfloat16)


@pytest.mark.parametrize("number", [0.5, 1, np.float32(0.5), np.float64(0.5), torch.tensor(0.5)], ids=str)
def test_numbers_of_any_type(kvq, calls, number):
    """The scale and eps are taken as decode attention takes its scale: anything that is a number."""
    cache = kvq.QuantizedKVCache(1, 2, 2, 64, 1, 1, device="cpu")
    kvq.kvq_prompt_attention(cache, rows(6, 4).view(2, 3, 4, 64), rows(6, 2).view(2, 3, 2, 64), rows(6, 2).view(2, 3, 2, 64), number)
    kvq.kvq_norm_rope(cache, rows(6, 4), rows(6, 2), None, None, eps=number)
    assert [what for what, _ in calls] == ["kvq_prompt_attention", "kvq_norm_rope"]
    for what, args in calls:
        types = getattr(kvq.lib(), what).argtypes
        floats = [a for a, t in zip(args, types) if t is ctypes.c_float]
        assert len(floats) == 1 and type(floats[0]) is float and floats[0] == float(number), what


@pytest.mark.parametrize("bad", [-1.0, np.float32(-1), torch.tensor(float("nan"))], ids=str)
def test_an_eps_that_is_not_one(kvq, calls, bad):
    cache = kvq.QuantizedKVCache(1, 2, 2, 64, 1, 1, device="cpu")
    with pytest.raises(ValueError):
        kvq.kvq_norm_rope(cache, rows(6, 4), rows(6, 2), None, None, eps=bad)
    assert not calls


@pytest.mark.parametrize("form", [list, tuple, np.array, lambda x: np.array(x, dtype=np.uint8), torch.tensor,
                                  lambda x: torch.tensor(x, dtype=torch.int32)],
                         ids=["list", "tuple", "int64 array", "uint8 array", "tensor", "int32 tensor"])
def test_axes_of_pairs_in_any_sequence(kvq, calls, form):
    """pair_axis is a sequence of numbers: an array's own bytes, eight for a number, are not its axes."""
    cache, axes = kvq.QuantizedKVCache(1, 2, 2, 64, 1, 1, device="cpu"), [(i * 3) // 32 for i in range(32)]
    kvq.kvq_norm_rope(cache, rows(6, 4), rows(6, 2), torch.zeros((3, 6), dtype=torch.int32), torch.ones(32), pair_axis=form(axes))
    (_, args), = calls
    assert [a for a in args if isinstance(a, bytes)] == [bytes(axes)]
    for bad in (axes[:-1], axes[:-1] + [3], [-1] + axes[1:]):
        with pytest.raises(ValueError):
            kvq.kvq_norm_rope(cache, rows(6, 4), rows(6, 2), torch.zeros((3, 6), dtype=torch.int32), torch.ones(32), pair_axis=bad)
    assert len(calls) == 1
