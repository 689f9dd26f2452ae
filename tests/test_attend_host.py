"""Refusals of the head norms, the cache and attention that need no device, and the codes of 8
bits that the GPU tests hold the cache to."""
import ctypes
import os

import pytest
import torch

from attend_util import coded, e4m3_values, read_back
from lora_adapter_application_amd import binding, build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    binding.load_library()


def test_calls_on_a_null_ctx():
    lib = binding.load_library()
    E = binding.LORA_ERR_INVALID_ARGUMENT
    out = ctypes.c_void_p(1)
    assert lib.lora_norm_rotary_group(None, None, 1, None, None, None, 1e-6, None, None, 0, None) == E
    assert lib.lora_cache_create(None, ctypes.byref(out), 0, 1, 64, 64, 1) == E and not out.value
    assert lib.lora_cache_create(None, None, 0, 1, 64, 64, 1) == E
    assert lib.lora_cache_destroy(None, None) == E
    assert lib.lora_cache_store(None, None, None, None, None, 0, None) == E
    assert lib.lora_cache_load(None, None, None, None, None, 0, None) == E
    assert lib.lora_attend_prepare(None, None, 1, None, None) == E
    assert lib.lora_attend(None, None, None, None, 1.0, None) == E


def test_tensors_on_the_host_and_unknown_kinds():
    with pytest.raises(ValueError):
        binding.AttendBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.lora_cache_create(None, 1, 64, 1, kind="int4")
    with pytest.raises(ValueError):
        binding.lora_cache_store(None, None, None, None, torch.zeros(2, dtype=torch.int32))


def test_codes_of_eight_bits():
    """The oracle's codes against torch's own 8-bit float, at what is representable and at ties."""
    v = e4m3_values()
    assert len(v) == 127 and v[-1] == 448 and v[1] == 2.0 ** -9
    assert torch.equal(v, v.float().to(torch.float8_e4m3fn).double())
    x = torch.cat((v, -v, (v[1:] + v[:-1]) / 2, -(v[1:] + v[:-1]) / 2))[None, :].float()
    codes, scale = coded(x, "fp8")                      # the largest is 448: the scale is 1
    assert scale.item() == 1 and torch.equal(codes, x.to(torch.float8_e4m3fn).double())
    x = torch.arange(-254, 255)[None, :].float() / 2
    codes, scale = coded(x, "int8")
    assert scale.item() == 1 and torch.equal(codes, torch.round(x.double()) + 0.0)
    assert torch.isnan(read_back(torch.tensor([[1.0, float("inf")]]), "int8")).all()
