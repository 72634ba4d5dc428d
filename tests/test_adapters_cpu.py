"""Refusals of the adapters' and the rotated append's entry points that are
decided on the host, without a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import deepseek_v4_flash_gb300 as ds4
    return ds4.lib()


@pytest.mark.parametrize("bad,status", [
    (dict(n_out=0), 1), (dict(n_out=(1 << 24) + 1), 1), (dict(n_in=0), 1), (dict(n_in=48), 1), (dict(n_in=(1 << 16) + 32), 1),
    (dict(slots=0), 1), (dict(slots=4097), 2), (dict(rank=0), 1), (dict(rank=257), 2), (dict(dtype=0), 1), (dict(dtype=3), 1),
    (dict(tokens=0), 1), (dict(tokens=65537), 1),
])
def test_adapters_create_refuses(L, bad, status):
    d = dict(n_out=64, n_in=64, slots=2, rank=8, dtype=1, tokens=4)
    d.update(bad)
    h = ctypes.c_void_p(123)
    assert L.ds4moe_adapters_create(d["n_out"], d["n_in"], d["slots"], d["rank"], d["dtype"], d["tokens"], ctypes.byref(h)) == status
    assert not h.value


def test_null_arguments(L):
    assert L.ds4moe_adapters_create(64, 64, 2, 8, 1, 4, None) == 1
    assert L.ds4moe_adapters_set(None, 0, 0, None, None, 1.0, None) == 1
    assert L.ds4moe_adapters_forward(None, None, 0, 0, None, 0, None, 0, None, 0, None) == 1
    assert L.ds4moe_adapters_get_device_error(None, None, None) == 1
    assert L.ds4moe_adapters_device_bytes(None) == 0 and L.ds4moe_adapters_launch_count(None) == 0
    L.ds4moe_adapters_destroy(None)
    assert L.ds4moe_kv_append_rope(None, None, None, None, 0, None, 0, None, 0, None, 0, 0, None, None, 1, 1, None) == 1


def test_rope_wants_device_memory():
    import deepseek_v4_flash_gb300 as ds4
    for bad in (torch.ones(8), torch.ones(8, dtype=torch.float64), [1.0] * 8):
        with pytest.raises(ValueError):
            ds4.Rope(bad)


def test_shared_attention_null_arguments(L):
    assert L.ds4moe_attn_reserve_shared(None, 1) == 1
    assert L.ds4moe_attn_decode_shared(None, None, None, 0, None, None, None, 1, 1, 1, None, 0, None) == 1
