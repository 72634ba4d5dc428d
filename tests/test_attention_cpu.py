"""Refusals of the attention and sampling entry points that are decided on
the host, without a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import deepseek_v4_flash_gb300 as ds4
    return ds4.lib()


@pytest.mark.parametrize("bad,status", [
    (dict(n_heads=0), 1), (dict(n_kv_heads=0), 1), (dict(n_heads=7), 1), (dict(n_heads=1), 1), (dict(head_dim=0), 1),
    (dict(head_dim=-64), 1), (dict(head_dim=96), 2), (dict(head_dim=1024), 2), (dict(n_heads=129, n_kv_heads=1), 2),
    (dict(window=-1), 1), (dict(n_sink=-1), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(max_seqs=0), 1), (dict(max_tokens=0), 1),
    (dict(max_seqs=1 << 20), 1), (dict(max_tokens=1 << 21), 1), (dict(dtype="fp32"), 1),
])
def test_attn_create_refuses(L, bad, status):
    import deepseek_v4_flash_gb300 as ds4
    d = dict(n_heads=8, n_kv_heads=2, head_dim=128, dtype="bf16", max_seqs=4, max_tokens=16)
    d.update(bad)
    h = ctypes.c_void_p(123)
    assert L.ds4moe_attn_create(ctypes.byref(ds4.AttentionDesc(**d).c()), ctypes.byref(h)) == status
    assert not h.value


def test_attn_null_arguments(L):
    import deepseek_v4_flash_gb300 as ds4
    d = ds4.AttentionDesc(8, 2, 128).c()
    assert L.ds4moe_attn_create(None, None) == 1
    assert L.ds4moe_attn_create(ctypes.byref(d), None) == 1
    d.abi_version = 99
    h = ctypes.c_void_p()
    assert L.ds4moe_attn_create(ctypes.byref(d), ctypes.byref(h)) == 1
    assert L.ds4moe_kv_append(None, None, None, 0, None, 0, 0, None, None, 1, 1, None) == 1
    assert L.ds4moe_attn_decode(None, None, None, 0, None, 1, 1, None, 0, None) == 1
    assert L.ds4moe_attn_prefill(None, None, None, 0, None, None, 1, 1, None, 0, None) == 1
    assert L.ds4moe_attn_get_device_error(None, None, None) == 1
    assert L.ds4moe_attn_device_bytes(None) == 0 and L.ds4moe_attn_launch_count(None) == 0
    L.ds4moe_attn_destroy(None)


def test_token_probs_refuses(L):
    f = L.ds4moe_token_probs
    buf = ctypes.cast(ctypes.create_string_buffer(64), ctypes.c_void_p)
    assert f(buf, 8, -1, 8, 1.0, buf, 8, None) == 1
    assert f(buf, 8, 1, 0, 1.0, buf, 8, None) == 1
    assert f(buf, 8, 1, (1 << 24) + 1, 1.0, buf, 8, None) == 1
    assert f(buf, 7, 2, 8, 1.0, buf, 8, None) == 1
    for t in (-0.5, float("nan"), float("inf"), 1e-40):
        assert f(buf, 8, 1, 8, t, buf, 8, None) == 1
    assert f(None, 8, 1, 8, 1.0, None, 8, None) == 1
    assert f(buf, 8, 1, 8, 1.0, buf, 8, None) == 1   # host memory
    assert f(None, 8, 0, 8, 1.0, None, 8, None) == 0  # empty is a no-op


def test_verify_refuses(L):
    f = L.ds4moe_verify_drafts
    buf = ctypes.cast(ctypes.create_string_buffer(64), ctypes.c_void_p)

    def call(n_seq=1, g=2, v=8, ts=8, ds=8, p=buf):
        return f(p, ts, p, ds, p, None, p, p, n_seq, g, v, p, p, None, None)
    assert call(n_seq=-1) == 1 and call(g=-1) == 1 and call(g=65) == 1 and call(v=0) == 1
    assert call(ts=7) == 1 and call(ds=7) == 1 and call(p=None) == 1
    assert call() == 1       # host memory
    assert call(n_seq=0) == 0


def test_python_checks():
    import deepseek_v4_flash_gb300 as ds4
    k = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ds4.KVCache(k, k, torch.zeros(1, 2, dtype=torch.int32))   # host memory
    with pytest.raises(ValueError):
        ds4.token_probs(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        ds4.verify_drafts(torch.zeros(1, 3, 8), None, torch.zeros(1, 2).int(), torch.zeros(1, 2), torch.zeros(1))


def test_row_strides():
    """How the binding reads the spacing of rows."""
    import deepseek_v4_flash_gb300 as ds4

    class T(torch.Tensor):  # a host tensor that answers as a device tensor
        is_cuda = True
    t = torch.zeros(3, 5, 4, 8).as_subclass(T)
    assert ds4._rows(t, "t", torch.float32, (4, 8)) == 32
    assert ds4._rows(t[:, :, 1:3], "t", torch.float32, (2, 8)) == 32
    assert ds4._rows(t[:1, :1], "t", torch.float32, (4, 8)) == 32
    for bad in (t[:, :3], t.transpose(0, 1), t[..., ::2], t.transpose(2, 3)):
        with pytest.raises(ValueError):
            ds4._rows(bad, "t", torch.float32, tuple(bad.shape[2:]))
