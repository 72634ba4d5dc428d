"""Outputs that the binding allocates for a call on another stream: their
memory is neither in use by what the current stream has queued, nor handed on
while the current stream still reads the output."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SLEEP = 100_000_000  # cycles: some 50 ms


def _calls():
    """(name, call(stream) -> outputs, their number of bytes each)."""
    import deepseek_v4_flash_gb300 as ds4
    g = torch.Generator(device="cuda").manual_seed(1)
    heads, dim, n = 64, 128, 512
    pool = torch.randn(2, n // 64, 64, 8, dim, generator=g, device="cuda").bfloat16()
    cache = ds4.KVCache(pool[0], pool[1], torch.arange(n // 64, dtype=torch.int32, device="cuda")[None])
    at = ds4.Attention(ds4.AttentionDesc(heads, 8, dim, max_tokens=n))
    q = torch.randn(n, heads, dim, generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    length = torch.tensor([n], dtype=torch.int32, device="cuda")
    logits = torch.randn(16, 70000, generator=g, device="cuda")
    B, G, V = 3000, 4, 40
    target = torch.softmax(torch.randn(B, G + 1, V, generator=g, device="cuda"), -1)
    draft = torch.softmax(torch.randn(B, G, V, generator=g, device="cuda"), -1)
    tokens = torch.randint(V, (B, G), generator=g, device="cuda", dtype=torch.int32)
    ua, us = torch.rand(B, G, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    torch.cuda.synchronize()
    return {
        "decode": lambda s: [at.decode(cache, q[None, :16], length, stream=s)],
        "prefill": lambda s: [at.prefill(cache, q, cu, length, stream=s)],
        "probs": lambda s: [ds4.token_probs(logits, 0.7, stream=s)],
        "verify": lambda s: list(ds4.verify_drafts(target, draft, tokens, ua, us, stream=s)),
    }


def _raw(stream, raw):
    return stream.cuda_stream if raw else stream


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["decode", "prefill", "probs", "verify"])
def test_memory_freed_on_the_current_stream(name, raw):
    """Blocks of the outputs' sizes are freed while the current stream has yet
    to read them: the call on the other stream must not get them."""
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    held = [torch.full_like(w, 7) for w in want]
    torch.cuda.synchronize()
    where = {t.data_ptr() for t in held}
    torch.cuda._sleep(SLEEP)
    copies = [t.clone() for t in held]  # queued behind the sleep
    held.clear()
    got = call(_raw(side, raw))
    assert not where & {t.data_ptr() for t in got}
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((c == 7).all() for c in copies)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["decode", "prefill", "probs", "verify"])
def test_output_dropped_while_the_current_stream_reads_it(name, raw):
    call = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    first = call(_raw(side, raw))
    torch.cuda.current_stream().wait_stream(side)
    where = {t.data_ptr() for t in first}
    torch.cuda._sleep(SLEEP)
    copies = [t.clone() for t in first]
    first.clear()
    second = call(_raw(side, raw))
    assert not where & {t.data_ptr() for t in second}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
    assert all(torch.equal(a, b) for a, b in zip(second, want))


def test_the_current_stream_given_by_name():
    """The current stream as an argument: the same as none."""
    for name, call in _calls().items():
        want = call(None)
        for s in (torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream):
            assert all(torch.equal(a, b) for a, b in zip(call(s), want)), name
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = call(0)  # the default stream, from another
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
