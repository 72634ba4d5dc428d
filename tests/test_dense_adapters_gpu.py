"""Dense.forward(adapters=): what is refused is refused before anything is
enqueued, and an output that it allocates for another stream comes from that
stream's memory."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SLEEP = 100_000_000  # cycles: some 50 ms


def _dense(n_out, n_in, n_tok, adapter_tokens=None):
    import deepseek_v4_flash_gb300 as ds4
    import synth
    dense = ds4.Dense(n_out, n_in, torch.from_numpy(synth.gen_q8_matrix(3, n_out, n_in, 0.05)).cuda(), max_tokens=n_tok)
    h = ds4.Adapters(n_out, n_in, 2, 8, max_tokens=adapter_tokens or n_tok)
    g = torch.Generator().manual_seed(4)
    for s in range(2):
        h.set(s, torch.randn(8, n_in, generator=g).bfloat16().cuda(), torch.randn(n_out, 8, generator=g).bfloat16().cuda())
    return ds4, dense, h, torch.randn(n_tok, n_in, generator=g).cuda()


def test_refused_before_anything_is_enqueued():
    n_out, n_in, n = 96, 128, 10
    ds4, dense, h, x = _dense(n_out, n_in, n, 4)
    slots = torch.zeros(n, dtype=torch.int32).cuda()
    y = torch.full((n, n_out), 3.0).cuda()

    def refused(*args, **kw):
        before = dense.launch_count(), h.launch_count()
        with pytest.raises((ValueError, ds4.Ds4MoeError)):
            dense.forward(*args, adapters=h, **kw)
        assert (dense.launch_count(), h.launch_count()) == before
        torch.cuda.synchronize()
        assert (y == 3).all()
    refused(x, y, slots=slots)  # more tokens than the adapters' handle takes
    refused(x, y, slots=slots[:5], n_tok=5)
    wide = torch.randn(4 * n_in + 1).cuda()
    refused(wide[1:].view(4, n_in), y[:4], slots=slots[:4])  # rows that are not 16-byte aligned
    both = torch.full((4, n_in), 3.0).cuda()
    kept = both.clone()
    refused(both, both.view(-1)[:4 * n_out].view(4, n_out), slots=slots[:4])  # y over x
    refused(both, both.view(-1)[n_in:n_in + 4 * n_out].view(4, n_out)[:3], slots=slots[:3], n_tok=3)
    refused(x[:4], y[:4], slots=slots[:4].cpu())
    refused(x[:4], y[:4], slots=slots[:3])
    refused(x[:4], y[:3], slots=slots[:4])
    assert torch.equal(both, kept)
    assert dense.forward(x[:4], y[:4], adapters=h, slots=slots[:4]) is not None
    assert (y[:4] != 3).any() and (y[4:] == 3).all()
    assert torch.equal(dense.forward(x, y, adapters=h, slots=slots[:3], n_tok=3)[:3], dense.forward(x[:3], adapters=h, slots=slots[:3]))


@pytest.mark.parametrize("with_adapters", [False, True])
@pytest.mark.parametrize("raw", [False, True])
def test_memory_freed_on_the_current_stream(raw, with_adapters):
    """A block of the output's size is freed while the current stream has yet to
    read it: the call on the other stream must not get it."""
    n_out, n_in, n = 4096, 256, 64
    ds4, dense, h, x = _dense(n_out, n_in, n)
    kw = dict(adapters=h, slots=torch.tensor([t % 3 - 1 for t in range(n)], dtype=torch.int32).cuda()) if with_adapters else {}
    want = dense.forward(x, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kept = [torch.empty_like(want) for _ in range(16)]  # noqa: F841 (blocks of the size that were free before)
    held = torch.full_like(want, 7)
    torch.cuda.synchronize()
    where = held.data_ptr()
    torch.cuda._sleep(SLEEP)
    copy = held.clone()  # queued behind the sleep
    del held
    got = dense.forward(x, stream=side.cuda_stream if raw else side, **kw)
    assert got.data_ptr() != where
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and (copy == 7).all()


@pytest.mark.parametrize("with_adapters", [False, True])
@pytest.mark.parametrize("raw", [False, True])
def test_output_dropped_while_the_current_stream_reads_it(raw, with_adapters):
    n_out, n_in, n = 4096, 256, 64
    ds4, dense, h, x = _dense(n_out, n_in, n)
    kw = dict(adapters=h, slots=torch.tensor([t % 3 - 1 for t in range(n)], dtype=torch.int32).cuda()) if with_adapters else {}
    want = dense.forward(x, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if raw else side
    kept = [torch.empty_like(want) for _ in range(16)]  # noqa: F841 (blocks of the size that were free before)
    first = dense.forward(x, stream=s, **kw)
    torch.cuda.current_stream().wait_stream(side)
    where = first.data_ptr()
    torch.cuda._sleep(SLEEP)
    copy = first.clone()
    del first
    second = dense.forward(x, stream=s, **kw)
    assert second.data_ptr() != where
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and torch.equal(second, want)
