"""Routing on another stream: ids and weights that the binding allocates come from
that stream's memory."""
import pytest
import torch

import synth
from tests.helpers import lib_desc, make_layer, to_device

pytestmark = pytest.mark.gpu

SLEEP = 100_000_000  # cycles: some 50 ms
TOKENS = 256


def _calls():
    import deepseek_v4_flash_gb300 as ds4
    spec = synth.TINY
    w = synth.gen_layer(spec, 11)
    layer = make_layer(spec, w, TOKENS)
    x = torch.from_numpy(synth.gen_x(spec, 11, TOKENS)).cuda()
    desc, router = lib_desc(spec, TOKENS), to_device({k: w[k] for k in ("router_w", "router_bias") if k in w})
    return {"route": lambda **kw: layer.route(x, **kw), "noalloc": lambda **kw: ds4.route_noalloc(desc, router, x, **kw)}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["route", "noalloc"])
def test_memory_freed_on_the_current_stream(name, raw):
    call = _calls()[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kept = [torch.empty_like(t) for t in want for _ in range(64)]  # noqa: F841 (blocks of the size that were free before)
    held = [torch.full_like(t, 7) for t in want for _ in range(4)]
    torch.cuda.synchronize()
    where = {t.data_ptr() for t in held}
    torch.cuda._sleep(SLEEP)
    copies = [t.clone() for t in held]  # queued behind the sleep
    held.clear()
    got = call(stream=side.cuda_stream if raw else side)
    assert not where & {t.data_ptr() for t in got}
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all((c == 7).all() for c in copies)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["route", "noalloc"])
def test_output_dropped_while_the_current_stream_reads_it(name, raw):
    call = _calls()[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if raw else side
    kept = [torch.empty_like(t) for t in want for _ in range(64)]  # noqa: F841 (blocks of the size that were free before)
    first = list(call(stream=s))
    torch.cuda.current_stream().wait_stream(side)
    where = {t.data_ptr() for t in first}
    torch.cuda._sleep(SLEEP)
    copies = [t.clone() for t in first]
    first.clear()
    second = call(stream=s)
    assert not where & {t.data_ptr() for t in second}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want)) and all(torch.equal(a, b) for a, b in zip(second, want))
