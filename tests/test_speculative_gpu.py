"""The example that runs the operators together: speculative decoding over the
paged cache."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _model(**kw):
    from examples.speculative_decode import Decoder
    return Decoder(**kw)


def _prompts():
    rng = np.random.default_rng(3)
    return [rng.integers(0, 1000, size=n).tolist() for n in (5, 17, 40, 1)]


@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_generate(temperature):
    from examples.speculative_decode import generate
    prompts = _prompts()
    model = _model()
    seqs, drafted, accepted = generate(model, prompts, 24, temperature=temperature)
    for p, s in zip(prompts, seqs):
        assert len(s) >= len(p) + 24 and s[:len(p)] == p and all(0 <= t < 1000 for t in s)
    assert 0 <= accepted <= drafted
    assert not any(model.device_errors())
    # the same numbers give the same tokens
    again, _, _ = generate(_model(), prompts, 24, temperature=temperature)
    assert again == seqs


def test_greedy_tokens_are_the_arg_max_of_their_own_steps():
    """At temperature 0 every token a step keeps is the arg max of the row
    before it, drafted or not."""
    from examples.speculative_decode import generate
    prompts = _prompts()
    model = _model()
    rows = []
    decode = model.decode

    def watched(tokens, kv_len):
        logits = decode(tokens, kv_len)
        rows.append((kv_len.tolist(), tokens.shape[1], logits.argmax(-1).tolist()))
        return logits
    model.decode = watched
    seqs, _, _ = generate(model, prompts, 24, temperature=0.0)
    for step, (lens, n, best) in enumerate(rows):
        nexts = rows[step + 1][0] if step + 1 < len(rows) else [len(s) + n - 1 for s in seqs]
        for b, s in enumerate(seqs):
            start = lens[b] - n + 1  # tokens in the sequence before this step's
            kept = nexts[b] - lens[b]
            assert s[start:start + kept] == best[b][:kept]


def test_decode_and_prefill_agree():
    """The logits after a prompt and after its last tokens fed as one decode
    call: the same positions through two kernels. Both round weights and
    outputs of the attention to bf16, so they differ by its roundings only
    (2^-8 each, through two layers); a routing decision may flip on one, so
    rows are compared by the median over the vocabulary."""
    prompts = _prompts()
    model = _model()
    full = model.prefill(prompts)
    other = _model()
    cut = [p[:max(1, len(p) - 1)] for p in prompts]
    other.prefill(cut)
    last = torch.tensor([[p[-1]] for p in prompts], dtype=torch.int32, device="cuda")
    step = other.decode(last, torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda"))[:, 0]
    err = (full - step).abs().median(dim=1).values / full.abs().median(dim=1).values
    assert (err < 0.05).all(), err
