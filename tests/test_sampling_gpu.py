"""Token probabilities and the verification of drafted tokens on the GPU
against their definitions (64 bits; whole-number arithmetic where a border
decides a token)."""
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu


def _ds4():
    import deepseek_v4_flash_gb300 as ds4
    return ds4


def _logits(rows, vocab, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * 3
    x[:, :: max(1, vocab // 7)] += 8
    return x


@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 1000, 8191, 8192, 8193, 50001, 129280, 262147, 500009])
@pytest.mark.parametrize("t", [1.0, 0.37, 1.9])
def test_probs(vocab, t):
    """Relative error: the difference from the maximum and its quotient by T
    are rounded, |z| 2^-24 each for an exponent z (three roundings with the
    maximum's own), the exponential by 2^-22, the sum by 2^-24 per addition
    of a chain (a chain is at most vocab / 512 + 32 long) and the quotient by
    2^-23."""
    ds4 = _ds4()
    x = _logits(3, vocab, vocab).cuda()
    got = ds4.token_probs(x, t).double()
    ref = torch.softmax(x.double() / t, -1)
    z = (x.double() - x.double().amax(-1, keepdim=True)).abs() / t
    rel = 3 * z * 2.0 ** -24 + 2.0 ** -22 + (vocab / 512 + 32) * 2.0 ** -24 + 2.0 ** -23 + \
        (3 * z * 2.0 ** -24 * ref).sum(-1, keepdim=True)
    tiny = torch.finfo(torch.float32).smallest_normal
    assert ((got - ref).abs() <= rel * ref + tiny).all()


def test_probs_temperature_zero():
    """The lowest index of the maximum."""
    ds4 = _ds4()
    for vocab in (1, 5, 1000, 129280):
        x = torch.zeros(4, vocab)
        x[0] = -math.inf
        x[1, vocab // 2:] = 3.0
        x[2, -1] = math.inf
        x[3] = torch.randn(vocab, generator=torch.Generator().manual_seed(1))
        got = ds4.token_probs(x.cuda(), 0.0).cpu()
        for r, at in enumerate([0, vocab // 2, vocab - 1, int(x[3].argmax())]):
            want = torch.zeros(vocab)
            want[at] = 1.0
            assert torch.equal(got[r], want), (vocab, r)


def test_probs_not_finite():
    ds4 = _ds4()
    for vocab in (40, 129280):
        x = _logits(4, vocab, 2)
        x[0, 3] = math.nan
        x[1, 5] = math.inf
        x[2] = -math.inf
        x[3, 1::2] = -math.inf
        got = ds4.token_probs(x.cuda(), 1.0).cpu()
        assert torch.isnan(got[0]).all()
        assert torch.isnan(got[1, 5]) and torch.isnan(got[2]).all()
        assert (got[3, 1::2] == 0).all() and abs(float(got[3].double().sum()) - 1) < 1e-5
        assert torch.isnan(ds4.token_probs(x[:1].cuda(), 0.0)).all()


def test_probs_in_place_strides_and_stream():
    ds4 = _ds4()
    wide = _logits(5, 4100, 3).cuda()
    x = wide[:, 3:3 + 4001]
    want = ds4.token_probs(x.contiguous(), 0.8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.equal(ds4.token_probs(x, 0.8), want)
    got = ds4.token_probs(x, 0.8, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    keep = wide.clone()
    ds4.token_probs(x, 0.8, out=x)
    assert torch.equal(x, want)
    assert torch.equal(wide[:, :3], keep[:, :3]) and torch.equal(wide[:, 4004:], keep[:, 4004:])
    assert torch.equal(ds4.token_probs(wide[0], 1.0), ds4.token_probs(wide[:1], 1.0)[0])
    assert ds4.token_probs(wide[:0], 1.0).shape == (0, 4100)


# ---------------------------------------------------------------------------

def _draw(weights, u):
    """The lowest v whose cumulative weight exceeds u * sum, in fractions."""
    ws = [Fraction(float(w)) for w in weights]
    total = sum(ws)
    if total == 0:
        return -1
    c = Fraction(0)
    for v, w in enumerate(ws):
        c += w
        if c > Fraction(float(u)) * total:
            return v
    raise AssertionError


def _verify(target, draft, tokens, ua, us, count):
    B, G = tokens.shape
    acc, out = [], []
    for b in range(B):
        n = 0
        while n < count[b]:
            t = int(tokens[b, n])
            if not 0 <= t < target.shape[2]:
                break
            q = Fraction(1) if draft is None else Fraction(float(draft[b, n, t]))
            if not Fraction(float(ua[b, n])) * q < Fraction(float(target[b, n, t])):
                break
            n += 1
        p = target[b, n]
        r = p
        if n < count[b]:
            if draft is None:
                r = p.clone()
                if 0 <= int(tokens[b, n]) < r.numel():
                    r[int(tokens[b, n])] = 0
            else:
                r = (p.double() - draft[b, n].double()).clamp(min=0)
            if not (r > 0).any():
                r = p
        acc.append(n)
        out.append([int(x) for x in tokens[b, :n]] + [_draw(r, us[b])] + [-1] * (G - n))
    return torch.tensor(acc, dtype=torch.int32), torch.tensor(out, dtype=torch.int32)


def _inputs(B, G, V, seed, near=0.5):
    g = torch.Generator().manual_seed(seed)
    base = torch.randn(B, G + 1, V, generator=g) * 2
    target = torch.softmax(base, -1)
    draft = torch.softmax(base[:, :G] + near * torch.randn(B, G, V, generator=g), -1)
    tokens = torch.multinomial(draft.reshape(-1, V), 1, generator=g).view(B, G).int() if G else torch.zeros(B, 0).int()
    return target, draft, tokens, torch.rand(B, G, generator=g), torch.rand(B, generator=g)


@pytest.mark.parametrize("V", [1, 2, 33, 1000, 4099])
@pytest.mark.parametrize("G", [0, 1, 3, 7])
@pytest.mark.parametrize("sure", [False, True])
def test_verify(V, G, sure):
    ds4 = _ds4()
    B = 9
    target, draft, tokens, ua, us = _inputs(B, G, V, 100 * G + V)
    us[0], us[1] = 0.0, 1 - 2.0 ** -24
    if G:
        ua[0], ua[1] = 0.0, 1 - 2.0 ** -24
    count = torch.tensor([G - (b % (G + 1)) for b in range(B)], dtype=torch.int32)
    d = None if sure else draft
    for cnt in (None, count):
        got = ds4.verify_drafts(target.cuda(), None if d is None else d.cuda(), tokens.cuda(), ua.cuda(), us.cuda(),
                                n_draft=None if cnt is None else cnt.cuda())
        want = _verify(target, d, tokens, ua, us, [G] * B if cnt is None else cnt.tolist())
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def test_verify_whole_vocabulary():
    """129280 tokens; the cumulative sums in 64 bits (a border lies within
    their error with probability below 1e-6)."""
    ds4 = _ds4()
    target, draft, tokens, ua, us = _inputs(6, 3, 129280, 5, near=0.3)
    n, out = ds4.verify_drafts(target.cuda(), draft.cuda(), tokens.cuda(), ua.cuda(), us.cuda())
    for b in range(6):
        k = int(n[b])
        t = tokens[b].tolist()
        for i in range(3):
            ok = float(ua[b, i]) * float(draft[b, i, t[i]]) < float(target[b, i, t[i]])
            assert ok if i < k else (not ok or i > k)
        r = target[b, k].double()
        if k < 3:
            r = (r - draft[b, k].double()).clamp(min=0)
        c = torch.cumsum(r, 0)
        assert int(out[b, k]) == int((c <= float(us[b]) * c[-1]).sum())
        assert out[b, :k].tolist() == t[:k] and (out[b, k + 1:] == -1).all()


def test_verify_edges():
    """Equal distributions leave nothing (the draw falls back to p), rows
    without mass give -1, drafted tokens outside the vocabulary are rejected."""
    ds4 = _ds4()
    V = 50
    target, draft, tokens, ua, us = _inputs(4, 2, V, 3)
    ua[:] = 0.999
    target[0, 0] = draft[0, 0]
    target[0, 0, tokens[0, 0]] = draft[0, 0, tokens[0, 0]] = 0.0  # p == q, the drafted token at 0
    target[1, 0] = 0.0
    target[2, 0] = math.nan
    tokens[3] = torch.tensor([V, -1])
    err = torch.zeros(1, dtype=torch.int32).cuda()
    count = torch.tensor([2, 2, 2, 9], dtype=torch.int32).cuda()
    n, out = ds4.verify_drafts(target.cuda(), draft.cuda(), tokens.cuda(), ua.cuda(), us.cuda(), n_draft=count,
                               err_flags=err)
    assert n.tolist() == [0, 0, 0, 0]
    assert int(out[0, 0]) == _draw(target[0, 0], us[0])
    assert int(out[1, 0]) == -1 and int(out[2, 0]) == -1
    assert int(out[3, 0]) == _draw((target[3, 0].double() - draft[3, 0].double()).clamp(min=0), us[3])
    assert int(err) == ds4.DEVERR_TOKEN_ID | ds4.DEVERR_LENGTH


def test_verify_accepts_what_the_target_prefers():
    """u q < p with u near one: accepted where p > q, and where q is 0 only if p > 0."""
    ds4 = _ds4()
    V = 8
    target = torch.full((1, 4, V), 0.125)
    draft = torch.full((1, 3, V), 0.125)
    draft[0, 2, 1] = 0.0
    ua = torch.tensor([[1 - 2.0 ** -24, 0.5, 0.9]])
    tokens = torch.tensor([[0, 5, 1]], dtype=torch.int32)
    n, out = ds4.verify_drafts(target.cuda(), draft.cuda(), tokens.cuda(), ua.cuda(), torch.tensor([0.99]).cuda())
    assert n.tolist() == [3] and out.tolist() == [[0, 5, 1, 7]]


def test_verify_draws_the_targets_distribution():
    """Accepting and drawing together reproduce p: 40000 sequences of one
    draft over 6 tokens; each count lies within 5 standard deviations."""
    ds4 = _ds4()
    N, V = 40000, 6
    p = torch.tensor([0.4, 0.05, 0.25, 0.1, 0.15, 0.05])
    q = torch.tensor([0.1, 0.3, 0.2, 0.2, 0.05, 0.15])
    g = torch.Generator().manual_seed(8)
    tokens = torch.multinomial(q, N, replacement=True, generator=g).int().view(N, 1)
    n, out = ds4.verify_drafts(p.expand(N, 2, V).contiguous().cuda(), q.expand(N, 1, V).contiguous().cuda(), tokens.cuda(),
                               torch.rand(N, 1, generator=g).cuda(), torch.rand(N, generator=g).cuda())
    first = out[:, 0].cpu()
    for v in range(V):
        sd = math.sqrt(N * float(p[v]) * (1 - float(p[v])))
        assert abs(int((first == v).sum()) - N * float(p[v])) < 5 * sd


def test_refusals():
    ds4 = _ds4()
    x = torch.zeros(2, 8).cuda()
    for t in (-1.0, math.nan, math.inf, 1e-40):
        with pytest.raises(ds4.Ds4MoeError):
            ds4.token_probs(x, t)
    with pytest.raises(ValueError):
        ds4.token_probs(x.half())
    with pytest.raises(ValueError):
        ds4.token_probs(x, out=torch.zeros(2, 9).cuda())
    target, draft, tokens, ua, us = (t.cuda() for t in _inputs(2, 2, 8, 1))
    with pytest.raises(ValueError):
        ds4.verify_drafts(target, draft[:, :1], tokens, ua, us)
    with pytest.raises(ValueError):
        ds4.verify_drafts(target, draft, tokens.long(), ua, us)
    with pytest.raises(ValueError):
        ds4.verify_drafts(target.double(), draft, tokens, ua, us)
    big = torch.zeros(1, ds4.MAX_DRAFT + 2, 4).cuda()
    with pytest.raises(ds4.Ds4MoeError):
        ds4.verify_drafts(big, None, torch.zeros(1, ds4.MAX_DRAFT + 1).int().cuda(),
                          torch.zeros(1, ds4.MAX_DRAFT + 1).cuda(), us[:1])
