"""Token probabilities and verification at batch sizes and vocabularies where
the launch differs: clusters made smaller for many rows, rows that are not
16-byte aligned, vocabularies above 2^17 (sums of coarser multiples)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _ds4():
    import deepseek_v4_flash_gb300 as ds4
    return ds4


@pytest.mark.parametrize("t", [1.0, 0.6])
@pytest.mark.parametrize("rows,vocab", [(320, 129280), (320, 129281), (320, 50001), (320, 50000), (77, 129281), (700, 9001),
                                        (40, 131072), (2000, 4097), (40, 16384), (320, 16385)])
def test_probs_of_a_batch(rows, vocab, t):
    """Error as for single rows: the exponent z = (x - max) / T carries three
    roundings of |z| 2^-24, the exponential 2^-22, a sum at most vocab / 512 +
    32 additions of 2^-24, the quotient 2^-23."""
    ds4 = _ds4()
    x = torch.randn(rows, vocab, generator=torch.Generator(device="cuda").manual_seed(vocab), device="cuda") * 3
    x[:, :: vocab // 7] += 8
    got = ds4.token_probs(x, t)
    tiny = torch.finfo(torch.float32).smallest_normal
    for a in range(0, rows, 64):
        z = x[a:a + 64].double() / t
        ref = torch.softmax(z, -1)
        z = (z - z.amax(-1, keepdim=True)).abs()
        rel = 3 * z * 2.0 ** -24 + 2.0 ** -22 + (vocab / 512 + 32) * 2.0 ** -24 + 2.0 ** -23 + \
            (3 * z * 2.0 ** -24 * ref).sum(-1, keepdim=True)
        assert ((got[a:a + 64].double() - ref).abs() <= rel * ref + tiny).all()
    assert torch.equal(ds4.token_probs(x, t, out=x), got)  # in place


@pytest.mark.parametrize("rows,vocab", [(1, 129281), (5, 129281), (5, 4099), (320, 50001), (320, 50000), (700, 9001), (3, 262147)])
@pytest.mark.parametrize("offset", [0, 1])
def test_temperature_zero_of_a_batch(rows, vocab, offset):
    """Ties, rows of -infinity, infinities and NaN; rows at any alignment."""
    ds4 = _ds4()
    g = torch.Generator(device="cuda").manual_seed(rows)
    wide = torch.randn(rows, vocab + 3, generator=g, device="cuda").round()  # whole numbers: many ties
    x = wide[:, offset:offset + vocab]
    x[0, vocab // 3] = x[0, vocab - 1] = 9.0
    if rows > 4:
        x[1] = -math.inf
        x[2, vocab // 2:] = math.inf
        x[3, vocab - 1] = math.nan
        x[4, 0] = -math.inf
    got = ds4.token_probs(x, 0.0)
    top = x.amax(-1, keepdim=True)
    at = torch.where(x == top, torch.arange(vocab, device="cuda"), vocab).amin(-1)
    want = torch.zeros_like(got)
    ok = ~torch.isnan(top[:, 0])
    want[torch.arange(rows, device="cuda")[ok], at[ok]] = 1.0
    assert torch.equal(got[ok], want[ok]) and torch.isnan(got[~ok]).all()


def _fixed(p, shift):
    """Probabilities as whole multiples of 2^-shift, rounded to the nearest."""
    return torch.round(p.double().nan_to_num(0.0).clamp(0, 1) * 2.0 ** shift).long()


def _verify(target, draft, tokens, ua, us, count):
    """The definition in whole numbers, a sequence at a time."""
    B, G = tokens.shape
    V = target.shape[2]
    lg = (V - 1).bit_length()
    shift = 62 - lg if lg > 17 else 45
    acc, out = [], []
    for b in range(B):
        n = 0
        while n < count[b]:
            x = int(tokens[b, n])
            q = 1.0 if draft is None else float(draft[b, n, x])
            if not float(ua[b, n]) * q < float(target[b, n, x]):  # 24 x 24 bits: exact in 64-bit floats
                break
            n += 1
        p = target[b, n]
        r = _fixed(p, shift)
        if n < count[b]:
            if draft is None:
                r[int(tokens[b, n])] = 0
            else:
                q = draft[b, n]
                r = torch.where(p > q, r - _fixed(q, shift), 0)
            if int(r.sum()) == 0:
                r = _fixed(p, shift)
        c = torch.cumsum(r, 0)
        total = int(c[-1])
        u = int(float(us[b]) * 2 ** 24)  # the uniform numbers are multiples of 2^-24
        assert u == float(us[b]) * 2 ** 24
        drawn = int((c <= total * u >> 24).sum()) if total else -1
        acc.append(n)
        out.append([int(x) for x in tokens[b, :n]] + [drawn] + [-1] * (G - n))
    return torch.tensor(acc, dtype=torch.int32), torch.tensor(out, dtype=torch.int32)


@pytest.mark.parametrize("B,G,V", [(64, 3, 129280), (64, 3, 129281), (200, 2, 50001), (400, 1, 9001), (400, 1, 9000), (3, 2, 131072),
                                   (3, 2, 131073), (4, 2, 200003), (2, 1, 500009), (1, 4, 129281)])
@pytest.mark.parametrize("sure", [False, True])
def test_verify_of_a_batch(B, G, V, sure):
    ds4 = _ds4()
    g = torch.Generator(device="cuda").manual_seed(B + V)
    base = torch.randn(B, G + 1, V, generator=g, device="cuda") * 2
    target = torch.softmax(base, -1)
    draft = torch.softmax(base[:, :G] + 0.5 * torch.randn(B, G, V, generator=g, device="cuda"), -1)
    del base
    tokens = torch.multinomial(draft.view(B * G, V), 1, generator=g).view(B, G).int()
    ua = torch.randint(2 ** 24, (B, G), generator=g, device="cuda") / 2.0 ** 24
    us = torch.randint(2 ** 24, (B,), generator=g, device="cuda") / 2.0 ** 24
    us[0] = 1 - 2.0 ** -24
    us[-1] = 0.0
    us[B // 2] = 2.0 ** -24
    count = torch.randint(0, G + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    count[0] = G
    d = None if sure else draft
    got = ds4.verify_drafts(target, d, tokens, ua, us, n_draft=count)
    want = _verify(target, d, tokens.cpu(), ua.cpu(), us.cpu(), count.tolist())
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
