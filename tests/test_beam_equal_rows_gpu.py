"""Beams with the same logits and the same score tie exactly, wherever their rows begin in memory and
however large their logits are: the lower beam first, all scores the same bits.

The score's only computed part is the row's sum.  Its terms are functions of the logit alone, times
exact powers of two, and are added in 64 bits: sums of the same terms in another order differ
by some 2^-52, which the fp32 scores (2^-24) show for fewer than one in 10^7 rows."""
import numpy as np
import pytest
import torch

import ssd_sequence_mixing_b200 as ssd

pytestmark = pytest.mark.gpu

RANGES = {  # logits drawn between these
    "usual": (-8, 8),
    "past_64": (56, 72),
    "at_64": (63.5, 64.5),
    "at_minus_64": (-64.5, -63.5),
    "at_192": (191.75, 192.5),
    "at_355": (354.5, 355.25),  # 512 ln 2
    "around_64": (-70, 70),
    "past_192": (180, 200),
    "negative": (-72, -56),
    "far_negative": (-2100, -2000),
    "wide": (-500, 500),
    "far": (5000, 5040),
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1023, 5003, 40001])
@pytest.mark.parametrize("which", list(RANGES))
def test_equal_rows_tie(which, vocab, dtype):
    lo, hi = RANGES[which]
    batch, beams = 96 if vocab < 40000 else 24, 8
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    row = (lo + (hi - lo) * torch.rand(batch, 1, vocab, generator=gen, device="cuda")).to(dtype)
    row[:, :, torch.randint(vocab, (vocab // 50,), generator=gen, device="cuda")] = -float("inf")
    logits = row.expand(batch, beams, vocab).contiguous()
    scores = (-20 * torch.rand(batch, 1, generator=gen, device="cuda")).expand(batch, beams).contiguous()
    got, tokens, parents = ssd.beam_select(logits, scores)
    # what one such beam alone gives: entries of equal scores come beam by beam, in that order
    alone, alone_tokens, _ = (t.cpu().tolist() for t in ssd.beam_select(row.contiguous(), scores[:, :1].contiguous(), count=beams))
    for b in range(batch):
        want = []
        for value in sorted(set(alone[b]), reverse=True):
            same = [t for s, t in zip(alone[b], alone_tokens[b]) if s == value]
            want += [(value, t, i) for i in range(beams) for t in same]
        assert list(zip(got[b].tolist(), tokens[b].tolist(), parents[b].tolist())) == want[:beams], b
    # ... and the scores are right: the terms' error is that of 2^x in fp32, 2^-22, and random from
    # term to term; the score's own rounding is 2^-24 of it, and of its parts where they cancel
    x = row[:, 0].double()
    want = scores[:, 0].double() + (x.amax(-1) - torch.logsumexp(x, -1))
    off = (got[:, 0].double() - want).abs() / (2.0 ** -22 + 2.0 ** -23 * want.abs())
    assert off.max() <= 1, float(off.max())


@pytest.mark.parametrize("large", [2.0 ** 20, 3e6, -3e6, 1e9, -1e9, 1e30, -3.4e38])
def test_logits_of_any_size(large):
    """Rows near one large value, rows that mix it with usual ones, and masks of the lowest value."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    near = torch.full((4, 2, 3001), large, device="cuda") + 40 * torch.rand(4, 2, 3001, generator=gen, device="cuda")
    usual = torch.randn(4, 2, 3001, generator=gen, device="cuda")
    mixed = torch.where(torch.rand(usual.shape, generator=gen, device="cuda") < 0.5, usual, near)
    first = usual.clone()
    first[..., :1500] = near[..., :1500]
    for logits in (near, mixed, first):
        x = logits.cpu().numpy().astype(np.float64)
        top = x.max(-1, keepdims=True)
        lse = top + np.log(np.exp(x - top).sum(-1, keepdims=True))
        score = (x - lse).reshape(4, -1)
        want = np.sort(score, axis=1)[:, ::-1][:, :2]
        got, tokens, parents = ssd.beam_select(logits.contiguous(), torch.zeros(4, 2, device="cuda"))
        got = got.double().cpu().numpy()
        at = parents.cpu().numpy().astype(np.int64) * 3001 + tokens.cpu().numpy()
        picked = np.take_along_axis(score, at, 1)
        # the sum's rounding, and that of x - lse formed in 64 bits
        tol = 2.0 ** -21 + 2.0 ** -23 * np.abs(want) + 2.0 ** -50 * abs(large)
        assert (np.abs(got - want) / tol).max() <= 1
        assert (np.abs(picked - want) / tol).max() <= 1
