"""The LM-head in 8 bits against 64 bits at the precision of fp32 sums, which the bounds of
tests/test_gpu_fp8.py (a worst case for every element) cannot tell from less.  Needs an
MI355X."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import fp8_cases as F
from tests import fp8_sums as S

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def z_of(pair, wq, ws, row):
    """z of every token and one row of the weight: with one column the LSE is its logit."""
    n = pair[0].shape[0]
    logp, lse = rlk.fused_lmhead_fp8(
        pair, wq[row:row + 1], ws[row // F.BLOCK: row // F.BLOCK + 1],
        torch.zeros(n, dtype=torch.int32, device=DEV), real_vocab=1, padded_vocab=256,
        num_vocab_tiles=1)
    assert (logp == 0).all()
    return lse


@pytest.mark.parametrize("k", [128, 1152, 4096])
@pytest.mark.parametrize("n", [1, 16, 40, 64, 65, 700])
def test_sums_are_fp32(n, k):
    """z of the streaming kernel (up to 64 tokens) and of the tile kernel."""
    print(f"case n {n} k {k}", flush=True)
    rows = 256 if n < 65 else 16
    pair, (wq, ws) = S.operands(n, k, rows, n + k, DEV)
    z, tol = S.product64(*pair, wq, ws)
    got = torch.stack([z_of(pair, wq, ws, r) for r in range(rows)], 1)
    off = S.rms(got - z)
    print(f"off by {off:.2e}, bound {tol:.2e}", flush=True)
    assert off <= tol


@pytest.mark.parametrize("n", [1, 48, 300])
def test_logp_of_likely_tokens(n):
    """logp near 0, where nothing else hides z's error: tokens that the model is nearly sure of,
    hidden_dim 4096 x 30011 columns.

    logp and LSE take z twice, so an error of z counts twice at most.  The exponentials' fp32
    sums: the target's column holds most of the sum, so the other terms' errors (8 half steps,
    and 2 |z - maximum| for the rounding of the argument, which stays below 32) count as their
    share of the sum, below a half; and the sum itself, LSE and logp are rounded, by half a step
    of a number below 32 each."""
    k, v = 4096, 30011
    gen = torch.Generator(device=DEV).manual_seed(n)
    sigma = 1.3 / k ** 0.5
    w = (torch.randn((v, k), generator=gen, device=DEV) * sigma).to(torch.bfloat16)
    tgt = torch.randint(0, v, (n,), generator=gen, device=DEV, dtype=torch.int32)
    h = torch.randn((n, k), generator=gen, device=DEV) + 14.0 / (k * sigma ** 2) * w[tgt.long()]
    h = h.to(torch.bfloat16)
    wq, ws = rlk.quantize_fp8(w, 128)
    hq, hs = rlk.quantize_fp8(h)
    logp, lse = rlk.fused_lmhead_fp8(h, wq, ws, tgt, real_vocab=v, num_vocab_tiles=64)
    z, tol = S.product64(hq, hs, wq, ws)
    ref = torch.logsumexp(z, 1)
    want = z.gather(1, tgt.long()[:, None])[:, 0] - ref
    assert (want > -1.0).float().mean() > 0.5
    # the target's own z has the largest magnitudes: the tolerance of these alone
    own = torch.stack([torch.tensor(S.product64(
        hq[i:i + 1], hs[i:i + 1], wq[t:t + 1], ws[t // F.BLOCK: t // F.BLOCK + 1])[1])
        for i, t in enumerate(tgt.tolist()[:32])])
    tol = 2 * max(tol, S.rms(own)) + (8 + 2 * 32 + 2 * 32) * S.HALF_F32
    print(f"logp off by {S.rms(logp - want):.2e}, LSE {S.rms(lse - ref):.2e}, bound {tol:.2e}",
          flush=True)
    assert S.rms(logp - want) <= tol and S.rms(lse - ref) <= tol


def test_every_width_of_the_tile():
    """A wide vocabulary, where the tile kernel takes 128, 192 or 256 tokens by how many rounds
    of the chip that makes: the streaming kernel's bits in each."""
    v, pad, k = 151936, 152064, 256
    pair, (wq, ws) = S.operands(1024, k, v, 5, DEV)
    pair = pair[0], pair[1].t().contiguous().t()
    tgt = torch.randint(0, v, (1024,), device=DEV, dtype=torch.int32)
    kw = dict(real_vocab=v, padded_vocab=pad)

    def calls(rows):
        p = pair[0][rows], pair[1][rows]
        return (rlk.lmhead_logits_fp8(p, wq, ws, **kw),
                *rlk.fused_lmhead_fp8(p, wq, ws, tgt[rows], num_vocab_tiles=64, **kw))

    ref = [torch.cat(x) for x in zip(*(calls(slice(i, i + 64)) for i in range(0, 1024, 64)))]
    for n in (65, 100, 150, 190, 250, 333, 500, 777, 1024):
        print(f"{n} tokens", flush=True)
        for got, want in zip(calls(slice(0, n)), ref):
            assert torch.equal(bits(got), bits(want[:n])), n
