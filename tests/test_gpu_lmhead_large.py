"""The LM-head operators where offsets pass 32 bits: tensors of more than 2^32 bytes, whose
last rows are compared with the same rows taken in a small call (the same bits) or with the
formula in 64 bits."""
from __future__ import annotations

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import fp8_cases as F
from tests import lmhead_cases as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bits(t):
    return t.contiguous().view(torch.uint8)


def test_cast_past_32_bits():
    """1.2 M rows x 4096 (9.8 GB): the last rows as in a call of their own."""
    rows = 1_200_037
    x = torch.empty((rows, 4096), dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    x[: 1 << 16].normal_(generator=gen)
    x[1 << 16:] = 0.5
    x[-300:].normal_(generator=gen)
    for block_rows in (1, 128):
        q, s = rlk.quantize_fp8(x, block_rows)
        first = rows // 128 * 128 - 128  # a whole block and the short one
        qt, st = rlk.quantize_fp8(x[first:], block_rows)
        assert torch.equal(bits(q[first:]), bits(qt))
        assert torch.equal(s[first // block_rows:], st)
        qt, st = rlk.quantize_fp8(x[:256], block_rows)
        assert torch.equal(bits(q[:256]), bits(qt)) and torch.equal(s[:256 // block_rows], st)
        assert (q[1 << 16: -428].view(torch.uint8) == 0x7e).all()  # 448
        del q, s


def test_logits_past_32_bits():
    """20000 tokens x 152576 columns (6.1 GB of logits): rows at either end as in a small call."""
    n, k, v, pad = 20000, 128, 151936, 152576
    c = C.make_case(n, k, v, v, 2, DEV)
    wp = rlk.quantize_fp8(c.w, 128)
    out = rlk.lmhead_logits_fp8(c.h, *wp, real_vocab=v, padded_vocab=pad)
    for rows in (slice(0, 70), slice(n - 70, n)):
        small = rlk.lmhead_logits_fp8(c.h[rows], *wp, real_vocab=v, padded_vocab=pad)
        assert torch.equal(bits(out[rows]), bits(small))
    z, err = F.product64(*rlk.quantize_fp8(c.h[n - 3:]), *wp, v)
    assert ((out[n - 3:, :v].double() - z).abs() <= err + C.HALF_BF16 * z.abs()).all()
    assert (out[:, v:] == -torch.inf).all()
    # one logit row at a stride of its own, far into a wide buffer
    del out, small
    ld = (1 << 31) // 8
    wide = torch.full((12, ld), 3.0, dtype=torch.bfloat16, device=DEV)  # 6.4 GB
    desc = rlk.make_desc(12, v, pad, ld, 1)
    rlk.rlk_lmhead_logits_fp8(desc, rlk.make_fp8_matrix(*(p := rlk.quantize_fp8(c.h[:12]))),
                              rlk.make_fp8_matrix(*wp), k, wide)
    small = rlk.lmhead_logits_fp8(c.h[:12], *wp, real_vocab=v, padded_vocab=pad)
    assert torch.equal(bits(wide[:, :pad]), bits(small)) and (wide[:, pad:] == 3.0).all()
    del p


@pytest.mark.parametrize("n", [40, 300])
def test_gradients_of_a_weight_past_32_bits(n):
    """hidden_dim 16384 x 151936 rows (5 GB of weight and of its gradient): dhidden, and the
    last rows of dweight, against the formula in 64 bits on a sample."""
    k, v, pad = 16384, 151936, 152000
    gen = torch.Generator(device=DEV).manual_seed(n)
    w = torch.empty((pad, k), dtype=torch.bfloat16, device=DEV)
    w.normal_(0.0, 1.3 / k ** 0.5, generator=gen)
    h = torch.randn((n, k), generator=gen, device=DEV).to(torch.bfloat16)
    tgt = torch.randint(0, v, (n,), generator=gen, device=DEV, dtype=torch.int32)
    tgt[0] = v - 1
    g = torch.randn(n, generator=gen, device=DEV)
    _, lse = rlk.fused_lmhead(h, w, tgt, None, real_vocab=v)
    dh, dw = rlk.fused_lmhead_backward(h, w, tgt, None, lse, g, None, real_vocab=v)
    hd, gd = h.double(), g.double()
    dz_all = torch.empty((n, v), dtype=torch.float64, device=DEV)
    ref_h = torch.zeros((n, k), dtype=torch.float64, device=DEV)
    for a in range(0, v, 16384):
        b = min(v, a + 16384)
        wd = w[a:b].double()
        dz = -gd[:, None] * (hd @ wd.T - lse.double()[:, None]).exp()
        hit = (tgt >= a) & (tgt < b)
        rows = hit.nonzero()[:, 0]
        dz[rows, tgt[rows].long() - a] += gd[rows]
        dz_all[:, a:b] = dz
        ref_h += dz @ wd
    ref_w = dz_all.T[-200:] @ hd
    # dz and the result are rounded to bf16, independently, by half a step at most each; the
    # roundings of fp32 sums, independent too, come to sqrt(K + V) 2^-24 = 2^-15 of the
    # magnitudes, which no sum here exceeds 2^5 times
    tol = 2 * C.HALF_BF16 + 2.0 ** -10
    off_h = float((dh.double() - ref_h).norm() / ref_h.norm())
    off_w = float((dw[v - 200:v].double() - ref_w).norm() / ref_w.norm())
    print(f"dhidden {off_h:.2e}, dweight {off_w:.2e}, tolerance {tol:.2e}", flush=True)
    assert off_h <= tol and off_w <= tol
    assert (bits(dw[v:]) == 0).all()
    ref_0 = dz_all.T[:100] @ hd
    assert float((dw[:100].double() - ref_0).norm() / ref_0.norm()) <= tol


def test_few_statistics_of_a_wide_vocabulary():
    """64 tokens x 20 M columns: z of few tokens passes 2^32 bytes in the workspace."""
    n, k, v = 64, 128, 20_000_123
    gen = torch.Generator(device=DEV).manual_seed(3)
    w = torch.randn((v, k), generator=gen, device=DEV).to(torch.bfloat16)
    wp = rlk.quantize_fp8(w, 128)
    h = torch.randn((200, k), generator=gen, device=DEV).to(torch.bfloat16)
    tgt = torch.randint(0, v, (200,), generator=gen, device=DEV, dtype=torch.int32)
    tgt[63] = v - 1
    few = rlk.fused_lmhead_fp8(h[:n], *wp, tgt[:n], real_vocab=v)
    many = rlk.fused_lmhead_fp8(h, *wp, tgt, real_vocab=v)  # the tile kernel
    assert torch.equal(few[0], many[0][:n]) and torch.equal(few[1], many[1][:n])
    hq, hs = rlk.quantize_fp8(h[62:64])
    zs = []
    for a in range(0, v, 1 << 22):
        b = min(v, a + (1 << 22))
        q, s = wp[0][a:b], wp[1][a // 128: (b + 127) // 128]
        zs.append(F.value64(hq, hs, 1) @ F.value64(q, s, 128).T)
    z = torch.cat(zs, 1)
    ref = torch.logsumexp(z, 1)
    want = z.gather(1, tgt[62:64].long()[:, None])[:, 0] - ref
    # z is off by its block's roundings (132 half steps of the magnitudes' sum) and by what
    # the matrix cores cut: 7 2^-13 of the largest product of each 8 columns, and 16 such are
    # at most four times the root of the sum of their squares; both sums are at most the
    # norms' product, but for subnormals (2^-6 of 448 at most: half as much again).  logp
    # takes it twice; the sum of exponentials adds nothing of that size
    norms = float(h[62:64].double().norm(dim=1).max() * w[:200000].double().norm(dim=1).max())
    tol = 2 * (132 * C.HALF_F32 + 4 * 7 * 2.0 ** -13) * 1.5 * norms
    assert ((few[0][62:].double() - want).abs() <= tol).all()
    assert ((few[1][62:].double() - ref).abs() <= tol).all()
