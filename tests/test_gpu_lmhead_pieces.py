"""The LM-head's gradients of few tokens over a vocabulary of several pieces, and seeded random
shapes of the LM-head's and the 8-bit head's calls.  Needs an MI355X."""
from __future__ import annotations

import math
import random

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import fp8_cases as F
from tests import fp8_sums as S
from tests import lmhead_cases as C
from tests.test_gpu_fp8 import check_stats

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


@pytest.mark.parametrize("n", [9, 20, 40])
@pytest.mark.parametrize("v", [1_060_033, 500_011])
def test_few_tokens_in_pieces(n, v):
    """Up to 64 tokens a piece holds 2^20 columns at most: 1060100 columns go in two of 530176,
    the last ending in a slab of 33 rows, or all padding."""
    print(f"case n {n} v {v}", flush=True)
    pad, piece = 1_060_100, 530_176
    c = C.make_case(n, 64, v, pad, n, DEV, mask_keep=1.0, ignore_frac=0.0)
    c.tgt[0], c.tgt[1], c.tgt[2] = 0, v - 1, min(piece, v - 2)  # either end, both pieces
    c.mask[3] = False
    _, lse = rlk.fused_lmhead(c.h, c.w, c.tgt, c.mask, real_vocab=v, num_vocab_tiles=64)
    dh, dw = rlk.fused_lmhead_backward(c.h, c.w, c.tgt, c.mask, lse, c.g, c.gl, real_vocab=v)
    rh, eh, rw, ew = C.gradients64(c, c.g, c.gl)
    h, w = C.worst(dh, rh, eh), C.worst(dw, rw, ew)
    print(f"error over bound: dhidden {h:.3f}, dweight {w:.3f}", flush=True)
    assert h <= 1.0 and w <= 1.0
    assert (bits(dw[v:]) == 0).all()
    only_h, _ = rlk.fused_lmhead_backward(c.h, c.w, c.tgt, c.mask, lse, c.g, c.gl, real_vocab=v,
                                          want_weight=False)
    _, only_w = rlk.fused_lmhead_backward(c.h, c.w, c.tgt, c.mask, lse, c.g, c.gl, real_vocab=v,
                                          want_hidden=False)
    assert torch.equal(bits(dh), bits(only_h)) and torch.equal(bits(dw), bits(only_w))


def log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def shape(seed, slab):
    """(n, k, v, pad, tiles, shards): sizes over their logarithm, a tile of 256 columns at
    least."""
    rng = random.Random(seed)
    n, k = log_int(rng, 1, 1200), slab * log_int(rng, 1, 1024 // slab)
    v = log_int(rng, 1, 9000)
    pad = max(v + rng.choice((0, 0, 1, 77, 300)), 256)
    tiles = rng.randint(1, max(1, pad // 256))
    return n, k, v, pad, tiles, rng.randint(1, tiles)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    n, k, v, pad, tiles, shards = shape(seed, 64)
    print(f"case n {n} k {k} v {v} pad {pad} tiles {tiles} shards {shards}", flush=True)
    c = C.make_case(n, k, v, pad, seed, DEV, mask_keep=(1.0, 0.6)[seed % 2])
    kw = dict(real_vocab=v, num_vocab_tiles=tiles)
    logp, lse = rlk.fused_lmhead(c.h, c.w, c.tgt, c.mask, **kw)
    again = rlk.fused_lmhead(c.h, c.w, c.tgt, c.mask, num_virtual_shards=shards, **kw)
    assert torch.equal(bits(logp), bits(again[0])) and torch.equal(bits(lse), bits(again[1]))
    _, _, z = C.forward64(c)
    check_stats(c, logp, lse, z,
                (k + 2) * C.HALF_F32 * (c.h.double().abs() @ c.w[:v].double().abs().T))
    g, gl = ((c.g, None), (c.g, c.gl), (None, c.gl))[seed % 3]
    dh, dw = rlk.fused_lmhead_backward(c.h, c.w, c.tgt, c.mask, lse, g, gl, real_vocab=v)
    rh, eh, rw, ew = C.gradients64(c, g, gl)
    h, w = C.worst(dh, rh, eh), C.worst(dw, rw, ew)
    print(f"error over bound: dhidden {h:.3f}, dweight {w:.3f}", flush=True)
    assert h <= 1.0 and w <= 1.0


@pytest.mark.parametrize("seed", range(100, 124))
def test_random_shapes_in_8_bits(seed):
    n, k, v, pad, tiles, shards = shape(seed, 128)
    print(f"case n {n} k {k} v {v} pad {pad} tiles {tiles} shards {shards}", flush=True)
    c = C.make_case(n, k, v, v, seed, DEV)
    wq, ws = rlk.quantize_fp8(c.w, 128)
    pair = rlk.quantize_fp8(c.h)
    for got, x, rows in ((pair, c.h, 1), ((wq, ws), c.w, 128)):
        q, s = F.cast64(x, rows)
        assert torch.equal(got[0].double(), q) and torch.equal(got[1].double(), s)
    z, _ = S.product64(*pair, wq, ws)
    # each element: the sum of the magnitudes of all that is added up, half a step each
    size = F.value64(*pair, 1).abs() @ F.value64(wq, ws, 128).abs().T
    err = (128 + k // 128 + 3) * C.HALF_F32 * size
    kw = dict(real_vocab=v, padded_vocab=pad)
    x = rlk.lmhead_logits_fp8(c.h, wq, ws, **kw)
    assert ((x[:, :v].double() - z).abs() <= err + C.HALF_BF16 * z.abs()).all()
    assert (x[:, v:] == -torch.inf).all()
    stats = rlk.fused_lmhead_fp8(c.h, wq, ws, c.tgt, c.mask, num_vocab_tiles=tiles, **kw)
    check_stats(c, *stats, z, err)
    again = rlk.fused_lmhead_fp8(pair, wq, ws, c.tgt, c.mask, num_vocab_tiles=tiles,
                                 num_virtual_shards=shards, **kw)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(stats, again))
