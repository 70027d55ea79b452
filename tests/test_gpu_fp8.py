"""The LM-head in 8-bit floating point: the cast against its definition (equal values), the
product and the statistics against 64 bits.  Needs an MI355X."""
from __future__ import annotations

import os
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import fp8_cases as F
from tests import lmhead_cases as C
from tests import lmhead_child

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
ROOT = Path(__file__).resolve().parent.parent


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    return torch.equal(bits(a), bits(b))


def equal_values(got, want):
    """Equal as numbers, NaN where NaN is wanted."""
    got = got.double()
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("n, k, ld", [(1, 128, 128), (3, 256, 320), (127, 128, 136),
                                      (129, 384, 384), (1000, 1152, 1160)])
def test_cast(n, k, ld, block_rows):
    gen = torch.Generator(device=DEV).manual_seed(n + k)
    buf = torch.randn((n, ld), generator=gen, device=DEV)
    buf *= torch.exp2(torch.randint(-30, 30, (n, 1), generator=gen, device=DEV).float())
    x = buf.to(torch.bfloat16)[:, :k]
    q, scale = rlk.quantize_fp8(x, block_rows)
    assert q.shape == (n, k) and scale.shape == (-(-n // block_rows), k // 128)
    qr, sr = F.cast64(x, block_rows)
    assert equal_values(scale, sr) and equal_values(q, qr)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_cast_special_values(block_rows):
    """Zeros; the smallest and the largest magnitudes of bf16; values midway between two e4m3
    values; blocks with infinity or NaN, which stay in their block."""
    vals = [0.0, 2.0 ** -133, 2.0 ** -126, 1e-38, 1.0, 2.0 ** 127, 3.3895313892515355e38]
    rows = []
    for v in vals:
        r = torch.zeros(256)
        r[:128] = torch.linspace(-1, 1, 128) * v
        r[5] = v
        rows.append(r)
    ties = torch.zeros(256)
    ties[:128] = torch.tensor([448.0 - i for i in range(128)])  # a scale of 1
    ties[128:] = torch.arange(128) * 2.0 ** -10  # e4m3 subnormals and below, under a scale of
    ties[128] = 448.0                            # 1 as well
    rows.append(ties)
    for bad in (float("inf"), float("-inf"), float("nan")):
        r = torch.linspace(-3, 3, 256)
        r[17] = bad
        rows.append(r)
    x = torch.stack(rows)
    if block_rows == 128:  # one row of blocks per row above
        x = x.repeat_interleave(128, 0)
    x = x.to(torch.bfloat16).to(DEV)
    q, scale = rlk.quantize_fp8(x, block_rows)
    qr, sr = F.cast64(x, block_rows)
    assert equal_values(scale, sr) and equal_values(q, qr)
    assert q.float()[:-3 * block_rows].isfinite().all()


def test_cast_of_nothing():
    q, scale = rlk.quantize_fp8(torch.empty((0, 256), dtype=torch.bfloat16, device=DEV), 128)
    assert q.shape == (0, 256) and scale.shape == (0, 2)


def make(n, k, v_real, v_pad, seed):
    """A case, its weight cast (rows from v_real on hold random bits) and the hidden states'."""
    c = C.make_case(n, k, v_real, v_pad, seed, DEV)
    clean = c.w.clone()
    clean[v_real:] = 0.0
    wq, ws = rlk.quantize_fp8(clean, 128)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    wq.view(torch.uint8)[v_real:] = torch.randint(0, 256, (v_pad - v_real, k), generator=gen,
                                                  device=DEV, dtype=torch.int32).to(torch.uint8)
    return c, (wq, ws), rlk.quantize_fp8(c.h)


SHAPES = [
    dict(n=1, k=128, v=256, pad=256), dict(n=1, k=1152, v=1003, pad=1024),
    dict(n=16, k=384, v=2500, pad=2560), dict(n=17, k=256, v=700, pad=701),
    dict(n=32, k=128, v=300, pad=515), dict(n=33, k=384, v=1500, pad=1500),
    dict(n=64, k=640, v=777, pad=1300), dict(n=65, k=128, v=1000, pad=1024),
    dict(n=257, k=512, v=2900, pad=3000), dict(n=600, k=384, v=513, pad=800),
]


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: "n{n}_k{k}_v{v}_p{pad}".format(**s))
def test_logits(s):
    print(f"case {s}", flush=True)
    n, v, pad = s["n"], s["v"], s["pad"]
    c, (wq, ws), (hq, hs) = make(n, s["k"], v, pad, 50 + n)
    z, err = F.product64(hq, hs, wq, ws, v)
    ld = (pad + 7) // 8 * 8 + 16
    out = torch.full((n, ld), 7.0, dtype=torch.bfloat16, device=DEV)
    rlk.rlk_lmhead_logits_fp8(rlk.make_desc(n, v, pad, ld, 1), rlk.make_fp8_matrix(hq, hs),
                              rlk.make_fp8_matrix(wq, ws), s["k"], out)
    torch.cuda.synchronize()
    off = (out[:, :v].double() - z).abs() / (err + C.HALF_BF16 * z.abs())
    print(f"error over bound {float(off.max()):.3f}", flush=True)
    assert off.max() <= 1.0
    assert (out[:, v:pad] == -torch.inf).all() and (out[:, pad:] == 7.0).all()
    # from bf16 hidden states; the scales with other strides
    assert same(rlk.lmhead_logits_fp8(c.h, wq, ws, real_vocab=v, padded_vocab=pad), out[:, :pad])
    wide = torch.full((ws.shape[0] * 2, ws.shape[1] * 3), float("nan"), device=DEV)[::2, ::3]
    wide.copy_(ws)
    got = rlk.lmhead_logits_fp8((hq, hs.contiguous()), wq, wide, real_vocab=v, padded_vocab=pad)
    assert same(got, out[:, :pad])
    got = rlk.lmhead_logits_fp8((hq, hs), wq, ws.t().contiguous().t(), real_vocab=v,
                                padded_vocab=pad)
    assert same(got, out[:, :pad])


@pytest.mark.parametrize("n", [1, 70])
def test_products_meet_in_groups_of_eight(n):
    """The property on which the products' error bound rests: with one column its LSE is z.
    A product beside one of 2^14 is kept down to 2^1 in the same 8 columns, and down to 2^-9 in
    others; what is cut goes towards zero; a subnormal lines the others up as 2^-6 would; a
    zero does not."""
    def z(at):
        """z of products {column: (h, w)}, as the streaming (n = 1) or the tile kernel has it."""
        h = torch.zeros((n, 128), device=DEV)
        w = torch.zeros((1, 128), device=DEV)
        for k, (a, b) in at.items():
            h[:, k], w[0, k] = a, b
        hq, wq = h.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn)
        assert (hq.float() == h).all() and (wq.float() == w).all()
        _, lse = rlk.fused_lmhead_fp8(
            (hq, torch.ones((n, 1), device=DEV)), wq, torch.ones((1, 1), device=DEV),
            torch.zeros(n, dtype=torch.int32, device=DEV), real_vocab=1, padded_vocab=256,
            num_vocab_tiles=1)
        assert (lse == lse[0]).all()
        return float(lse[0])

    top = (2.0 ** 7, 2.0 ** 7)
    for sign in (1.0, -1.0):
        assert z({8: top, 15: (sign * 2.0, 1.0)}) == 2.0 ** 14 + sign * 2.0
        assert z({8: top, 15: (sign, 1.0)}) == 2.0 ** 14
        assert z({8: top, 15: (sign * 1.875, 2.0)}) == 2.0 ** 14 + sign * 2.0
        for k in (7, 16, 127):
            assert z({8: top, k: (sign * 2.0 ** -9, 1.0)}) == 2.0 ** 14 + sign * 2.0 ** -9
    assert z({0: (2.0 ** -9, 2.0 ** 8), 1: (2.0 ** -5, 2.0 ** -6)}) == 0.5 + 2.0 ** -11
    assert z({0: (2.0 ** -9, 2.0 ** 8), 1: (2.0 ** -6, 2.0 ** -6)}) == 0.5
    assert z({0: (0.0, 448.0), 1: (2.0 ** -9, 2.0 ** -9)}) == 2.0 ** -18


def check_stats(c, logp, lse, z, err):
    """logp and LSE of z (64 bits): LSE moves by no more than z's largest error, the sum of
    exponentials is off by at most 128 half steps and, through the rounding of its
    arguments, 2 half steps of their mean magnitude (taken: the largest); logp by both."""
    ref = torch.logsumexp(z, 1)
    tol = err.amax(1) + (128 + 4 * ref.abs() + 2 * (z.amax(1) - z.amin(1))) * C.HALF_F32
    assert ((lse.double() - ref).abs() <= tol).all()
    act = c.active
    zt = z.gather(1, torch.where(act, c.tgt, 0).long()[:, None])[:, 0]
    want = torch.where(act, zt - ref, 0.0)
    assert ((logp.double() - want).abs() <= torch.where(act, 2 * tol, 0.0)).all()


@pytest.mark.parametrize("s", SHAPES, ids=lambda s: "n{n}_k{k}_v{v}_p{pad}".format(**s))
def test_statistics(s):
    print(f"case {s}", flush=True)
    n, v, pad = s["n"], s["v"], s["pad"]
    c, (wq, ws), pair = make(n, s["k"], v, pad, 150 + n)
    tiles = max(1, pad // 300)
    kw = dict(real_vocab=v, padded_vocab=pad, num_vocab_tiles=tiles)
    logp, lse = rlk.fused_lmhead_fp8(pair, wq, ws, c.tgt, c.mask, **kw)
    z, err = F.product64(*pair, wq, ws, v)
    check_stats(c, logp, lse, z, err)
    again = rlk.fused_lmhead_fp8(c.h, wq, ws, c.tgt, c.mask, **kw)
    assert same(again[0], logp) and same(again[1], lse)
    for shards in range(2, tiles + 1):
        got = rlk.fused_lmhead_fp8(pair, wq, ws, c.tgt, c.mask, num_virtual_shards=shards, **kw)
        assert same(got[0], logp) and same(got[1], lse), shards


def test_rows_do_not_depend_on_the_batch():
    """The streaming kernel (1, 16, 17, 40, 64 tokens) and the tile kernel in its widths (65,
    150, 250, 300) give a token the same bits: logits, logp and LSE."""
    c, (wq, ws), _ = make(300, 384, 2900, 3000, 61)
    kw = dict(real_vocab=2900, padded_vocab=3000)
    full = rlk.lmhead_logits_fp8(c.h, wq, ws, **kw)
    logp, lse = rlk.fused_lmhead_fp8(c.h, wq, ws, c.tgt, c.mask, num_vocab_tiles=7, **kw)
    for n in (1, 16, 17, 40, 64, 65, 150, 250):
        for at in (0, 300 - n):
            rows = slice(at, at + n)
            h = c.h[rows].contiguous()
            assert same(rlk.lmhead_logits_fp8(h, wq, ws, **kw), full[rows]), n
            got = rlk.fused_lmhead_fp8(h, wq, ws, c.tgt[rows].contiguous(),
                                       c.mask[rows].contiguous(), num_vocab_tiles=7, **kw)
            assert same(got[0], logp[rows]) and same(got[1], lse[rows]), n


def test_logits_feed_the_materialised_path():
    """forward() on the 8-bit logits gives the statistics of their bf16 values."""
    c, (wq, ws), _ = make(130, 256, 2900, 3000, 62)
    x = rlk.lmhead_logits_fp8(c.h, wq, ws, real_vocab=2900, padded_vocab=3000)
    logp, lse = rlk.forward(x, c.tgt, c.mask, real_vocab=2900, num_vocab_tiles=7)
    check_stats(c, logp, lse, x[:, :2900].double(), torch.zeros((130, 1), device=DEV))


@pytest.mark.parametrize("n", [3, 70])
def test_non_finite_blocks(n):
    """A NaN in a hidden state makes its row NaN and no other; in the weight, the 128 logits
    of its block of rows (and with them every row's LSE)."""
    c, (wq, ws), _ = make(n, 256, 600, 600, 63)
    kw = dict(real_vocab=600)
    ref = rlk.lmhead_logits_fp8(c.h, wq, ws, **kw)
    h = c.h.clone()
    h[1, 200] = float("nan")
    got = rlk.lmhead_logits_fp8(h, wq, ws, **kw)
    assert got[1].isnan().all() and same(got[2:], ref[2:]) and same(got[0], ref[0])
    logp, lse = rlk.fused_lmhead_fp8(h, wq, ws, c.tgt, None, num_vocab_tiles=2, **kw)
    assert lse[1].isnan() and lse[2:].isfinite().all()
    w = c.w.clone()
    w[300, 10] = float("inf")
    wq2, ws2 = rlk.quantize_fp8(w, 128)
    got = rlk.lmhead_logits_fp8(c.h, wq2, ws2, **kw)
    assert got[:, 256:384].isnan().all()
    assert same(got[:, :256], ref[:, :256]) and same(got[:, 384:], ref[:, 384:])
    logp, lse = rlk.fused_lmhead_fp8(c.h, wq2, ws2, c.tgt, None, num_vocab_tiles=2, **kw)
    assert lse.isnan().all()


def test_targets_masks_and_validate():
    c, (wq, ws), _ = make(40, 256, 600, 640, 64)
    kw = dict(real_vocab=600, padded_vocab=640, num_vocab_tiles=2)
    none = torch.zeros(40, dtype=torch.bool, device=DEV)
    logp, lse = rlk.fused_lmhead_fp8(c.h, wq, ws, c.tgt, none, **kw)
    assert (bits(logp) == 0).all() and lse.isfinite().all()
    tgt = c.tgt.clone()
    tgt[:] = 3
    tgt[5] = 610  # a padded column
    logp, _ = rlk.fused_lmhead_fp8(c.h, wq, ws, tgt, None, **kw)
    assert logp[5].isnan() and logp[6:].isfinite().all()
    with pytest.raises(rlk.RlkError) as ei:
        rlk.fused_lmhead_fp8(c.h, wq, ws, tgt, None, validate=True, **kw)
    assert ei.value.status == rlk.RLK_ERR_TARGET_RANGE
    rlk.fused_lmhead_fp8(c.h, wq, ws, c.tgt, c.mask, validate=True, **kw)
    # no token
    logp, lse = rlk.fused_lmhead_fp8(c.h[:0], wq, ws, c.tgt[:0], None, **kw)
    assert logp.shape == (0,)
    assert rlk.lmhead_logits_fp8(c.h[:0], wq, ws, real_vocab=600).shape == (0, 640)


@pytest.mark.parametrize("n", [20, 300])
def test_other_stream_and_graph_replays(n):
    """Cast, logits, statistics and the statistics of the logits as they run together:
    captured once, replayed on changing inputs, and on a side stream."""
    k, v, pad = 256, 2900, 3000
    sets = [make(n, k, v, pad, s) for s in (71, 72, 73)]
    st = {"h": sets[0][0].h.clone(), "tgt": sets[0][0].tgt.clone(),
          "mask": sets[0][0].mask.clone(), "wq": sets[0][1][0].clone(),
          "ws": sets[0][1][1].clone()}

    def load(i):
        c, (wq, ws), _ = sets[i]
        for name, x in (("h", c.h), ("tgt", c.tgt), ("mask", c.mask), ("wq", wq), ("ws", ws)):
            st[name].copy_(x)

    def calls(stream=None):
        kw = dict(real_vocab=v, padded_vocab=pad, stream=stream)
        pair = rlk.quantize_fp8(st["h"], stream=stream)
        x = rlk.lmhead_logits_fp8(pair, st["wq"], st["ws"], **kw)
        logp, lse = rlk.fused_lmhead_fp8(st["h"], st["wq"], st["ws"], st["tgt"], st["mask"],
                                         num_vocab_tiles=7, **kw)
        lp2, lse2 = rlk.forward(x, st["tgt"], st["mask"], real_vocab=v, num_vocab_tiles=7,
                                stream=stream)
        return [*pair, x, logp, lse, lp2, lse2]

    refs = []
    for i in range(3):
        load(i)
        out = calls()
        torch.cuda.synchronize()
        refs.append([bits(t).clone() for t in out])
    load(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = calls(side)  # a stream other than the current one
    side.synchronize()
    assert all(torch.equal(bits(t), r) for t, r in zip(out, refs[1]))
    load(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og = calls()
    torch.cuda.synchronize()
    for rep, i in enumerate((1, 0, 2, 2, 1)):
        print(f"replay {rep} on set {i}", flush=True)
        load(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(t), r) for t, r in zip(og, refs[i])), f"replay {rep}"
        calls()
        torch.cuda.synchronize()


def test_split_launches_give_the_same_bits(tmp_path):
    """Launches of at most so many threads (read once per process: child processes)."""
    ref = lmhead_child.run_all()
    for limit in (1024, 5000):
        print(f"launch limit {limit} threads (child process)", flush=True)
        out = tmp_path / f"bits_{limit}.pt"
        env = dict(os.environ, RLK_MAX_LAUNCH_THREADS=str(limit))
        r = subprocess.run([sys.executable, "-u", "-m", "tests.lmhead_child", str(out)], cwd=ROOT,
                           env=env, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, f"{r.stdout[-2000:]}\n{r.stderr[-3000:]}"
        got = torch.load(out, weights_only=True)
        assert set(got) == set(ref)
        for m, x in ref.items():
            assert torch.equal(x, got[m]), f"{m} differs with a {limit}-thread launch limit"
