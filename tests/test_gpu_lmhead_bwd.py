"""GPU parity of the LM-head's gradients against a plain form in 64 bits, with bounds
derived from the roundings the kernel makes (tests/lmhead_cases.py).  Needs an MI355X."""
from __future__ import annotations

import os
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import lmhead_cases as C
from tests import lmhead_child

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
ROOT = Path(__file__).resolve().parent.parent


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def lse_of(c):
    """The LSE of every row as the library gives it."""
    _, lse = rlk.fused_lmhead(c.h, c.w, c.tgt, c.mask, real_vocab=c.v_real,
                              padded_vocab=max(c.w.shape[0], 256), num_vocab_tiles=1)
    return lse


def backward(c, g, gl, **kw):
    return rlk.fused_lmhead_backward(c.h, c.w, c.tgt, c.mask, lse_of(c), g, gl,
                                     real_vocab=c.v_real, **kw)


CASES = [
    # tokens, K, real and padded vocabulary, share of rows kept
    dict(n=1, k=64, v=256, pad=256, keep=1.0),
    dict(n=2, k=64, v=1, pad=1, keep=1.0),
    dict(n=37, k=64, v=40, pad=77, keep=0.8),
    # few tokens, in each width of their kernels; 64 of them at most
    dict(n=5, k=192, v=3001, pad=3100, keep=0.6),
    dict(n=16, k=320, v=700, pad=1024, keep=1.0),
    dict(n=17, k=128, v=2500, pad=2560, keep=0.5),
    dict(n=32, k=1088, v=900, pad=900, keep=1.0),
    dict(n=64, k=448, v=5000, pad=5001, keep=0.9),
    dict(n=65, k=448, v=5000, pad=5001, keep=0.9),
    dict(n=300, k=128, v=2500, pad=2560, keep=0.8),
    dict(n=257, k=320, v=3000, pad=3000, keep=0.5),
    dict(n=255, k=192, v=5001, pad=5120, keep=1.0),
    dict(n=513, k=448, v=1023, pad=1300, keep=0.1),
    dict(n=1100, k=64, v=257, pad=300, keep=0.9),
]


@pytest.mark.parametrize("terms", ["logp", "lse", "both"])
@pytest.mark.parametrize("c", CASES, ids=lambda c: "n{n}_k{k}_v{v}_p{pad}".format(**c))
def test_gradients_match_the_formula(c, terms):
    print(f"case {c} {terms}", flush=True)
    case = C.make_case(c["n"], c["k"], c["v"], c["pad"], 11 + c["n"], DEV, mask_keep=c["keep"])
    g = case.g if terms != "lse" else None
    gl = case.gl if terms != "logp" else None
    dh, dw = backward(case, g, gl)
    torch.cuda.synchronize()
    rh, eh, rw, ew = C.gradients64(case, g, gl)
    h, w = C.worst(dh, rh, eh), C.worst(dw, rw, ew)
    print(f"error over bound: dhidden {h:.3f}, dweight {w:.3f}", flush=True)
    assert h <= 1.0 and w <= 1.0
    assert (bits(dw[c["v"]:]) == 0).all()  # +0 in the padding
    # the same bits again, and when only one of the two is asked for
    dh2, none = backward(case, g, gl, want_weight=False)
    assert none is None
    none, dw2 = backward(case, g, gl, want_hidden=False)
    assert none is None
    assert torch.equal(bits(dh), bits(dh2)) and torch.equal(bits(dw), bits(dw2))


@pytest.mark.parametrize("v", [33000, 5001])
def test_many_pieces(v):
    """16500 tokens take the vocabulary in pieces of at most 16384 columns: 33100 columns in
    three, the last ending in padding or the last two all padding."""
    case = C.make_case(16500, 64, v, 33100, 5, DEV)
    dh, dw = backward(case, case.g, case.gl)
    rh, eh, rw, ew = C.gradients64(case, case.g, case.gl)
    assert C.worst(dh, rh, eh) <= 1.0 and C.worst(dw, rw, ew) <= 1.0


@pytest.mark.parametrize("live", [1, 200, 256, 257, 800])
def test_few_live_rows(live):
    """Of 1100 tokens only `live` are active, anywhere in the batch: dh's sums are then taken
    in more parts (25 to each tile of 256 tokens if all were live, up to 125)."""
    case = C.make_case(1100, 320, 33000, 33024, 17, DEV, mask_keep=1.0, ignore_frac=0.0)
    gen = torch.Generator(device=DEV).manual_seed(live)
    case.mask[torch.randperm(1100, generator=gen, device=DEV)[live:]] = False
    dh, dw = backward(case, case.g, None)
    rh, eh, rw, ew = C.gradients64(case, case.g, None)
    h, w = C.worst(dh, rh, eh), C.worst(dw, rw, ew)
    print(f"error over bound: dhidden {h:.3f}, dweight {w:.3f}", flush=True)
    assert h <= 1.0 and w <= 1.0
    assert (bits(dh[~case.mask]) == 0).all()


def test_equal_gradients_round_without_bias():
    """A mean's gradient is the same for every row.  The target's entry of dz is then near
    that one number in every row; its rounding must not shift all of them alike.  The
    norm-wise error stays that of independent roundings: half a step is at most 2^-8, so a
    rounding's relative error has a mean square of at most 2^-16 / 3, and the two that meet
    in dweight (dz, the result) give at most sqrt(2 / 3) 2^-8."""
    case = C.make_case(500, 128, 4000, 4000, 3, DEV, mask_keep=1.0, ignore_frac=0.0, peaked=0.0)
    for scale in (1.0 / 500, 1.0 / 3.0, 1e-30, 1e30):
        g = torch.full((500,), -scale, device=DEV)
        dh, dw = backward(case, g, None)
        rh, _, rw, _ = C.gradients64(case, g, None)
        # in units of the scale: 64 bits hold the squares of 1e30
        off_h = ((dh.double() - rh) / scale).norm() / (rh / scale).norm()
        off_w = ((dw.double() - rw) / scale).norm() / (rw / scale).norm()
        print(f"scale {scale:.3g}: dhidden {off_h:.2e}, dweight {off_w:.2e}", flush=True)
        assert off_h <= (2 / 3) ** 0.5 * 2 ** -8 and off_w <= (2 / 3) ** 0.5 * 2 ** -8


@pytest.mark.parametrize("n", [40, 300])
def test_masked_rows_may_hold_anything(n):
    """Rows that no term reaches: their hidden states, LSE and gradients are not read."""
    case = C.make_case(n, 128, 1000, 1024, 7, DEV)
    lse = lse_of(case)
    kw = dict(real_vocab=1000)
    ref = rlk.fused_lmhead_backward(case.h, case.w, case.tgt, case.mask, lse, case.g, None, **kw)
    off = ~case.active
    assert off.any() and case.active.any()
    gen = torch.Generator(device=DEV).manual_seed(1)
    h = case.h.clone()
    h[off] = C.garbage((int(off.sum()), 128), gen, DEV)
    lse2, g2 = lse.clone(), case.g.clone()
    lse2[off] = float("nan")
    g2[off] = float("inf")
    tgt2 = case.tgt.clone()
    tgt2[~case.mask] = 2 ** 31 - 1
    got = rlk.fused_lmhead_backward(h, case.w, tgt2, case.mask, lse2, g2, None, **kw)
    assert torch.equal(bits(got[0]), bits(ref[0])) and torch.equal(bits(got[1]), bits(ref[1]))
    assert (bits(got[0][off]) == 0).all()
    # an active row with g == 0 and no LSE term is not reached either
    g3 = case.g.clone()
    row = int(case.active.nonzero()[0])
    g3[row] = 0.0
    h[row] = float("nan")
    got = rlk.fused_lmhead_backward(h, case.w, case.tgt, case.mask, lse2, g3, None, **kw)
    assert torch.isfinite(got[0].float()).all() and torch.isfinite(got[1].float()).all()
    assert (bits(got[0][row]) == 0).all()


def test_no_live_row():
    for n in (20, 70):
        no_live_row(n)


def no_live_row(n):
    case = C.make_case(n, 64, 600, 640, 9, DEV)
    none = torch.zeros(n, dtype=torch.bool, device=DEV)
    lse = lse_of(case)
    for mask, g in ((none, case.g), (case.mask, torch.zeros(n, device=DEV))):
        dh, dw = rlk.fused_lmhead_backward(case.h, case.w, case.tgt, mask, lse, g, None,
                                           real_vocab=600)
        assert (bits(dh) == 0).all() and (bits(dw) == 0).all()
    # no token at all: dweight is zero
    dh, dw = rlk.fused_lmhead_backward(case.h[:0], case.w, case.tgt[:0], None, lse[:0],
                                       case.g[:0], None, real_vocab=600)
    assert dh.shape == (0, 64) and (bits(dw) == 0).all()


def test_bad_target_and_validate():
    case = C.make_case(40, 64, 600, 640, 10, DEV, mask_keep=1.0, ignore_frac=0.0)
    lse = lse_of(case)
    tgt = case.tgt.clone()
    tgt[5] = 610  # a padded column
    dh, dw = rlk.fused_lmhead_backward(case.h, case.w, tgt, None, lse, case.g, None,
                                       real_vocab=600)
    rows = torch.arange(40, device=DEV) != 5
    assert torch.isnan(dh[5].float()).all() and torch.isfinite(dh[rows].float()).all()
    assert torch.isnan(dw[:600].float()).all() and (bits(dw[600:]) == 0).all()
    with pytest.raises(rlk.RlkError) as ei:
        rlk.fused_lmhead_backward(case.h, case.w, tgt, None, lse, case.g, None, real_vocab=600,
                                  validate=True)
    assert ei.value.status == rlk.RLK_ERR_TARGET_RANGE
    rlk.fused_lmhead_backward(case.h, case.w, case.tgt, None, lse, case.g, None, real_vocab=600,
                              validate=True)


@pytest.mark.parametrize("n", [50, 90])
def test_non_finite_rows_stay_in_their_rows(n):
    """An infinite upstream gradient, or a hidden state that is not finite, reaches its row
    of dhidden; the other rows keep their bits.  The scale is taken from finite gradients."""
    case = C.make_case(n, 64, 600, 600, 12, DEV, mask_keep=1.0, ignore_frac=0.0)
    lse = lse_of(case)
    top = int(case.g.abs().argmax())  # this row keeps the scale what it was
    row = (top + 1) % n
    ref, _ = rlk.fused_lmhead_backward(case.h, case.w, case.tgt, None, lse, case.g, None,
                                       real_vocab=600)
    rest = torch.arange(n, device=DEV) != row
    g = case.g.clone()
    g[row] = float("inf")
    dh, _ = rlk.fused_lmhead_backward(case.h, case.w, case.tgt, None, lse, g, None,
                                      real_vocab=600)
    assert torch.equal(bits(dh[rest]), bits(ref[rest]))
    assert not torch.isfinite(dh[row].float()).any()
    h = case.h.clone()
    h[row, 3] = float("nan")
    lse2 = lse.clone()
    lse2[row] = float("nan")
    dh, dw = rlk.fused_lmhead_backward(h, case.w, case.tgt, None, lse2, case.g, None,
                                       real_vocab=600)
    assert torch.equal(bits(dh[rest]), bits(ref[rest]))
    assert torch.isnan(dh[row].float()).all() and torch.isnan(dw.float()).all()


@pytest.mark.parametrize("n", [20, 300])
def test_infinite_weight_stays_in_its_row(n):
    """A weight entry of -inf where every hidden state is positive: that logit is -inf, its
    probability 0 and its row of dweight 0; the rows gathered behind the last live one meet it
    with hidden states of zero (0 * inf), which must not show."""
    case = C.make_case(n, 64, 600, 600, 13, DEV)
    case.h[:, 7] = case.h[:, 7].abs() + 0.125
    case.tgt[case.tgt == 100] = 99
    case.w[100, 7] = float("-inf")
    lse = lse_of(case)
    assert lse.isfinite().all()
    _, dw = rlk.fused_lmhead_backward(case.h, case.w, case.tgt, case.mask, lse, case.g, case.gl,
                                      real_vocab=600, want_hidden=False)
    assert dw.float().isfinite().all() and (dw[100] == 0).all()


@pytest.mark.parametrize("n", [9, 100, 300])
def test_workspace_contents_do_not_matter(n):
    case = C.make_case(n, 128, 1000, 1024, 21, DEV)
    lse = lse_of(case)
    desc = rlk.make_desc(n, 1000, 1024, 1024, 4)
    need = rlk.rlk_logp_fused_lmhead_bwd_workspace_bytes(desc, 128, True, True)
    out = []
    for fill in (0, 255, 127):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        dh, dw = torch.empty_like(case.h), torch.empty_like(case.w)
        rlk.rlk_logp_fused_lmhead_bwd(desc, case.h, case.w, 128, case.tgt,
                                      case.mask.view(torch.uint8), lse, case.g, case.gl, dh, dw,
                                      ws)
        out.append((bits(dh).clone(), bits(dw).clone()))
    for o in out[1:]:
        assert torch.equal(o[0], out[0][0]) and torch.equal(o[1], out[0][1])


def test_forward_rows_do_not_depend_on_the_batch():
    """The forward's streaming kernel (up to 64 tokens) and its tiles of 128 (65, 128 tokens),
    192 (333, 777) and 256 (1024) give a token the same bits, whatever the virtual shards."""
    case = C.make_case(1024, 64, 50021, 50176, 19, DEV)
    kw = dict(real_vocab=50021, num_vocab_tiles=61)
    logp, lse = rlk.fused_lmhead(case.h, case.w, case.tgt, case.mask, **kw)
    for n in (1, 16, 17, 40, 64, 65, 128, 333, 777):
        for at in (0, 1024 - n):
            rows = slice(at, at + n)
            for shards in (1, 3):
                got = rlk.fused_lmhead(case.h[rows], case.w, case.tgt[rows], case.mask[rows],
                                       num_virtual_shards=shards, **kw)
                assert torch.equal(bits(got[0]), bits(logp[rows])), (n, shards)
                assert torch.equal(bits(got[1]), bits(lse[rows])), (n, shards)


def test_autograd_function():
    """The differentiable function: autograd's gradients are the backward call's, a leaf
    that needs none costs none, and the loss moves along the gradient as the plain loss
    in 64 bits does (central differences)."""
    case = C.make_case(90, 128, 700, 768, 31, DEV, scale=1.0 / 90)
    case.w[700:] = 0.0
    h = case.h.clone().requires_grad_(True)
    w = case.w.clone().requires_grad_(True)
    kw = dict(real_vocab=700, num_vocab_tiles=3)
    logp, lse = rlk.lmhead_selected_token_logprob(h, w, case.tgt, case.mask, **kw)
    ref = rlk.fused_lmhead(case.h, case.w, case.tgt, case.mask, **kw)
    assert torch.equal(bits(logp), bits(ref[0])) and torch.equal(bits(lse), bits(ref[1]))
    ((logp * case.g).sum() + (lse * case.gl).sum()).backward()
    dh, dw = rlk.fused_lmhead_backward(case.h, case.w, case.tgt, case.mask, ref[1], case.g,
                                       case.gl, real_vocab=700)
    assert torch.equal(bits(h.grad), bits(dh)) and torch.equal(bits(w.grad), bits(dw))

    # only the hidden states; a broadcast gradient (of a sum); LSE not used
    h2 = case.h.clone().requires_grad_(True)
    logp, _ = rlk.lmhead_selected_token_logprob(h2, case.w, case.tgt, case.mask, **kw)
    (-logp.sum()).backward()
    dh2, _ = rlk.fused_lmhead_backward(case.h, case.w, case.tgt, case.mask, ref[1],
                                       torch.full((90,), -1.0, device=DEV), None, real_vocab=700)
    assert torch.equal(bits(h2.grad), bits(dh2))

    def loss(hh, ww):
        z = hh @ ww.T
        l64 = torch.logsumexp(z, 1)
        at = torch.where(case.active, case.tgt, 0).long()[:, None]
        lp = torch.where(case.active, z.gather(1, at)[:, 0] - l64, 0.0)
        return float((lp * case.g.double()).sum() + (l64 * case.gl.double()).sum())

    h64, w64 = case.h.double(), case.w[:700].double()
    gen = torch.Generator(device=DEV).manual_seed(4)
    eps = 1e-4
    for name, x, grad in (("hidden", h64, dh), ("weight", w64, dw[:700])):
        d = torch.randn(x.shape, generator=gen, device=DEV, dtype=torch.float64)
        # lean towards the gradient, so that the derivative along d does not cancel
        d = d / d.norm() + grad.double() / grad.double().norm()
        hp = (h64 + eps * d, w64) if name == "hidden" else (h64, w64 + eps * d)
        hm = (h64 - eps * d, w64) if name == "hidden" else (h64, w64 - eps * d)
        numeric = (loss(*hp) - loss(*hm)) / (2 * eps)
        along = float((grad.double() * d).sum())
        # the gradient's own error is at most 2^-7 of its norm (two roundings of half a
        # step), and d has a norm of at most 2; the difference's is of the order eps^2
        tol = 2 * 2.0 ** -7 * float(grad.double().norm())
        print(f"{name}: {along:.6e} against {numeric:.6e} (tolerance {tol:.1e})", flush=True)
        assert abs(along - numeric) <= tol


@pytest.mark.parametrize("n", [30, 300])
def test_other_stream_and_graph_replays(n):
    """A captured forward and backward, replayed on changing inputs with eager work between,
    gives the eager bits; a call on a side stream gives them too."""
    k, v, pad = 128, 5000, 5120
    sets = [C.make_case(n, k, v, pad, s, DEV, mask_keep=keep)
            for s, keep in ((41, 0.8), (42, 0.2), (43, 1.0))]
    names = ("h", "w", "tgt", "mask", "g", "gl")
    st = {m: getattr(sets[0], m).clone() for m in names}
    desc = rlk.make_desc(n, v, pad, pad, 16)
    w_f = torch.empty(rlk.rlk_logp_fused_lmhead_workspace_bytes(desc), dtype=torch.uint8,
                      device=DEV)
    w_b = torch.empty(rlk.rlk_logp_fused_lmhead_bwd_workspace_bytes(desc, k, True, True),
                      dtype=torch.uint8, device=DEV)

    def outputs():
        return {"logp": torch.empty(n, device=DEV), "lse": torch.empty(n, device=DEV),
                "dh": torch.empty((n, k), dtype=torch.bfloat16, device=DEV),
                "dw": torch.empty((pad, k), dtype=torch.bfloat16, device=DEV)}

    def calls(o):
        m = st["mask"].view(torch.uint8)
        rlk.rlk_logp_fused_lmhead(desc, st["h"], st["w"], k, st["tgt"], m, o["logp"], o["lse"],
                                  w_f)
        rlk.rlk_logp_fused_lmhead_bwd(desc, st["h"], st["w"], k, st["tgt"], m, o["lse"], st["g"],
                                      st["gl"], o["dh"], o["dw"], w_b)

    def load(i):
        for m in names:
            st[m].copy_(getattr(sets[i], m))

    refs = []
    for i in range(3):
        load(i)
        o = outputs()
        calls(o)
        torch.cuda.synchronize()
        refs.append({m: bits(x).clone() for m, x in o.items()})
    side = torch.cuda.Stream()
    load(1)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = outputs()
        calls(o)
    side.synchronize()
    for m, x in o.items():
        assert torch.equal(bits(x), refs[1][m]), m
    og = outputs()
    load(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(og)
    torch.cuda.synchronize()
    for rep, i in enumerate((1, 0, 2, 2, 1)):
        print(f"replay {rep} on set {i}", flush=True)
        load(i)
        graph.replay()
        torch.cuda.synchronize()
        for m, x in og.items():
            assert torch.equal(bits(x), refs[i][m]), f"{m} differs on replay {rep}"
        o = outputs()
        calls(o)
        torch.cuda.synchronize()


def test_calls_on_several_streams_at_once():
    """Gradients and 8-bit statistics of three batches, each on a stream of its own, in turn
    and without waiting: the bits of the calls made alone."""
    kw = dict(real_vocab=12003)
    runs = []
    for n in (30, 100, 500):
        case = C.make_case(n, 512, 12003, 12003, n, DEV)
        pair = rlk.quantize_fp8(case.w, 128)
        _, lse = rlk.fused_lmhead(case.h, case.w, case.tgt, case.mask, num_vocab_tiles=40, **kw)

        def call(stream=None, case=case, pair=pair, lse=lse):
            return (*rlk.fused_lmhead_backward(case.h, case.w, case.tgt, case.mask, lse, case.g,
                                               case.gl, stream=stream, **kw),
                    *rlk.fused_lmhead_fp8(case.h, *pair, case.tgt, case.mask, stream=stream,
                                          num_vocab_tiles=40, **kw))
        runs.append((call, call(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [(call(stream), ref) for _ in range(10) for call, ref, stream in runs]
    torch.cuda.synchronize()
    for i, (out, ref) in enumerate(got):
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, ref)), i


def test_no_token_through_autograd():
    case = C.make_case(5, 64, 300, 300, 8, DEV)
    h, w = case.h[:0].clone().requires_grad_(True), case.w.clone().requires_grad_(True)
    logp, lse = rlk.lmhead_selected_token_logprob(h, w, case.tgt[:0], None, real_vocab=300,
                                                  num_vocab_tiles=1)
    (logp.sum() + lse.sum()).backward()
    assert h.grad.shape == (0, 64) and (bits(w.grad) == 0).all()


@pytest.mark.parametrize("n", [30, 300])
def test_captured_training_step(n):
    """Forward, loss and autograd's backward captured as one graph (no eager graph of the same
    leaves alive), replayed on changing inputs with eager steps on other leaves between."""
    k, v = 128, 2900
    sets = [C.make_case(n, k, v, v, s, DEV) for s in (51, 52, 53)]
    names = ("h", "w", "tgt", "mask", "g", "gl")
    st = {m: getattr(sets[0], m).clone() for m in names}

    def step(h, w, tgt, mask, g, gl):
        h, w = h.detach().requires_grad_(True), w.detach().requires_grad_(True)
        logp, lse = rlk.lmhead_selected_token_logprob(h, w, tgt, mask, real_vocab=v,
                                                      num_vocab_tiles=7)
        loss = (logp * g).sum() + (lse * gl).sum()
        return (loss.detach(), *torch.autograd.grad(loss, (h, w)))

    def eager(i):
        return [bits(x).clone() for x in step(*(getattr(sets[i], m) for m in names))[1:]]

    refs = [eager(i) for i in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # autograd's own warm-up, off the capturing stream
        step(*(st[m] for m in names))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*(st[m] for m in names))
    torch.cuda.synchronize()
    for rep, i in enumerate((1, 0, 2, 2, 1)):
        print(f"replay {rep} on set {i}", flush=True)
        for m in names:
            st[m].copy_(getattr(sets[i], m))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out[1:], refs[i]):
            assert torch.equal(bits(a), b), f"replay {rep}"
        assert all(torch.equal(a, b) for a, b in zip(eager(2 - i), refs[2 - i]))


def test_second_derivatives_are_refused():
    case = C.make_case(20, 64, 300, 300, 3, DEV)
    h = case.h.clone().requires_grad_(True)
    logp, _ = rlk.lmhead_selected_token_logprob(h, case.w, case.tgt, case.mask, real_vocab=300,
                                                num_vocab_tiles=1)
    (grad,) = torch.autograd.grad(logp.sum(), h, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|does not require grad"):
        grad.float().sum().backward()


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
