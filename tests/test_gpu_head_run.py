"""The prediction head's products, its logits, the logit rules and the selected-token
log-probability together, as they are used: decoding, a training step, captured graphs, several
streams, split launches, tensors past 2^32 bytes.  Needs an MI355X."""
from __future__ import annotations

import os
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import vocab_selected_token_amd as rlk
from tests import linear_cases as L
from tests import process_cases as P
from tests.head_child import run_all, run_halves
from tests.test_gpu_streams import check as check_beside_a_busy_stream

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
BF16 = torch.bfloat16
ROOT = Path(__file__).resolve().parent.parent
K, V, PAD, CAP = 192, 3001, 3016, 6.0


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def head_inputs(n, seed):
    """Hidden states, a residual block, an LM-head and rules for n rows."""
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    p = P.make_case(n, V, PAD, seed, DEV, "all")
    return {"h": normal(n, K).bfloat16(), "w1": (normal(K, K) * 0.1).bfloat16(),
            "b1": normal(K).bfloat16(), "w2": (normal(V, K) * 0.3).bfloat16(),
            "b2": normal(V), "tgt": p.tgt, "mask": p.mask, "g": p.g, "gl": p.gl,
            **{"r_" + k: t for k, t in p.rules.items()}}


def rules_of(s):
    return rlk.LogitRules(**{k[2:]: t for k, t in s.items() if k.startswith("r_")})


def block(s):
    return rlk.linear_forward(s["h"], s["w1"], s["b1"], s["h"], activation="silu")[0]


@pytest.mark.parametrize("n", [1, 20, 90])
def test_decoding(n):
    """Block, logits, rules in place, and the logp of the token that was chosen: the existing
    forward() of the processed bf16 logits differs from the fused one by their rounding alone."""
    s = head_inputs(n, 5 + n)
    h = block(s)
    c = L.Case(s["h"], s["w1"], s["b1"], s["h"], torch.zeros(n, K, device=DEV), "silu")
    assert L.worst(h, *L.forward64(c)) <= 1.0
    z = rlk.lmhead_logits(h, s["w2"], s["b2"], cap=CAP, real_vocab=V, padded_vocab=PAD)
    raw = z.clone()
    rules = rules_of(s)
    fused = rlk.processed_forward(z, s["tgt"], rules, s["mask"], real_vocab=V)
    y = rlk.process_logits(z, rules, real_vocab=V, out=z)
    case = P.Case(raw, V, PAD, {k[2:]: t for k, t in s.items() if k.startswith("r_")}, s["tgt"],
                  s["mask"], s["g"], s["gl"])
    want, _, err = P.processed64(case)
    odd = want == -torch.inf
    bound = torch.where(odd, 0.0, err + P.HALF_BF16 * (want.abs() + err))
    assert P.worst(y[:, :V], want, bound) <= 1.0
    logp, lse = rlk.forward(y, s["tgt"], s["mask"], real_vocab=V, num_vocab_tiles=11)
    logp64, lse64, *_, e_logp, e_lse, _ = P.logp64(case)
    # each rounded y is off by half a step at most, and so is the LSE by the largest of them
    step = P.HALF_BF16 * torch.where(odd, 0.0, want.abs()).amax(1)
    assert ((lse.double() - lse64).abs() <= step + 2 * e_lse).all()
    assert ((logp.double() - logp64).abs() <= 2 * step + 2 * e_logp).all()
    assert P.worst(fused[0], logp64, e_logp) <= 1.0 and P.worst(fused[1], lse64, e_lse) <= 1.0


def step(s):
    """Loss and gradients of one training step through all of it."""
    h, w1, b1, w2, b2 = (s[k].detach().requires_grad_(True) for k in ("h", "w1", "b1", "w2", "b2"))
    y = rlk.head_linear(h, w1, b1, h, activation="silu")
    z = rlk.head_linear(y, w2, b2, activation="softcap", cap=CAP)
    logp, lse = rlk.processed_selected_token_logprob(z, s["tgt"], rules_of(s), s["mask"],
                                                     real_vocab=V)
    loss = (logp * s["g"]).sum() + (lse * s["gl"]).sum()
    return [loss.detach(), *torch.autograd.grad(loss, (h, w1, b1, w2, b2))]


@pytest.mark.parametrize("n", [2, 40, 200])
def test_training_step(n):
    """Autograd's step is the raw calls one after another, bit for bit (the products are held to 64
    bits where they are tested, the log-probabilities and their gradient here)."""
    s = head_inputs(n, 50 + n)
    loss, dh, dw1, db1, dw2, db2 = step(s)
    rules = rules_of(s)
    y, y_saved = rlk.linear_forward(s["h"], s["w1"], s["b1"], s["h"], activation="silu",
                                    save=True)
    z, z_saved = rlk.linear_forward(y, s["w2"], s["b2"], activation="softcap", cap=CAP, save=True)
    logp, lse = rlk.processed_forward(z, s["tgt"], rules, s["mask"], real_vocab=V)
    dz = rlk.processed_backward(z, s["tgt"], rules, s["mask"], lse, s["g"], s["gl"], real_vocab=V,
                                out_dtype=BF16)
    dy, rw2, rb2 = rlk.linear_backward(y, s["w2"], dz, z_saved, activation="softcap", cap=CAP,
                                       want_bias=True)
    dh1, rw1, rb1 = rlk.linear_backward(s["h"], s["w1"], dy, y_saved, activation="silu",
                                        want_bias=True, bias_dtype=BF16)
    for got, want in ((dw1, rw1), (db1, rb1), (dw2, rw2), (db2, rb2), (dh, dh1 + dy)):
        assert torch.equal(bits(got), bits(want))
    case = P.Case(z.detach(), V, V, {k[2:]: t for k, t in s.items() if k.startswith("r_")},
                  s["tgt"], s["mask"], s["g"], s["gl"])
    logp64, lse64, *_, e_logp, e_lse, _ = P.logp64(case)
    assert P.worst(logp, logp64, e_logp) <= 1.0 and P.worst(lse, lse64, e_lse) <= 1.0
    want, err = P.gradient64(case, s["g"], s["gl"], P.HALF_BF16)
    assert P.worst(dz, want, err) <= 1.0


def calls(s, o, ws):
    """Every entry point once, on buffers that are there."""
    n = s["h"].shape[0]
    mask = s["mask"].view(torch.uint8)
    d1 = rlk.rlk_linear_desc(n, K, K, K, K, K, K, rlk.ACTIVATIONS["silu"], rlk.RLK_DTYPE_BF16,
                             rlk.RLK_DTYPE_F16, 0.0)
    d2 = rlk.rlk_linear_desc(n, K, V, PAD, PAD, 0, PAD, rlk.ACTIVATIONS["softcap"],
                             rlk.RLK_DTYPE_F32, rlk.RLK_DTYPE_F32, CAP)
    dl = rlk.make_desc(n, V, PAD, PAD, 1)
    r = rules_of(s).struct
    rlk.rlk_linear_fwd(d1, s["h"], s["w1"], s["b1"], s["h"], o["y"], o["ysaved"])
    rlk.rlk_linear_fwd(d2, o["y"], s["w2"], s["b2"], None, o["z"], o["zsaved"])
    rlk.rlk_logits_process(dl, o["z"], r, o["p"], PAD, rlk.RLK_DTYPE_F32)
    rlk.rlk_logp_processed_fwd(dl, o["z"], r, s["tgt"], mask, o["logp"], o["lse"], ws[0])
    rlk.rlk_logp_processed_bwd(dl, o["z"], r, s["tgt"], mask, o["lse"], s["g"], s["gl"], o["dz"],
                               PAD, rlk.RLK_DTYPE_BF16, ws[0])
    rlk.rlk_linear_bwd(d2, o["y"], s["w2"], o["zsaved"], o["dz"], PAD, o["dy"], o["dw2"], o["db2"],
                       ws[1])
    rlk.rlk_linear_bwd(d1, s["h"], s["w1"], o["ysaved"], o["dy"], K, o["dh"], o["dw1"], o["db1"],
                       ws[2])
    return d1, d2, dl


def buffers(n):
    def e(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device=DEV)

    f = torch.float32
    return {"y": e(n, K), "ysaved": e(n, K, dtype=torch.float16), "z": e(n, PAD),
            "zsaved": e(n, PAD, dtype=f), "p": e(n, PAD, dtype=f), "logp": e(n, dtype=f),
            "lse": e(n, dtype=f), "dz": e(n, PAD), "dy": e(n, K), "dw2": e(V, K),
            "db2": e(V, dtype=f), "dh": e(n, K), "dw1": e(K, K), "db1": e(K)}


@pytest.mark.parametrize("n", [3, 90])
def test_graph_replays_match_eager(n):
    """All calls captured as one graph and replayed on changing inputs, with eager calls on the
    same buffers between; inputs are shared, so histories have one length."""
    sets = [head_inputs(n, 70 + i) for i in range(3)]
    total = max(s["r_history"].numel() for s in sets)
    for s in sets:
        s["r_history"] = torch.nn.functional.pad(s["r_history"], (0, total - s["r_history"].numel()))
    st = {k: torch.empty_like(t) for k, t in sets[0].items()}
    ws = [torch.empty(8 << 20, dtype=torch.uint8, device=DEV) for _ in range(3)]

    def load(i):
        for k, t in sets[i].items():
            st[k].copy_(t)

    refs = []
    for i in range(3):
        load(i)
        o = buffers(n)
        for t in o.values():
            t.fill_(3)
        d1, d2, dl = calls(st, o, ws)
        torch.cuda.synchronize()
        refs.append({k: bits(t[:, :V] if k in ("z", "zsaved", "p", "dz") else t).clone()
                     for k, t in o.items()})
    assert rlk.rlk_linear_bwd_workspace_bytes(d2) <= 8 << 20
    og = buffers(n)
    load(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(st, og, ws)
    torch.cuda.synchronize()
    for rep, i in enumerate((1, 0, 2, 2, 1)):
        print(f"replay {rep} on set {i}", flush=True)
        load(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, t in og.items():
            got = bits(t[:, :V] if k in ("z", "zsaved", "p", "dz") else t)
            assert torch.equal(got, refs[i][k]), f"{k} differs on replay {rep}"
        calls(st, og, ws)
        torch.cuda.synchronize()


def test_captured_training_step():
    """Forward, loss and autograd's backward as one graph (no eager graph of the same leaves
    alive), replayed on changing inputs with eager steps on other leaves between."""
    n = 40
    sets = [head_inputs(n, 80 + i) for i in range(3)]
    total = max(s["r_history"].numel() for s in sets)
    for s in sets:
        s["r_history"] = torch.nn.functional.pad(s["r_history"], (0, total - s["r_history"].numel()))
    st = {k: t.clone() for k, t in sets[0].items()}
    refs = [[bits(t).clone() for t in step(s)[1:]] for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # autograd's own warm-up, off the capturing stream
        step(st)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(st)
    torch.cuda.synchronize()
    for rep, i in enumerate((1, 0, 2, 2)):
        print(f"replay {rep} on set {i}", flush=True)
        for k, t in sets[i].items():
            st[k].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        # (the loss is torch's own sum)
        assert all(torch.equal(bits(a), b) for a, b in zip(outs[1:], refs[i])), rep
        step(sets[(i + 1) % 3])
        torch.cuda.synchronize()


def test_calls_on_several_streams_at_once():
    runs = []
    for n in (3, 60, 150):
        s = head_inputs(n, 90 + n)
        rules = rules_of(s)
        z = rlk.lmhead_logits(block(s), s["w2"], s["b2"], real_vocab=V, padded_vocab=PAD)
        _, lse = rlk.processed_forward(z, s["tgt"], rules, s["mask"], real_vocab=V)
        _, saved = rlk.linear_forward(s["h"], s["w1"], activation="gelu", save=True)

        def call(stream=None, s=s, rules=rules, z=z, lse=lse, saved=saved):
            kw = dict(stream=stream)
            return (rlk.process_logits(z, rules, real_vocab=V, **kw),
                    *rlk.processed_forward(z, s["tgt"], rules, s["mask"], real_vocab=V, **kw),
                    rlk.processed_backward(z, s["tgt"], rules, s["mask"], lse, s["g"],
                                           real_vocab=V, **kw),
                    rlk.lmhead_logits(s["h"], s["w2"], s["b2"], real_vocab=V, **kw),
                    *rlk.linear_backward(s["h"], s["w1"], s["h"], saved, activation="gelu",
                                         want_bias=True, **kw))
        runs.append((call, call(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [(call(stream), ref) for _ in range(8) for call, ref, stream in runs]
    torch.cuda.synchronize()
    for i, (out, ref) in enumerate(got):
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, ref)), i


def raw_calls():
    s = head_inputs(100, 99)
    rules = rules_of(s)
    z = rlk.lmhead_logits(s["h"], s["w2"], s["b2"], real_vocab=V, padded_vocab=PAD)
    _, saved = rlk.linear_forward(s["h"], s["w1"], activation="silu", save=True)
    _, lse = rlk.processed_forward(z, s["tgt"], rules, s["mask"], real_vocab=V)
    torch.cuda.synchronize()
    return {
        "process_logits": lambda **kw: rlk.process_logits(z, rules, real_vocab=V, **kw),
        "processed_forward": lambda **kw: rlk.processed_forward(z, s["tgt"], rules, s["mask"],
                                                                real_vocab=V, **kw),
        "processed_backward": lambda **kw: rlk.processed_backward(
            z, s["tgt"], rules, s["mask"], lse, s["g"], real_vocab=V, **kw),
        "linear_forward": lambda **kw: rlk.linear_forward(s["h"], s["w1"], activation="silu",
                                                          save=True, **kw),
        "linear_backward": lambda **kw: rlk.linear_backward(s["h"], s["w1"], s["h"], saved,
                                                            activation="silu", want_bias=True,
                                                            **kw),
        "lmhead_logits": lambda **kw: rlk.lmhead_logits(s["h"], s["w2"], s["b2"], real_vocab=V,
                                                        **kw),
    }


@pytest.mark.parametrize("name", ["process_logits", "processed_forward", "processed_backward",
                                  "linear_forward", "linear_backward", "lmhead_logits"])
def test_calls_beside_a_busy_stream(name):
    print(f"case {name}", flush=True)
    check_beside_a_busy_stream(raw_calls()[name], ())


def test_split_launches_give_the_same_bits(tmp_path):
    ref = run_all()
    for limit in (1024, 70000):
        print(f"launch limit {limit} threads (child process)", flush=True)
        out = tmp_path / f"bits_{limit}.pt"
        env = dict(os.environ, RLK_MAX_LAUNCH_THREADS=str(limit))
        r = subprocess.run([sys.executable, "-u", "-m", "tests.head_child", str(out)], cwd=ROOT,
                           env=env, capture_output=True, text=True, timeout=100)
        assert r.returncode == 0, f"child with limit {limit} failed:\n{r.stdout[-2000:]}\n{r.stderr[-3000:]}"
        got = torch.load(out, weights_only=True)
        assert set(got) == set(ref)
        for key in ref:
            for a, b in zip(ref[key], got[key]):
                assert torch.equal(a, b), f"{key} differs with a {limit}-thread launch limit"


def test_split_launches_of_half_tiles(tmp_path):
    """Blocks of 512 threads: the second launch begins with whole tiles (after 1000 blocks), and
    among the halves (after 1290)."""
    (want,) = run_halves()["halves"]
    for blocks in (1000, 1290):
        print(f"launch limit {blocks} blocks (child process)", flush=True)
        out = tmp_path / f"halves_{blocks}.pt"
        env = dict(os.environ, RLK_MAX_LAUNCH_THREADS=str(512 * blocks))
        r = subprocess.run([sys.executable, "-u", "-m", "tests.head_child", str(out), "halves"],
                           cwd=ROOT, env=env, capture_output=True, text=True, timeout=100)
        assert r.returncode == 0, f"{r.stdout[-2000:]}\n{r.stderr[-3000:]}"
        (got,) = torch.load(out, weights_only=True)["halves"]
        assert torch.equal(got, want)


def test_rows_past_4_gib():
    """15000 rows of 151936 logits, 4.6 GB: the last rows have the bits that they have alone."""
    n, v = 15000, 151936
    x = torch.zeros(n, v, dtype=BF16, device=DEV)
    c = P.make_case(3, v, v, 3, DEV, "all")
    c.tgt[:], c.mask[:] = 7, True
    c.rules["allow_index"][:] = -1
    x[-3:] = torch.where(torch.isfinite(c.x.float()), c.x, 1.0)
    c.x = x[-3:].clone()
    many = {k: t if k in ("history", "bias", "allow") else torch.cat([t[:1].expand(n - 3), t])
            for k, t in c.rules.items()}
    tgt = torch.full((n,), 7, dtype=torch.int32, device=DEV)
    g = torch.cat([torch.zeros(n - 3, device=DEV), c.g])
    few, all_ = rlk.LogitRules(**c.rules), rlk.LogitRules(**many)
    logp, lse = rlk.processed_forward(x, tgt, all_, real_vocab=v)
    a, b = rlk.processed_forward(c.x, c.tgt, few, real_vocab=v)
    assert torch.equal(bits(logp[-3:]), bits(a)) and torch.equal(bits(lse[-3:]), bits(b))
    d = rlk.processed_backward(x, tgt, all_, None, lse, g, real_vocab=v, out_dtype=BF16)
    want = rlk.processed_backward(c.x, c.tgt, few, None, b, c.g, real_vocab=v, out_dtype=BF16)
    assert torch.equal(bits(d[-3:]), bits(want))
    rlk.process_logits(x, all_, real_vocab=v, out=x)
    assert torch.equal(bits(x[-3:]), bits(rlk.process_logits(c.x, few, real_vocab=v)))


def test_outputs_past_4_gib():
    """16000 tokens x 64 x 151936 in small whole numbers: the last rows and columns are exact."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    m, n = 16000, 151936
    x = torch.randint(-2, 3, (m, 64), generator=gen, device=DEV).bfloat16()
    w = torch.randint(-2, 3, (n, 64), generator=gen, device=DEV).bfloat16()
    y, _ = rlk.linear_forward(x, w)
    for rows, cols in ((slice(-9, None), slice(None)), (slice(None), slice(-9, None)),
                       (slice(14130, 14140), slice(70000, 90000))):
        want = x[rows].double() @ w[cols].double().T
        assert torch.equal(y[rows, cols], want.bfloat16())
