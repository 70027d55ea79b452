"""What the LM-head operators cost: selected-token log-probability straight from
the hidden states with its gradients, and the same head with weights held in
8-bit floating point.

Four operators, each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and, where ``own`` is true, as the calls a user makes of
the library:

* ``train``   logp and LSE of z = hidden . weight^T, and the gradients of a loss
  that reads them, to the hidden states and to the weight: the softmax cross
  entropy of a language model is -logp.
* ``score8``  logp and LSE from an e4m3 weight with one scale per 128 x 128 block;
  the hidden states are cast within the call, one scale per token and 128 columns.
* ``logits8`` the same product, written out as bf16 logits.
* ``quant8``  the cast itself, by tokens (1 x 128) or for a weight (128 x 128).
"""
import math

import torch

own = False

BLOCK = 128            # columns (and weight rows) that share a scale
E4M3_MAX = 448.0       # the largest finite e4m3 value
SMALLEST = 2.0 ** -126  # a scale is never below the smallest normal number
IGNORE = -100


def listed():
    return [
        # two short sequences of 16 tokens, 8 of them prompt: the smallest training step
        {"name": "train_b2s16", "op": "train", "n": 32, "k": 1024, "v": 151936, "v_pad": 151936,
         "seq": 16, "prompt": 8, "keep": 1.0, "ignore": 0.0, "lse_grad": False, "wrt": "both"},
        # a 1024-token microbatch over the padded vocabulary, a quarter of it masked, with an
        # LSE penalty beside the policy-gradient loss
        {"name": "train_microbatch", "op": "train", "n": 1024, "k": 2048, "v": 151936,
         "v_pad": 152576, "seq": 128, "prompt": 0, "keep": 0.75, "ignore": 0.03, "lse_grad": True,
         "wrt": "both"},
        # odd sizes, head frozen: adapters are trained below it, so only the hidden states
        # need a gradient
        {"name": "train_frozen_head", "op": "train", "n": 777, "k": 1088, "v": 50021,
         "v_pad": 50176, "seq": 777, "prompt": 0, "keep": 0.9, "ignore": 0.05, "lse_grad": False,
         "wrt": "hidden"},
        # one long sequence, 512 tokens of it prompt: an ordinary large step
        {"name": "train_s4096", "op": "train", "n": 4096, "k": 4096, "v": 151936,
         "v_pad": 152576, "seq": 4096, "prompt": 512, "keep": 1.0, "ignore": 0.05,
         "lse_grad": False, "wrt": "both"},
        # one sequence's newest token is scored while decoding
        {"name": "score8_1", "op": "score8", "n": 1, "k": 4096, "v": 151936, "v_pad": 152576},
        # ragged: a mixed batch of short continuations, odd vocabulary
        {"name": "score8_333", "op": "score8", "n": 333, "k": 2176, "v": 50021, "v_pad": 50176},
        # a long sequence's log-probabilities under the rollout's 8-bit head
        {"name": "score8_s4096", "op": "score8", "n": 4096, "k": 4096, "v": 151936,
         "v_pad": 152576},
        # sampling: 16 sequences decode together
        {"name": "logits8_16", "op": "logits8", "n": 16, "k": 4096, "v": 151936,
         "v_pad": 152576},
        # drafted tokens of a few sequences, odd vocabulary
        {"name": "logits8_65", "op": "logits8", "n": 65, "k": 896, "v": 32003, "v_pad": 32003},
        # a microbatch's logits, kept for a loss of the caller's own
        {"name": "logits8_1024", "op": "logits8", "n": 1024, "k": 2048, "v": 151936,
         "v_pad": 152576},
        # the hidden states of a long sequence
        {"name": "quant8_tokens", "op": "quant8", "n": 4096, "k": 4096, "block_rows": 1},
        # the whole head, as after every weight update
        {"name": "quant8_weight", "op": "quant8", "n": 151936, "k": 4096, "block_rows": 128},
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    op = rng.choice(("train", "score8", "logits8", "quant8"))
    if op == "quant8":
        rows = rng.choice((1, BLOCK))
        return {"op": op, "n": log_int(1, 4096 if rows == 1 else 151936),
                "k": BLOCK * log_int(1, 32), "block_rows": rows}
    v = log_int(1000, 151936)
    case = {"op": op, "n": log_int(1, 4096), "v": v,
            "v_pad": rng.choice((v, -(-v // 128) * 128, -(-v // 1024) * 1024))}
    if op == "train":
        case |= {"k": 64 * log_int(1, 64), "seq": case["n"], "prompt": case["n"] // 8,
                 "keep": rng.choice((1.0, 0.75, 0.4)), "ignore": rng.choice((0.0, 0.05)),
                 "lse_grad": rng.random() < 0.4, "wrt": rng.choice(("both", "both", "hidden"))}
    else:
        case["k"] = BLOCK * log_int(1, 32)
    return case


def tiles(case):
    """64 tiles, or as many as leave at least 256 columns to each."""
    return max(1, min(64, case["v_pad"] // 256))


def live_share(case):
    """Which training rows reach the gradients, as a share."""
    return (1.0 - case["prompt"] / case["seq"]) * case["keep"] * (1.0 - case["ignore"])


def work(case):
    n, k = case["n"], case["k"]
    if case["op"] == "quant8":
        scales = -(-n // case["block_rows"]) * (k // BLOCK)
        return {"bytes": 3 * n * k + 4 * scales, "flops": 3 * n * k}
    v, v_pad = case["v"], case["v_pad"]
    if case["op"] == "train":
        both = case["wrt"] == "both"
        live = n if case["lse_grad"] else n * live_share(case)
        data = 2 * n * k * 2 + 2 * v * k + (2 * v_pad * k if both else 0)
        return {"bytes": data + 21 * n, "flops": 2 * n * v * k + (4 if both else 2) * live * v * k}
    data = 2 * n * k + v * k + 4 * -(-v // BLOCK) * (k // BLOCK)
    return {"bytes": data + (13 * n if case["op"] == "score8" else 2 * n * v_pad),
            "flops": 2 * n * v * k}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    n, k = case["n"], case["k"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["op"] == "quant8":
        x = normal(n, k)
        # a weight's entries, or hidden states with a few columns far above the rest
        x *= 0.02 if case["block_rows"] > 1 else 1.0 + 20.0 * (normal(k).abs() > 2.8)
        return {"case": case, "x": x.to(torch.bfloat16)}

    v, v_pad = case["v"], case["v_pad"]
    targets = torch.randint(0, v, (n,), generator=gen, device=dev)
    sigma = 1.3 / math.sqrt(k)
    weight = (normal(v_pad, k) * sigma).to(torch.bfloat16)
    # half the tokens are likely under the model: their hidden state leans to the target's
    # row so that its logit stands about 12 above the rest
    hidden = normal(n, k)
    lean = (torch.rand(n, generator=gen, device=dev) < 0.5).float() * (12.0 / (k * sigma * sigma))
    hidden = (hidden + lean[:, None] * weight[targets].float()).to(torch.bfloat16)
    mask = torch.rand(n, generator=gen, device=dev) < case.get("keep", 1.0)
    mask &= torch.arange(n, device=dev) % case.get("seq", 1) >= case.get("prompt", 0)
    targets[torch.rand(n, generator=gen, device=dev) < case.get("ignore", 0.0)] = IGNORE
    state = {"case": case, "hidden": hidden, "targets": targets.to(torch.int32), "mask": mask}
    if case["op"] == "train":
        # per-token weights of a policy gradient, averaged over the batch
        state["g"] = normal(n) / n
        state["gl"] = normal(n) / (10 * n) if case["lse_grad"] else None
        state["weight"] = weight.requires_grad_(case["wrt"] == "both")
        state["hidden"].requires_grad_(True)
    else:
        state["weight_q"], state["weight_scale"] = cast(weight, BLOCK)
    return state


def blocks_of(x, rows):
    """x [n, k] as [n / rows, rows, k / 128, 128], short blocks filled up with zeros."""
    n, k = x.shape
    x = torch.nn.functional.pad(x, (0, 0, 0, -n % rows))
    return x.reshape(-1, rows, k // BLOCK, BLOCK)


def cast(x, rows):
    """(e4m3 values, fp32 scale of each rows x 128 block): the scale maps the block's largest
    magnitude to 448."""
    b = blocks_of(x.float(), rows)
    # a quotient, not a product with 1/448: many entries lie midway between two e4m3 values, and
    # the last bit of the scale decides them
    most = torch.full((), E4M3_MAX, device=x.device)
    scale = (b.abs().amax((1, 3)) / most).clamp_min(SMALLEST)
    q = (b / scale[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.reshape(-1, x.shape[1])[: x.shape[0]], scale


def uncast(q, scale, rows):
    b = blocks_of(q.float(), rows) * scale[:, None, :, None]
    return b.reshape(-1, q.shape[1])[: q.shape[0]]


def run(state):
    case = state["case"]
    if own:
        return run_own(state, case)
    if case["op"] == "quant8":
        return cast(state["x"], case["block_rows"])
    v = case["v"]
    if case["op"] == "train":
        return plain_train(state, case)
    hidden = uncast(*cast(state["hidden"], 1), 1)
    z = hidden @ uncast(state["weight_q"], state["weight_scale"], BLOCK)[:v].T
    if case["op"] == "logits8":
        z = torch.nn.functional.pad(z, (0, case["v_pad"] - v), value=-math.inf)
        return z.to(torch.bfloat16)
    act = state["mask"] & (state["targets"] != IGNORE)
    return plain_logp(z, state["targets"], act)[:2]


def plain_logp(z, targets, act):
    """logp (0 on rows that are not active), LSE and the column to gather."""
    top = z.amax(1)
    lse = top + (z - top[:, None]).exp().sum(1).log()
    at = torch.where(act, targets, 0).long()[:, None]
    return torch.where(act, z.gather(1, at)[:, 0] - lse, 0.0), lse, at


def plain_train(state, case):
    v, g, gl = case["v"], state["g"], state["gl"]
    hidden = state["hidden"].detach().float()
    weight = state["weight"].detach()[:v].float()
    act = state["mask"] & (state["targets"] != IGNORE)
    z = hidden @ weight.T
    logp, lse, at = plain_logp(z, state["targets"], act)
    g = torch.where(act, g, 0.0)
    # dz = g (onehot - p) + gl p
    dz = (z - lse[:, None]).exp() * ((0.0 if gl is None else gl) - g)[:, None]
    dz.scatter_add_(1, at, g[:, None])
    out = [logp, lse, (dz @ weight).to(torch.bfloat16)]
    if case["wrt"] == "both":
        dw = torch.nn.functional.pad(dz.T @ hidden, (0, 0, 0, case["v_pad"] - v))
        out.append(dw.to(torch.bfloat16))
    return out


def run_own(state, case):
    import vocab_selected_token_amd as rlk

    if case["op"] == "quant8":
        return rlk.quantize_fp8(state["x"], case["block_rows"])
    size = {"real_vocab": case["v"], "padded_vocab": case["v_pad"]}
    if case["op"] == "logits8":
        return rlk.lmhead_logits_fp8(state["hidden"], state["weight_q"], state["weight_scale"],
                                     **size)
    size["num_vocab_tiles"] = tiles(case)
    if case["op"] == "score8":
        return rlk.fused_lmhead_fp8(state["hidden"], state["weight_q"], state["weight_scale"],
                                    state["targets"], state["mask"], **size)
    logp, lse = rlk.lmhead_selected_token_logprob(state["hidden"], state["weight"],
                                                  state["targets"], state["mask"], **size)
    wrt = [state["hidden"]] + ([state["weight"]] if case["wrt"] == "both" else [])
    outs, grads = ([logp], [state["g"]]) if state["gl"] is None else \
        ([logp, lse], [state["g"], state["gl"]])
    return [logp.detach(), lse.detach(), *torch.autograd.grad(outs, wrt, grads)]


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "quant8":
            return exact_cast(s["x"], case["block_rows"])
        v, n = case["v"], case["n"]
        if case["op"] == "train":
            h, w = s["hidden"].double(), s["weight"][:v].double()
        else:
            h, w = (exact_uncast(*exact_cast(s["hidden"], 1), 1),
                    exact_uncast(s["weight_q"], s["weight_scale"], BLOCK)[:v])
        z = torch.mm(h, w.t())
        if case["op"] == "logits8":
            out = torch.full((n, case["v_pad"]), -math.inf, dtype=torch.float64, device=z.device)
            out[:, :v] = z
            return out
        live = (s["mask"] & (s["targets"] != IGNORE)).nonzero()[:, 0]
        cols = s["targets"][live].long()
        lse = torch.logsumexp(z, 1)
        logp = torch.zeros(n, dtype=torch.float64, device=z.device)
        logp[live] = z[live, cols] - lse[live]
        if case["op"] == "score8":
            return logp, lse
        # the loss is sum_r g_r logp_r + gl_r lse_r
        coef = torch.zeros(n, dtype=torch.float64, device=z.device)
        coef[live] = -s["g"][live].double()
        if s["gl"] is not None:
            coef += s["gl"].double()
        dz = z.sub_(lse[:, None]).exp_().mul_(coef[:, None])
        dz[live, cols] += s["g"][live].double()
        outs = [logp, lse, dz.mm(w)]
        if case["wrt"] == "both":
            dw = torch.zeros((case["v_pad"], case["k"]), dtype=torch.float64, device=z.device)
            dw[:v] = dz.t().mm(h)
            outs.append(dw)
        return outs


def exact_cast(x, rows):
    """The cast's definition, computed in 64 bits: quotients are rounded to 32 bits, then to
    e4m3's 3 fraction bits (exponents from -6), to even."""
    n, k = x.shape
    q = torch.zeros((n, k), dtype=torch.float64, device=x.device)
    scale = torch.zeros((-(-n // rows), k // BLOCK), dtype=torch.float64, device=x.device)
    step = max(rows, 8192)
    for r0 in range(0, n, step):
        part = x[r0: r0 + step].double()
        ids = torch.arange(part.shape[0], device=x.device) // rows
        top = part.abs().unflatten(1, (-1, BLOCK)).amax(2)
        best = torch.zeros((int(ids[-1]) + 1, top.shape[1]), dtype=torch.float64, device=x.device)
        best = best.scatter_reduce(0, ids[:, None].expand_as(top), top, "amax")
        s = (best / E4M3_MAX).float().clamp_min(SMALLEST).double()
        scale[r0 // rows: r0 // rows + s.shape[0]] = s
        part = (part / s[ids].repeat_interleave(BLOCK, 1)).float().double()
        unit = torch.exp2(torch.floor(torch.log2(part.abs().clamp_min(2.0 ** -6))) - 3)
        q[r0: r0 + step] = (torch.round(part / unit) * unit).clamp(-E4M3_MAX, E4M3_MAX)
    return q, scale


def exact_uncast(q, scale, rows):
    ids = torch.arange(q.shape[0], device=q.device) // rows
    return q.double() * scale.double()[ids].repeat_interleave(BLOCK, 1)
