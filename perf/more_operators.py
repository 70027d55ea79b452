"""What the operators around the logits cost: what a sampler does to them, the
log-probability under the distribution that it samples from, and the dense products of a
prediction head.

Four operators, each in its plain form (elementary torch operations in 32 bits, rounded once
at the end) and, where ``own`` is true, as the calls a user makes of the library:

* ``process``  penalties for repeated tokens, a bias, a temperature and a grammar's mask, applied
  to bf16 logits in one pass.
* ``logp``     logp and LSE of the selected tokens under the processed logits, and the gradient of
  a loss that reads them, to the raw logits.
* ``linear``   residual + act(x . weight^T + bias) for inference: a head's residual block, or
  logits with a bias and a soft cap.
* ``train``    the same product with the gradients of all its inputs.
"""
import math

import torch

own = False

IGNORE = -100


def listed():
    return [
        # one sequence decodes: its newest token's logits under all rules at once
        {"name": "process_1", "op": "process", "n": 1, "v": 151936, "v_pad": 152576,
         "history": 2000, "prompt": 0.5, "biases": 1, "grammars": 1, "out": "bf16"},
        # 65 drafted tokens, odd vocabulary, fp32 out for a sampler of the caller's own
        {"name": "process_65", "op": "process", "n": 65, "v": 32003, "v_pad": 32003,
         "history": 700, "prompt": 0.3, "biases": 0, "grammars": 5, "out": "fp32"},
        # a full serving batch with long histories, few requests with a bias or a grammar
        {"name": "process_512", "op": "process", "n": 512, "v": 151936, "v_pad": 152576,
         "history": 8192, "prompt": 0.7, "biases": 3, "grammars": 8, "out": "bf16"},
        # two sequences of 16 tokens, 8 of them prompt: the smallest training step
        {"name": "logp_b2s16", "op": "logp", "n": 32, "v": 151936, "v_pad": 151936, "seq": 16,
         "prompt": 0.5, "keep": 1.0, "biases": 0, "grammars": 0, "lse_grad": False},
        # a 1024-token microbatch over the padded vocabulary, a quarter of it masked, with an
        # LSE penalty beside the policy-gradient loss, some tokens sampled under a grammar
        {"name": "logp_microbatch", "op": "logp", "n": 1024, "v": 151936, "v_pad": 152576,
         "seq": 128, "prompt": 0.0, "keep": 0.75, "biases": 0, "grammars": 6, "lse_grad": True},
        # one long sequence, an eighth of it prompt, with a banned-words bias
        {"name": "logp_s4096", "op": "logp", "n": 4096, "v": 151936, "v_pad": 151936, "seq": 4096,
         "prompt": 0.125, "keep": 1.0, "biases": 1, "grammars": 0, "lse_grad": False},
        # one token through a head's residual block while decoding
        {"name": "linear_1", "op": "linear", "n": 1, "k": 4096, "v": 4096, "v_pad": 4096,
         "act": "silu", "bias": "bf16", "residual": True},
        # 16 sequences decode together: logits with a bias and a soft cap
        {"name": "logits_16", "op": "linear", "n": 16, "k": 4096, "v": 151936, "v_pad": 152576,
         "act": "softcap", "bias": "fp32", "residual": False},
        # a microbatch's logits, kept for a loss of the caller's own
        {"name": "logits_1024", "op": "linear", "n": 1024, "k": 2048, "v": 151936,
         "v_pad": 152576, "act": "softcap", "bias": "none", "residual": False},
        # the head's residual block in the smallest training step
        {"name": "train_b2s16", "op": "train", "n": 32, "k": 1024, "v": 1024, "v_pad": 1024,
         "act": "silu", "bias": "bf16", "residual": True},
        # a dense layer with odd sizes and no residual
        {"name": "train_777", "op": "train", "n": 777, "k": 1088, "v": 2501, "v_pad": 2501,
         "act": "gelu", "bias": "fp32", "residual": False},
        # one long sequence through the residual block
        {"name": "train_s4096", "op": "train", "n": 4096, "k": 4096, "v": 4096, "v_pad": 4096,
         "act": "silu", "bias": "bf16", "residual": True},
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    op = rng.choice(("process", "logp", "linear", "train"))
    if op in ("process", "logp"):
        v = log_int(1000, 151936)
        case = {"op": op, "n": log_int(1, 512 if op == "process" else 4096), "v": v,
                "v_pad": rng.choice((v, -(-v // 128) * 128, -(-v // 1024) * 1024)),
                "biases": rng.choice((0, 1, 3)), "grammars": rng.choice((0, 1, 6))}
        if op == "process":
            return case | {"history": log_int(1, 8192), "prompt": rng.choice((0.0, 0.4, 1.0)),
                           "out": rng.choice(("bf16", "fp32"))}
        seq = log_int(1, case["n"])
        case["n"] -= case["n"] % seq
        return case | {"seq": seq, "prompt": rng.choice((0.0, 0.25)),
                       "keep": rng.choice((1.0, 0.75, 0.4)), "lse_grad": rng.random() < 0.4}
    act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu", "softcap"))
    bias = rng.choice(("none", "bf16", "fp32"))
    k = 64 * log_int(1, 64)
    if op == "linear" and rng.random() < 0.5:
        v = log_int(1000, 151936)
        return {"op": op, "n": log_int(1, 1024 * 2048 // max(k, 2048)), "k": k, "v": v,
                "v_pad": rng.choice((v, -(-v // 128) * 128)),
                "act": rng.choice(("none", "softcap")), "bias": bias, "residual": False}
    v = log_int(64, 4096)
    return {"op": op, "n": log_int(1, 4096), "k": k, "v": v, "v_pad": v, "act": act, "bias": bias,
            "residual": rng.random() < 0.5}


CAP = 30.0
SIZES = {"none": 0, "bf16": 2, "fp32": 4}


def history_tokens(case):
    """Tokens of all histories, about, each counted once where rows share them."""
    return case["n"] * case["history"] // 2 if case["op"] == "process" else case["n"]


def work(case):
    n, v, v_pad = case["n"], case["v"], case["v_pad"]
    if case["op"] in ("process", "logp"):
        tables = 4 * v * case["biases"] + v // 8 * case["grammars"] + 4 * history_tokens(case)
        if case["op"] == "process":
            return {"bytes": 2 * n * v + SIZES[case["out"]] * n * v_pad + tables + 48 * n,
                    "flops": 4 * n * v}
        return {"bytes": 2 * n * v + 2 * n * v_pad + tables + 64 * n, "flops": 16 * n * v}
    k = case["k"]
    data = 2 * n * k + 2 * v * k + SIZES[case["bias"]] * v
    if case["op"] == "linear":
        return {"bytes": data + 2 * n * v_pad + (2 * n * v if case["residual"] else 0),
                "flops": 2 * n * v * k}
    return {"bytes": 2 * data + 4 * n * v + (4 * n * v if case["residual"] else 0),
            "flops": 6 * n * v * k}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    make = logit_inputs if case["op"] in ("process", "logp") else linear_inputs
    return make(case, gen, dev) | {"case": case}


def logit_inputs(case, gen, dev):
    n, v, v_pad = case["n"], case["v"], case["v_pad"]

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    def tokens(count):
        """Few tokens are frequent and many are rare: the rank's logarithm is uniform."""
        return (torch.exp(uniform(count) * math.log(v)).long() - 1).clamp(0, v - 1)

    ld = -(-v_pad // 8) * 8
    logits = (torch.randn((n, ld), generator=gen, device=dev) * 2.5).to(torch.bfloat16)
    logits[:, v:] = math.nan  # padding may hold anything
    row = torch.arange(n, device=dev)
    if case["op"] == "process":
        # histories of every length up to the longest, one after another
        lengths = (uniform(n) * (case["history"] + 1)).long()
        if n == 1:
            lengths[:] = case["history"]
        ends = lengths.cumsum(0)
        begins = ends - lengths
        total = int(ends[-1])
        history = tokens(total)
        splits = begins + (lengths * case["prompt"]).long()
        targets = None
    else:
        # a token's history is what its own sequence holds in front of it
        seq, prompt = case["seq"], int(case["seq"] * case["prompt"])
        history = tokens(n)
        begins = row // seq * seq
        ends = row
        splits = torch.minimum(begins + prompt, ends)
        total = n // seq * (seq * (seq - 1) // 2)
        targets = history.roll(-1)
        mask = (uniform(n) < case["keep"]) & (row % seq >= prompt)
        # half the tokens are likely under the model
        at = row[uniform(n) < 0.5]
        logits[at, targets[at]] += 12.0
    state = {"logits": logits, "history": history.to(torch.int32), "begins": begins,
             "splits": splits, "ends": ends, "total": total,
             # most requests take one or two of the penalties
             "repetition": torch.where(uniform(n) < 0.6, 1.0 + 0.3 * uniform(n), 1.0),
             "presence": torch.where(uniform(n) < 0.4, 2.0 * uniform(n), 0.0),
             "frequency": torch.where(uniform(n) < 0.4, uniform(n), 0.0),
             "temperature": 0.6 + 0.6 * uniform(n),
             "bias": None, "bias_index": None, "allow": None, "allow_index": None}
    if case["biases"]:
        # a few words are pushed or banned
        state["bias"] = torch.where(uniform(case["biases"], v) < 0.002,
                                    20.0 * (uniform(case["biases"], v) - 0.7), 0.0)
        index = torch.randint(-1, case["biases"], (n,), generator=gen, device=dev)
        state["bias_index"] = (index if n > 1 else index * 0).to(torch.int32)
    if case["grammars"]:
        # a state of a grammar allows from a few hundred tokens up to most of them
        share = torch.exp(uniform(case["grammars"]) * math.log(0.003))
        allow = uniform(case["grammars"], -(-v // 32) * 32) < share[:, None]
        index = torch.randint(-1, case["grammars"], (n,), generator=gen, device=dev)
        if n == 1:
            index[:] = 0
        at = targets if targets is not None else tokens(n)  # no row without a token
        held = index >= 0
        allow[index[held], at[held]] = True
        bits = allow.view(case["grammars"], -1, 32).long() << torch.arange(32, device=dev)
        state["allow"] = bits.sum(2).to(torch.int32)  # (keeps the low 32 bits)
        state["allow_index"] = index.to(torch.int32)
    if case["op"] == "logp":
        # per-token weights of a policy gradient, averaged over the batch
        state["g"] = torch.randn(n, generator=gen, device=dev) / n
        state["gl"] = torch.randn(n, generator=gen, device=dev) / (10 * n) \
            if case["lse_grad"] else None
        state["targets"], state["mask"] = targets.to(torch.int32), mask
        logits.requires_grad_(True)
    return state


def linear_inputs(case, gen, dev):
    n, k, v = case["n"], case["k"], case["v"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    train = case["op"] == "train"
    # logits reach the bend of the soft cap
    sigma = (8.0 if case["act"] == "softcap" else 1.3) / math.sqrt(k)
    weight = (normal(case["v_pad"], k) * sigma).to(torch.bfloat16)
    state = {"x": normal(n, k).to(torch.bfloat16), "weight": weight, "bias": None, "residual": None}
    if case["bias"] != "none":
        state["bias"] = (normal(v) * 0.5).to(
            torch.bfloat16 if case["bias"] == "bf16" else torch.float32)
    if case["residual"]:
        state["residual"] = normal(n, v).to(torch.bfloat16)
    if train:
        state["dy"] = (normal(n, v) / n).to(torch.bfloat16)
        for name in ("x", "weight", "bias", "residual"):
            if state[name] is not None:
                state[name].requires_grad_(True)
    return state


def run(state):
    case = state["case"]
    if own:
        return run_own(state, case)
    with torch.no_grad():
        if case["op"] == "process":
            y, _ = plain_processed(state, case)
            y = torch.nn.functional.pad(y, (0, case["v_pad"] - case["v"]), value=-math.inf)
            return y.to(torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        if case["op"] == "logp":
            return plain_logp(state, case)
        return plain_linear(state, case)


def plain_counts(state, n, v):
    """How often each token occurs in each row's prompt and among its generated tokens."""
    dev = state["history"].device
    lengths = state["ends"] - state["begins"]
    rows = torch.repeat_interleave(torch.arange(n, device=dev), lengths,
                                   output_size=state["total"])
    at = torch.arange(state["total"], device=dev) - (lengths.cumsum(0) - lengths)[rows] \
        + state["begins"][rows]
    where = rows * v + state["history"][at].long()
    generated = (at >= state["splits"][rows]).int()
    of_prompt = torch.zeros(n * v, dtype=torch.int32, device=dev)
    of_output = of_prompt.clone()
    of_prompt.index_add_(0, where, 1 - generated)
    of_output.index_add_(0, where, generated)
    return of_prompt.view(n, v), of_output.view(n, v)


def plain_processed(state, case):
    """The processed logits in fp32 and their derivative to the raw ones."""
    n, v = case["n"], case["v"]
    x = state["logits"][:, :v].float()
    of_prompt, of_output = plain_counts(state, n, v)
    seen = (of_prompt + of_output) > 0
    rho = state["repetition"][:, None]
    slope = torch.where(seen, torch.where(x > 0, 1.0 / rho, rho), 1.0)
    y = torch.where(seen, torch.where(x > 0, x / rho, x * rho), x)
    y = y - state["frequency"][:, None] * of_output - state["presence"][:, None] * (of_output > 0)
    if state["bias"] is not None:
        index = state["bias_index"][:, None]
        y = y + torch.where(index >= 0, state["bias"][index[:, 0].clamp_min(0).long()], 0.0)
    y = y / state["temperature"][:, None]
    slope = slope / state["temperature"][:, None]
    if state["allow"] is not None:
        index = state["allow_index"][:, None]
        column = torch.arange(v, device=x.device)
        words = state["allow"][:, column // 32] >> (column % 32) & 1
        barred = (index >= 0) & (words[index[:, 0].clamp_min(0).long()] == 0)
        y = torch.where(barred, -math.inf, y)
        slope = torch.where(barred, 0.0, slope)
    return y, slope


def plain_logp(state, case):
    y, slope = plain_processed(state, case)
    top = y.amax(1)
    lse = top + (y - top[:, None]).exp().sum(1).log()
    act = state["mask"] & (state["targets"] != IGNORE)
    at = torch.where(act, state["targets"], 0).long()[:, None]
    logp = torch.where(act, y.gather(1, at)[:, 0] - lse, 0.0)
    g = torch.where(act, state["g"], 0.0)
    coef = -g if state["gl"] is None else state["gl"] - g
    # dy = g (onehot - p) + gl p
    dy = (y - lse[:, None]).exp() * coef[:, None]
    dy.scatter_add_(1, at, g[:, None])
    dx = torch.nn.functional.pad(dy * slope, (0, state["logits"].shape[1] - case["v"]))
    return logp, lse, dx.to(torch.bfloat16)


def plain_act(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).float()
    if act == "softcap":
        t = (z / CAP).tanh()
        return CAP * t, 1.0 - t * t
    if act == "silu":
        s = 1.0 / (1.0 + (-z).exp())
        return z * s, s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        phi = 0.5 * (1.0 + (z * math.sqrt(0.5)).erf())
        return z * phi, phi + z * (-0.5 * z * z).exp() * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = (c * (z + 0.044715 * z * z * z)).tanh()
    return 0.5 * z * (1.0 + t), \
        0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 0.134145 * z * z)


def plain_linear(state, case):
    v = case["v"]
    x, w = state["x"].float(), state["weight"][:v].float()
    z = x @ w.T
    if state["bias"] is not None:
        z = z + state["bias"].float()
    y, slope = plain_act(z, case["act"])
    if state["residual"] is not None:
        y = y + state["residual"].float()
    if case["op"] == "linear":
        y = torch.nn.functional.pad(y, (0, case["v_pad"] - v), value=-math.inf)
        return y.to(torch.bfloat16)
    dz = state["dy"].float() * slope
    out = [y.to(torch.bfloat16), (dz @ w).to(torch.bfloat16), (dz.T @ x).to(torch.bfloat16)]
    if state["bias"] is not None:
        out.append(dz.sum(0).to(state["bias"].dtype))
    if state["residual"] is not None:
        out.append(state["dy"])
    return out


def run_own(state, case):
    import vocab_selected_token_amd as rlk

    if case["op"] in ("process", "logp"):
        rules = rlk.LogitRules(
            repetition=state["repetition"], presence=state["presence"],
            frequency=state["frequency"], temperature=state["temperature"],
            history=state["history"], history_begin=state["begins"],
            history_split=state["splits"], history_end=state["ends"], bias=state["bias"],
            bias_index=state["bias_index"], allow=state["allow"],
            allow_index=state["allow_index"])
        size = {"real_vocab": case["v"], "padded_vocab": case["v_pad"]}
        if case["op"] == "process":
            return rlk.process_logits(
                state["logits"], rules, **size,
                out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        logp, lse = rlk.processed_selected_token_logprob(state["logits"], state["targets"], rules,
                                                         state["mask"], **size)
        outs, grads = ([logp], [state["g"]]) if state["gl"] is None else \
            ([logp, lse], [state["g"], state["gl"]])
        return [logp.detach(), lse.detach(), *torch.autograd.grad(outs, state["logits"], grads)]
    cap = CAP if case["act"] == "softcap" else None
    if case["op"] == "linear" and case["act"] in ("none", "softcap") and not case["residual"]:
        return rlk.lmhead_logits(state["x"], state["weight"], state["bias"], cap=cap,
                                 real_vocab=case["v"], padded_vocab=case["v_pad"])
    y = rlk.head_linear(state["x"], state["weight"], state["bias"], state["residual"],
                        activation=case["act"], cap=cap)
    if case["op"] == "linear":
        return y
    inputs = [state[name] for name in ("x", "weight", "bias", "residual")
              if state[name] is not None]
    return [y.detach(), *torch.autograd.grad(y, inputs, state["dy"])]


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        if case["op"] in ("linear", "train"):
            return exact_linear(case, s)
        n, v = case["n"], case["v"]
        step = max(1, (1 << 27) // v)
        parts = [exact_rows(case, s, r, min(n, r + step)) for r in range(0, n, step)]
        outs = [torch.cat(p) for p in zip(*parts)]
        return outs if case["op"] == "logp" else outs[0]


def exact_rows(case, s, r0, r1):
    v, dev = case["v"], s["logits"].device
    y = s["logits"][r0:r1, :v].double()
    per_row = {k: s[k][r0:r1].double()[:, None]
               for k in ("repetition", "presence", "frequency", "temperature")}
    slope = torch.ones_like(y)
    begins, splits, ends = (s[k][r0:r1].tolist() for k in ("begins", "splits", "ends"))

    def found(starts):
        """(row, token, how often) of the histories from `starts` on."""
        keys = [s["history"][b:e].long() + i * v for i, (b, e) in enumerate(zip(starts, ends))]
        key, count = torch.cat(keys).unique(return_counts=True)
        return key // v, key % v, count

    i, seen, _ = found(begins)
    of_y, rho = y[i, seen], per_row["repetition"][i, 0]
    slope[i, seen] = torch.where(of_y > 0, 1.0 / rho, rho)
    y[i, seen] = of_y * slope[i, seen]
    i, out, count = found(splits)
    y[i, out] -= per_row["frequency"][i, 0] * count + per_row["presence"][i, 0]
    if s["bias"] is not None:
        table = torch.cat([s["bias"].double(), s["bias"].new_zeros((1, v)).double()])
        y += table[s["bias_index"][r0:r1].long()]  # (index -1: the row of zeros)
    y /= per_row["temperature"]
    slope /= per_row["temperature"]
    if s["allow"] is not None:
        bits = s["allow"].long()[:, :, None].bitwise_right_shift(torch.arange(32, device=dev))
        free = (bits & 1).bool().flatten(1)[:, :v]
        free = torch.cat([free, free.new_ones((1, v))])[s["allow_index"][r0:r1].long()]
        y.masked_fill_(~free, -math.inf)
        slope.masked_fill_(~free, 0.0)
    if case["op"] == "process":
        out = torch.full((r1 - r0, case["v_pad"]), -math.inf, dtype=torch.float64, device=dev)
        out[:, :v] = y
        return (out,)
    lse = torch.logsumexp(y, 1)
    live = (s["mask"][r0:r1] & (s["targets"][r0:r1] != IGNORE)).nonzero()[:, 0]
    cols, g = s["targets"][r0:r1][live].long(), s["g"][r0:r1][live].double()
    logp = torch.zeros_like(lse)
    logp[live] = y[live, cols] - lse[live]
    # the loss is sum_r g_r logp_r + gl_r lse_r
    coef = torch.zeros_like(lse)
    coef[live] = -g
    if s["gl"] is not None:
        coef += s["gl"][r0:r1].double()
    dy = y.sub_(lse[:, None]).exp_().mul_(coef[:, None])
    dy[live, cols] += g
    dx = torch.zeros((r1 - r0, s["logits"].shape[1]), dtype=torch.float64, device=dev)
    dx[:, :v] = dy * slope
    return logp, lse, dx


def exact_linear(case, s):
    v = case["v"]
    x, w = s["x"].double(), s["weight"][:v].double()
    z = torch.mm(x, w.t())
    if s["bias"] is not None:
        z += s["bias"].double()
    with torch.enable_grad():
        z.requires_grad_(True)
        f = torch.nn.functional
        y = {"none": lambda t: t * 1.0, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
             "gelu_tanh": lambda t: f.gelu(t, approximate="tanh"),
             "softcap": lambda t: CAP * torch.tanh(t / CAP)}[case["act"]](z)
        if case["op"] == "train":
            dz, = torch.autograd.grad(y, z, s["dy"].double())
    y = y.detach()
    if s["residual"] is not None:
        y += s["residual"].double()
    if case["op"] == "linear":
        out = torch.full((case["n"], case["v_pad"]), -math.inf, dtype=torch.float64,
                         device=y.device)
        out[:, :v] = y
        return out
    outs = [y, dz.mm(w), dz.t().mm(x)]
    if s["bias"] is not None:
        outs.append(dz.sum(0))
    if s["residual"] is not None:
        outs.append(s["dy"].double())
    return outs
