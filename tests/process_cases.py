"""Seeded cases of the logit rules and their plain form in 64 bits, with the error an fp32
kernel may make (input synthesis and arithmetic only)."""
from __future__ import annotations

import math
from dataclasses import dataclass, field

import torch

IGNORE = -100
HALF_BF16 = 2.0 ** -8   # half a step, relative
H = 2.0 ** -24          # of fp32
TINY = 1e-37            # what flushing subnormal results to zero may cost


@dataclass
class Case:
    x: torch.Tensor  # bf16 [N, pad rounded up to 8]; columns >= v hold random bit patterns
    v: int
    pad: int
    rules: dict = field(default_factory=dict)  # LogitRules' arguments
    tgt: torch.Tensor = None
    mask: torch.Tensor = None
    g: torch.Tensor = None
    gl: torch.Tensor = None

    @property
    def active(self):
        return self.mask & (self.tgt != IGNORE)

    def row(self, r):
        """The case of row r alone."""
        rules = {}
        for k, t in self.rules.items():
            one = k in ("history", "bias", "allow")
            if one and k != "history" and k + "_index" not in self.rules and t.dim() == 2 \
                    and t.shape[0] > 1:
                t = t[r: r + 1]
            rules[k] = t if one else t[r: r + 1].contiguous()
        return Case(self.x[r: r + 1].contiguous(), self.v, self.pad, rules,
                    *(t[r: r + 1].contiguous() for t in (self.tgt, self.mask, self.g, self.gl)))


def garbage(shape, gen, device):
    return torch.randint(-32768, 32768, shape, generator=gen, device=device,
                         dtype=torch.int32).to(torch.int16).view(torch.bfloat16)


KINDS = ("none", "penalties", "bias", "allow", "all")


def make_case(n, v, pad, seed, device, kind="all", longest=300):
    gen = torch.Generator(device=device).manual_seed(seed)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=device)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device=device)

    ld = (pad + 7) // 8 * 8
    x = (torch.randn((n, ld), generator=gen, device=device) * 3).to(torch.bfloat16)
    x[:, v:] = garbage((n, ld - v), gen, device)
    rules = {}
    if kind in ("penalties", "all"):
        rules["repetition"] = torch.where(uniform(n) < 0.7, 0.7 + uniform(n), 1.0)
        rules["presence"] = torch.where(uniform(n) < 0.5, uniform(n) * 2 - 0.5, 0.0)
        rules["frequency"] = torch.where(uniform(n) < 0.5, uniform(n), 0.0)
        lengths = ints(0, longest + 1, n)
        lengths[ints(0, n, 1)] = longest
        ends = lengths.cumsum(0) + 3  # the first starts off any vector's boundary
        begins = ends - lengths
        # few distinct tokens, so that many occur several times; some of no column at all
        pool = torch.cat([ints(0, v, max(1, longest // 3)), torch.tensor(
            [-1, -100, v, v + 5, 2 ** 31 - 1, -2 ** 31], device=device)])
        rules["history"] = pool[ints(0, pool.numel(), int(ends[-1]) + 2)].to(torch.int32)
        rules["history_begin"], rules["history_end"] = begins, ends
        rules["history_split"] = begins + (lengths * uniform(n)).long()
    if kind in ("bias", "all"):
        rules["bias"] = torch.where(uniform(3, v + 3) < 0.3, uniform(3, v + 3) * 8 - 4, 0.0)
        rules["bias_index"] = ints(-2, 5, n).to(torch.int32)  # outside the table: none
    if kind == "all":
        rules["temperature"] = 0.5 + uniform(n)
    tgt = ints(0, v, n).to(torch.int32)
    if kind in ("allow", "all"):
        words = (v + 31) // 32
        rules["allow"] = ints(-2 ** 31, 2 ** 31, 4, words).to(torch.int32)
        index = ints(-1, 5, n).to(torch.int32)
        rules["allow_index"] = index
        # no table bars the targets
        free = torch.zeros(4, words * 32, dtype=torch.bool, device=device)
        held = (index >= 0) & (index < 4)
        free[index[held].long(), tgt[held].long()] = True
        rules["allow"] |= pack(free)
        # what is barred holds anything
        barred = ~allowed(rules, n, v, device)
        x[:, :v] = torch.where(barred & (uniform(n, v) < 0.5), garbage((n, v), gen, device),
                               x[:, :v])
    mask = uniform(n) < 0.8
    tgt[uniform(n) < 0.1] = IGNORE
    g = torch.randn(n, generator=gen, device=device)
    gl = torch.randn(n, generator=gen, device=device) * 0.3
    return Case(x, v, pad, rules, tgt, mask, g, gl)


def pack(bits):
    """bool [R, 32 W] as int32 words [R, W], bit j % 32 of word j / 32."""
    w = bits.view(bits.shape[0], -1, 32).long() << torch.arange(32, device=bits.device)
    w = w.sum(2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def table_rows(rules, name, n):
    """For each row the table's row, or -1."""
    t = rules[name]
    count = 1 if t.dim() == 1 else t.shape[0]
    if name + "_index" in rules:
        at = rules[name + "_index"].long()
        return torch.where((at >= 0) & (at < count), at, -1)
    at = torch.arange(n, device=t.device)
    return at * 0 if count == 1 else at


def allowed(rules, n, v, device):
    out = torch.ones(n, v, dtype=torch.bool, device=device)
    if "allow" not in rules:
        return out
    t = rules["allow"].reshape(-1, rules["allow"].shape[-1])
    at = table_rows(rules, "allow", n)
    for r in range(n):
        if at[r] >= 0:
            bits = (t[at[r]].long()[:, None] >> torch.arange(32, device=device)) & 1
            out[r] = bits.flatten()[:v].bool()
    return out


def processed64(c: Case):
    """(y, slope, error bound of y) in 64 bits, [N, v]; row by row, as the rules say it.

    The bound: x1 is a product with rho or its rounded reciprocal (2 half steps), the penalty
    a product and a sum (2), then two sums and a product with the rounded 1 / T (1, 1 and 2)."""
    n, v, r_ = c.x.shape[0], c.v, c.rules
    x = c.x[:, :v].double()
    on = allowed(r_, n, v, x.device)
    x = torch.where(on, x, 0.0)
    slope, y, err = torch.ones_like(x), x.clone(), torch.zeros_like(x)
    hist = r_.get("history")
    bias_at = table_rows(r_, "bias", n) if "bias" in r_ else None
    for r in range(n):
        rho = float(r_["repetition"][r]) if "repetition" in r_ else 1.0
        ap = float(r_["presence"][r]) if "presence" in r_ else 0.0
        af = float(r_["frequency"][r]) if "frequency" in r_ else 0.0
        if hist is not None:
            b = max(int(r_["history_begin"][r]), 0)
            e = max(min(int(r_["history_end"][r]), hist.numel()), b)
            m = int(r_["history_split"][r]) if "history_split" in r_ else b
            m = min(max(m, b), e)
            tokens, made = hist[b:e].long(), hist[m:e].long()
            tokens, made = (t[(t >= 0) & (t < v)] for t in (tokens, made))
            seen = torch.zeros(v, dtype=torch.bool, device=x.device)
            seen[tokens] = True
            count = torch.bincount(made, minlength=v).double()
            slope[r] = torch.where(seen, torch.where(x[r] > 0, 1.0 / rho, rho), 1.0)
            y[r] = x[r] * slope[r]
            err[r] = torch.where(seen, 2 * H * y[r].abs(), 0.0)
            fine = count * af + ap * (count > 0)
            y[r] -= fine
            err[r] += 2 * H * (count * abs(af) + abs(ap) * (count > 0)) + H * y[r].abs()
        if bias_at is not None and bias_at[r] >= 0:
            y[r] += r_["bias"].reshape(-1, r_["bias"].shape[-1])[bias_at[r], :v].double()
            err[r] += H * y[r].abs()
        if "temperature" in r_:
            t = float(r_["temperature"][r])
            y[r] /= t
            slope[r] /= t
            err[r] = err[r] / t + 2 * H * y[r].abs()
    y = torch.where(on, y, -math.inf)
    slope = torch.where(on, slope, 0.0)
    return y, slope, torch.where(on, err * 1.001, 0.0)


def logp64(c: Case):
    """(logp, lse, p, their error bounds e_logp, e_lse and the relative one of p) in 64 bits.

    A term exp(y - top) is off by y's error, by the rounding of the difference and of its product
    with log2 e (3 half steps of |y - top|) and by the exponential's 2 steps; a piece's sum has
    32 terms a lane and 6 levels of lanes, the merge an exponential and a few roundings."""
    y, slope, err = processed64(c)
    lse = torch.logsumexp(y, 1)
    top = y.amax(1, keepdim=True)
    p = torch.where(y == -math.inf, 0.0, (y - lse[:, None]).exp())
    far = torch.where(p > 0, (y - top).abs(), 0.0)
    e_lse = err.amax(1) + (p * 3 * H * far).sum(1) + 64 * H + H * lse.abs()
    at = torch.where(c.active, c.tgt, 0).long()[:, None]
    of_t = y.gather(1, at)[:, 0]
    logp = torch.where(c.active, of_t - lse, 0.0)
    e_logp = torch.where(c.active, e_lse + err.gather(1, at)[:, 0] + H * logp.abs(), 0.0)
    rel = err + e_lse[:, None] + 3 * H * torch.where(p > 0, (y - lse[:, None]).abs(), 0.0) + 6 * H
    return logp, lse, p, slope, e_logp, e_lse, rel


def gradient64(c: Case, g, gl, half):
    """(dx [N, pad], its error bound) in 64 bits; `half` is half a step of its type."""
    _, _, p, slope, _, _, rel = logp64(c)
    n, v = p.shape
    g = torch.where(c.active, g.double(), 0.0) if g is not None else torch.zeros_like(p[:, 0])
    gl = gl.double() if gl is not None else torch.zeros_like(g)
    coef = (gl - g)[:, None]
    dy = coef * p
    e = coef.abs() * p * (rel + 2 * H)
    rows = torch.arange(n, device=p.device)
    at = torch.where(c.active, c.tgt, 0).long()
    dy[rows, at] += g
    e[rows, at] += H * dy[rows, at].abs()
    d = torch.zeros(n, c.pad, dtype=torch.float64, device=p.device)
    ed = d.clone()
    d[:, :v] = dy * slope
    # the slope is a product of two rounded reciprocals, taken times dy
    ed[:, :v] = (e + 5 * H * dy.abs()) * slope.abs() + half * d[:, :v].abs()
    ed[:, :v] += TINY * (slope > 0)
    return d, ed


def worst(got, want, err):
    """The largest error over its bound; -inf, and elements with a zero bound, have to be equal."""
    got = got.double()
    odd = ~torch.isfinite(want)
    assert torch.equal(got[odd], want[odd]), "infinities differ"
    d = torch.where(odd, 0.0, got - torch.where(odd, 0.0, want)).abs()
    assert torch.isfinite(d).all(), "non-finite values"
    assert (d[err == 0] == 0).all(), "an element that must be exact is not"
    return float((d / err.clamp_min(1e-300)).max()) if d.numel() else 0.0
