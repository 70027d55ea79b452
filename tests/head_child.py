"""Child process of the split-launch test of the logit rules and the dense products: runs them on
one seeded case and saves the output bits to the path it is given.  The library reads
RLK_MAX_LAUNCH_THREADS once per process.

    python -m tests.head_child OUT.pt [halves]
"""
from __future__ import annotations

import sys

import torch

import vocab_selected_token_amd as rlk
from tests import linear_cases as L
from tests import process_cases as P

DEV = torch.device("cuda")


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).cpu()


def run_all():
    out = {}
    for n, v, pad in ((70, 17000, 17003), (900, 150001, 150016)):  # one span a block, and four
        c = P.make_case(n, v, pad, n, DEV, "all")
        r = rlk.LogitRules(**c.rules)
        kw = dict(real_vocab=v, padded_vocab=pad)
        y = rlk.process_logits(c.x, r, **kw)
        logp, lse = rlk.processed_forward(c.x, c.tgt, r, c.mask, **kw)
        d = rlk.processed_backward(c.x, c.tgt, r, c.mask, lse, c.g, c.gl,
                                   out_dtype=torch.bfloat16, **kw)
        # (the large one's rows by their sums of bits)
        whole = (y, logp, lse, d) if n < 100 else \
            (bits(y).sum(1).to(torch.int32), logp, lse, bits(d).sum(1).to(torch.int32))
        out[f"rules_{n}"] = tuple(bits(t) for t in whole)
    for m, k, n in ((3, 640, 5000), (40, 192, 30000), (17, 128, 9000), (150, 192, 700),
                    (700, 64, 3000)):
        c = L.make_case(m, k, n, "silu", m, DEV)
        y, saved = rlk.linear_forward(c.x, c.w, c.bias, c.residual, activation="silu", save=True)
        out[f"linear_{m}"] = tuple(bits(t) for t in (y, *rlk.linear_backward(
            c.x, c.w, c.dy, saved, activation="silu", want_bias=True)))
    torch.cuda.synchronize()
    return out


def run_halves():
    """A product whose last 40 of 1320 tiles go in halves; sums of its rows' bits."""
    c = L.make_case(1000, 64, 84480, "silu", 5, DEV)
    y, _ = rlk.linear_forward(c.x, c.w, c.bias, c.residual, activation="silu")
    torch.cuda.synchronize()
    return {"halves": (bits(y).sum(1).to(torch.int32),)}


if __name__ == "__main__":
    print("head child: running", flush=True)
    torch.save(run_halves() if sys.argv[2:] == ["halves"] else run_all(), sys.argv[1])
    print("head child: done", flush=True)
