"""Child process of the LM-head's split-launch tests: runs its entry points on one seeded
case and saves the output bits.  The library reads RLK_MAX_LAUNCH_THREADS once per process.

    python -m tests.lmhead_child OUT.pt
"""
from __future__ import annotations

import sys

import torch

import vocab_selected_token_amd as rlk
from tests import lmhead_cases as C


def run_all():
    dev = torch.device("cuda")
    c = C.make_case(300, 128, 2900, 3000, 77, dev)
    kw = dict(real_vocab=2900, num_vocab_tiles=7)
    out = {}
    out["logp"], out["lse"] = rlk.fused_lmhead(c.h, c.w, c.tgt, c.mask, **kw)
    out["dh"], out["dw"] = rlk.fused_lmhead_backward(c.h, c.w, c.tgt, c.mask, out["lse"], c.g,
                                                     c.gl, real_vocab=2900)
    _, out["dw0"] = rlk.fused_lmhead_backward(c.h[:0], c.w, c.tgt[:0], None, out["lse"][:0],
                                              c.g[:0], real_vocab=2900)
    torch.cuda.synchronize()
    return {k: v.contiguous().view(torch.uint8).cpu() for k, v in out.items()}


def main(out_path: str) -> int:
    torch.save(run_all(), out_path)
    print("child: done", flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main(sys.argv[1]))
