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
    out["dh20"], out["dw20"] = rlk.fused_lmhead_backward(
        c.h[:20], c.w, c.tgt[:20], c.mask[:20], out["lse"][:20], c.g[:20], real_vocab=2900)
    wq, ws = rlk.quantize_fp8(c.w[:2900], 128)
    out["wq"], out["ws"] = wq, ws
    for n in (300, 20):  # the tile kernel, the streaming one
        h = c.h[:n]
        out[f"hq{n}"], out[f"hs{n}"] = rlk.quantize_fp8(h)
        out[f"logits{n}"] = rlk.lmhead_logits_fp8(h, wq, ws, real_vocab=2900, padded_vocab=3000)
        out[f"logp{n}"], out[f"lse{n}"] = rlk.fused_lmhead_fp8(
            h, wq, ws, c.tgt[:n], c.mask[:n], real_vocab=2900, padded_vocab=3000,
            num_vocab_tiles=7)
    torch.cuda.synchronize()
    return {k: v.reshape(-1).view(torch.uint8).cpu() for k, v in out.items()}


def main(out_path: str) -> int:
    torch.save(run_all(), out_path)
    print("child: done", flush=True)
    return 0


if __name__ == "__main__":
    sys.exit(main(sys.argv[1]))
