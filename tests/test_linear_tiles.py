"""Each size of tile of the dense products against exact results, forward and backward.

Which tile a call takes follows from its sizes and the costs in the source (best_tile); a model of
that rule says here, without a GPU, which tile each shape below reaches, so that another choice of
tiles cannot leave one untested."""
from __future__ import annotations

import re

import pytest

import vocab_selected_token_amd.build_lib as build_lib
from tests import test_gpu_linear as G

SOURCE = (build_lib.CSRC / "rlk_linear.hip").read_text()
TABLE = re.search(r"kTileCosts\[\] = \{(.*?)\};", SOURCE, re.S).group(1)
COSTS = [(int(a), int(b), int(fit), [float(t) for t in time.split(",")])
         for a, b, fit, time in re.findall(r"\{(\d+), (\d+), (\d+), \{([^}]*)\}\}", TABLE)]


def tiles(x, y, a, b):
    return -(-x // a) * -(-y // b)


def best(blocks):
    costs = []
    for a, b, fit, time in COSTS:
        full, rest = divmod(blocks(a, b), 256 * fit)
        costs.append(full * time[fit - 1] + (time[(rest - 1) // 256] if rest else 0.0))
    return costs.index(min(costs))


def forward_tile(m, k, n):
    return best(lambda a, b: tiles(n, m, a, b))


def backward_tile(m, k, n, want_x=True, want_weight=True):
    return best(lambda a, b: (tiles(k, m, a, b) if want_x else 0)
                + (tiles(k, n, a, b) if want_weight else 0))


# tokens, in, out, and the tiles of the forward, of the gradients together, of dx's alone and of
# dW's alone; rows and columns of every tile are left over (in is a multiple of 64, not of 128)
SHAPES = {(1030, 192, 13001): (0, 3, 3, 3), (1030, 2112, 4101): (2, 0, 3, 0),
          (4101, 2112, 1030): (2, 0, 0, 3), (1101, 1472, 3001): (1, 1, 3, 2),
          (1501, 1088, 1499): (3, 1, 3, 3), (701, 2112, 1501): (3, 2, 3, 1),
          (1501, 2112, 701): (3, 2, 1, 3), (3001, 1472, 1101): (1, 1, 2, 3)}


def test_every_tile_is_reached():
    assert [(a, b) for a, b, *_ in COSTS] == [(256, 256), (128, 128), (128, 64), (64, 64)]
    for s, want in SHAPES.items():
        got = (forward_tile(*s), backward_tile(*s), backward_tile(*s, want_weight=False),
               backward_tile(*s, want_x=False))
        assert got == want, (s, got)
    for of in zip(*SHAPES.values()):
        assert set(of) == {0, 1, 2, 3}
    # the order in which the launchers take them
    for launch in ("launch_tiles", "launch_grads"):
        taken = re.findall(launch + r"<(\d), (\d), (\d)>\(a, stream\)", SOURCE)
        assert taken == [("8", "4", "4"), ("4", "4", "2"), ("4", "2", "2"), ("2", "2", "2")]


@pytest.mark.gpu
@pytest.mark.parametrize("m, k, n", SHAPES)
def test_whole_numbers(m, k, n):
    G.test_whole_numbers_are_exact(m, k, n)


@pytest.mark.gpu
@pytest.mark.parametrize("m, k, n", SHAPES)
def test_an_activation(m, k, n):
    """Both dtypes of the bias (and of what is kept of z), with and without a residual; dx, dW and db
    alone, whose tiles are others, have the bits that they have together."""
    G.test_forward(m, k, n, "silu")
    for bias in (G.BF16, None):
        G.backward_case(m, k, n, "silu", bias or G.torch.float32)
