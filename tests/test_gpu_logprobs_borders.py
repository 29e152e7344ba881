"""Ranks and alternatives beside the borders of a cut row's pieces.

A row's memory is read in groups of 8 logits on 16-byte boundaries, while its
pieces end at multiples of 8 logits: in a row that starts off such a boundary
a group lies in two pieces.  Equal logits of lower ids, on either side of the
border, stand in front of a given token of that group.  Rank and order are
whole numbers and have to be those of the definition; tolerances of the rest as
in test_gpu_logprobs."""
import math

import pytest

from tests.gpu_util import need_gpu, torch
from tests.test_gpu_logprobs import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def borders(m, T, V):
    """Where the pieces of each of T rows of V logits start and end, from the workspace the call asks for: with k = 0
    48 bytes a piece or less, with k = 1 8 more a piece."""
    n = [m.moe_logprobs_workspace_size(m.logprob_args(logits=0x10000, T=T, V=V, entropy=0x20000, k=k,
                                                      top_ids=0x30000 if k else None)) for k in (0, 1)]
    splits = (n[1] - n[0]) // (8 * T)
    assert splits > 1
    piece = ((V + splits - 1) // splits + 7) // 8 * 8
    return [b for b in range(piece, V, piece)]


def around(m, T, V):
    """T ids, as many as there are from 9 in front of a border to 9 behind it."""
    ids = sorted({i for b in borders(m, T, V) for i in range(b - 9, b + 10) if 0 <= i < V} | {0, V - 1})
    return torch.tensor([ids[t * len(ids) // T] if T < len(ids) else ids[t % len(ids)] for t in range(T)], dtype=torch.int32)


KINDS = {
    "equal": lambda T, V, g: torch.full((T, V), 1.5),
    "few": lambda T, V, g: torch.randint(-2, 3, (T, V), generator=g).float(),
    "least": lambda T, V, g: torch.where(torch.rand(T, V, generator=g) < 0.01, 1.0, -math.inf),
}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("T,V", [(98, 10001), (16, 131069)])
def test_ranks_beside_borders(m, T, V, shift, kind):
    """Every place of a border in a group: all rows `shift` logits off a 16-byte boundary (row strides of whole groups)."""
    need_gpu()
    l = KINDS[kind](T, V, torch.Generator().manual_seed(V + shift))
    ids = around(m, T, V)
    for dtype in (torch.bfloat16, torch.float32):
        if dtype == torch.bfloat16 or shift < 4:
            run(m, l.to(dtype), 1.0, ids, k=shift % 3, pad=-V % 8, shift=shift)


@pytest.mark.parametrize("pad", [0, 1, 2, 3])
def test_ranks_of_rows_that_start_anywhere(m, pad):
    """Odd row strides: each row starts at another place of a group."""
    need_gpu()
    T, V = 98, 12345
    g = torch.Generator().manual_seed(pad)
    for kind in ("equal", "few"):
        l = KINDS[kind](T, V, g)
        run(m, l.to(torch.bfloat16), 1.0, around(m, T, V), k=20, pad=pad, shift=pad)
        run(m, l, 0.5, around(m, T, V), k=0, pad=pad)
