"""Scored routing where its fast choice works at its limits, against the rule in
64 bits: NaN keys at every place of a lane."""
import itertools

import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.test_gpu_route_scored import check


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


# one group taken, of `gs` experts over two lanes or more of every shape but the widest
@pytest.mark.gpu
@pytest.mark.parametrize("gs,G", [(5, 1), (8, 1), (16, 1), (17, 1), (17, 8), (17, 16), (17, 32), (17, 60)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_two_nan_keys_rank_by_id(m, gs, G, score):
    """Two NaN logits among the taken group's experts and room for one of them: the lower id."""
    need_gpu()
    pairs = list(itertools.combinations(range(gs), 2))
    rng = np.random.default_rng(gs * G)
    E, T = gs * G, len(pairs)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    taken = G // 2 * gs
    logits[:, taken:taken + gs] += 8.0
    for t, (i, j) in enumerate(pairs):
        logits[t, [taken + i, taken + j]] = np.nan
    for rows in (logits, logits[:min(T, 60)], logits[-1:]):
        check(m, rows, gs - 1, score=score, n_group=G, topk_group=1, group_rank="max")
        check(m, rows, gs - 1, score=score, n_group=G, topk_group=1, group_rank="max",
              bias=np.zeros(E, np.float32))
