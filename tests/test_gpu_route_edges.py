"""Scored routing where its fast choice works at its limits, against the rule in
64 bits: NaN keys at every place of a lane, groups whose two best keys cancel,
and weights of experts at -inf beside tiny ones."""
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


@pytest.mark.gpu
@pytest.mark.parametrize("big", [100.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(16, 8), (64, 8), (128, 4)])
def test_groups_whose_best_keys_cancel(m, E, G, score, big):
    """A forced expert (bias +big) and none but banned ones (-big) beside it in every group: a group's rank is
    the small difference of two large keys, and decides between groups whose scores are close."""
    need_gpu()
    T, gs = 1500, E // G
    rng = np.random.default_rng(int(big) + E)
    logits = (rng.standard_normal((T, 1)) + rng.standard_normal((T, E)) * (20.0 / big)).astype(np.float32)
    bias = np.full(E, -big, np.float32)
    bias[rng.integers(0, gs, G) + gs * np.arange(G)] = big
    check(m, logits, 2, score=score, n_group=G, topk_group=2, group_rank="top2", bias=bias)
    check(m, logits[:40], 2, score=score, n_group=G, topk_group=G - 1, group_rank="top2", bias=bias)


@pytest.mark.gpu
@pytest.mark.parametrize("gap", [0.0, 300.0, 700.0])
@pytest.mark.parametrize("E", [3, 40, 300])
def test_infinitely_low_logits_weigh_nothing(m, E, gap):
    """The largest logit kept out by its bias, one `gap` below it taken together with logits of -inf: their weight is
    0, however small the sum that divides them."""
    need_gpu()
    logits = np.full((70, E), -np.inf, np.float32)
    logits[:, 0] = 800.0
    logits[:, 1] = 800.0 - gap
    bias = np.zeros(E, np.float32)
    bias[0] = -np.inf
    for rows in (logits, logits[:1]):
        check(m, rows, 2, score="softmax", bias=bias)
        check(m, rows, 2, score="softmax", bias=bias, renormalize=False)
