"""Pins of the FP64 attention oracle: closed forms, and torch's softmax under a mask built another way."""
import math

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 0), (3, 2), (4, 9), (100, 1)])
def test_matches_a_masked_softmax(window, sinks):
    g = torch.Generator().manual_seed(window + sinks)
    q, k, v = (torch.randn(n, 8, generator=g, dtype=torch.float64) for n in (6, 11, 11))
    pos = np.array([-2, 0, 3, 7, 9, 10])
    o, lse, spread = oracle.attention(q, k, v, pos, 0.3, window, sinks)
    for i, p in enumerate(pos):
        seen = [j for j in range(11) if j <= p and (not window or p - j < window or j < sinks)]
        if not seen:
            assert lse[i] == -np.inf and not o[i].any() and not spread[i].any()
            continue
        x = 0.3 * (q[i] * k[seen]).sum(1)
        a = torch.softmax(x, 0)
        assert abs(lse[i] - float(torch.logsumexp(x, 0))) < 1e-12
        assert np.allclose(o[i], (a[:, None] * v[seen]).sum(0), atol=1e-12)
        assert np.allclose(spread[i], (a[:, None] * v[seen].abs()).sum(0), atol=1e-12)


def test_equal_keys_average_the_visible_values():
    k, v = np.ones((7, 4)), np.arange(28.0).reshape(7, 4)
    o, lse, _ = oracle.attention(np.full((1, 4), 2.0), k, v, [6], 0.5, window=2, sinks=1)
    assert np.allclose(o[0], v[[0, 5, 6]].mean(0)) and math.isclose(lse[0], 4.0 + math.log(3))
