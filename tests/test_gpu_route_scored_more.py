"""Routing by scores on the GPU where its documentation allows what the other tests do not do."""

import numpy as np
import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_route_scored import TYPES, check, logits, some_bias

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups", [(3, 256, 1), (70, 16, 2), (70, 60, 5), (70, 128, 1), (70, 192, 12), (70, 256, 8),
                                        (40, 512, 16), (20, 1024, 32)])
def test_closed_experts_are_never_chosen(T, E, groups, score, kind):
    """Closed by a bias of -inf or NaN, by a logit of -inf or (for a token that is not in the sums) a mask, half
    of them and more; experts past the last, in a lane's registers, are closed as well."""
    rng = np.random.default_rng(E + T)
    x = logits(rng, T, E, kind)
    shut = rng.permutation(E)
    x[:, torch.from_numpy(shut[:E // 4]).to(dev())] = -torch.inf
    bias = some_bias(rng, E)
    bias[shut[E // 4:E // 2]] = -np.inf
    bias[shut[E // 2:5 * E // 8]] = np.nan
    mask = rng.random(T) > 0.2
    k = min(8, E // groups)
    for b in (bias, None):
        for opened in {groups, max(1, groups // 2)}:
            got = check(x, k, b, score, groups, opened, min(2, E // groups), mask, True, 2.5)
            never = shut[:E // 4] if b is None else shut[:5 * E // 8]
            assert not np.isin(got["expert_ids"], never).any()
            assert (got["expert_ids"][~mask] == -1).all()
