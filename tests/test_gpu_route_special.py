"""Softmax routing of rows with NaN, infinite and far-apart logits: the same stated order at every number of
experts (the register body and the plain one above 1024) and with every way of choosing, ids compared exactly
with a plain 64-bit form. Scores lie at least 2^-16 of themselves apart, or are equal; the last row's differ
by more than 32 bits can hold, where no sum of scores is asked for."""
import numpy as np
import pytest

import block_reference as ref
from test_gpu_route_grouped import run

pytestmark = pytest.mark.gpu


def rows(E):
    rng = np.random.default_rng(E)
    x = np.stack([rng.permutation(np.linspace(-8, 8, E)) for _ in range(8)])
    x[0, :] = -np.inf
    x[0, :10] = np.nan
    x[0, [20, 30, E - 1]] = [1.0, 2.0, -3.0]       # few experts, NaN at lower indices than the masked ones
    x[1, E - 3] = np.inf                           # scores of 0 beside one of 1
    x[2, :2], x[2, 2], x[2, [3, 50]] = np.nan, -np.inf, np.inf
    x[3], x[3, E - 1] = np.nan, -np.inf
    x[4], x[4, 0] = -np.inf, np.nan
    x[5, :3] = [0.0, 5.0, np.inf]
    x[6], x[6, [7, 9]] = -0.0, 0.0                 # equal, whatever their sign
    x[7] = -np.inf
    x[7, rng.choice(E, 32, replace=False)] = -10.0 * np.arange(32)  # scores down to 1e-134
    return x.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("K", [1, 8, 20])
@pytest.mark.parametrize("E,groups,kept", [(64, 4, 2), (66, 6, 3), (320, 8, 4), (896, 1, 1), (1000, 8, 5), (1100, 4, 2), (4096, 64, 8)])
def test_softmax_special_rows(moe, E, groups, kept, K):
    x = rows(E)
    for g, k, rule in ((1, 1, "max"), (groups, kept, "max"), (groups, kept, "top2")):
        ids, w = run(moe, x, None, K, scoring="softmax", groups=g, kept=k, rule=rule, scale=2.0)
        for t in range(x.shape[0] - (rule == "top2" and g > 1)):
            eid, ew = ref.route(x[t], None, K, "softmax", g, k, rule, True, 2.0)
            np.testing.assert_array_equal(ids[t], eid, err_msg=f"groups {g} {rule}, row {t}")
            assert np.all(np.abs(w[t] - ew) <= 1e-5 * np.abs(ew) + 1e-30)
