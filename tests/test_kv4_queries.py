"""GPU test of what the 4-bit cache's attention of many rows holds of bf16 queries:
they become fp16 times a power of two for each row, which by the contract
(include/qsa.h) keeps all bits of elements down to 2^-24 of the row's largest."""
import numpy as np
import pytest

import kv4_cases as kc
from test_kv4_parity import tbs  # noqa: F401
from test_kv4_precision import check_norm, one_head

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("large", [1.0, 1.75, 1.9921875])
@pytest.mark.parametrize("D", [64, 128])
def test_elements_far_below_the_largest(tbs, D, large):  # noqa: F811
    """One dimension of the queries, where the keys are zero, 2^23 to 2^24 times the others."""
    rng = np.random.default_rng(D)
    k, v = rng.standard_normal((1500, D)) * 2, rng.standard_normal((1500, D)) * 2
    k[:, 3] = 0.0
    c = one_head(1, k, v, np.full(1500, 0.5), 2.0 ** rng.uniform(-6, -5, 1500), 64)
    q = rng.uniform(1, 2, (1, 128, 16, D)) * rng.choice([-1.0, 1.0], (1, 128, 16, D)) * large
    q[..., 3] = 2.0 ** 24 * large
    check_norm(tbs, c, kc.ROUND["bf16"](q), "bf16", D ** -0.5 / large, "kv4_attend_many_kernel")
