"""Cache operators on batches of unlike requests, and where CTAs of a cluster
exchange results block after block.  References and tolerances are those of
test_gpu_cache_ops."""
import numpy as np
import pytest

from test_gpu_cache_ops import _pool, _randn, _starts, _weights_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q,prefix", [([300, 200], [3000, 20]), ([64, 700, 1], [0, 1500, 9])])
def test_key_weights_of_many_row_blocks_in_a_cluster(q, prefix):
    """Three and more blocks of 128 query rows, a unit's tiles over a cluster of
    eight CTAs, most of which have no tile of the short request: the CTAs
    exchange their rows' sums block after block, hardly apart in time."""
    import torch
    _weights_case(1, 1, 4, 128, "bf16", prefix=prefix, q=q)
    pool, n = _pool(1, 1, 4, 128, "bf16"), len(q)
    co, qo = _starts([a + b for a, b in zip(prefix, q)]), _starts(q).astype(np.int32)
    ck, Q = _randn(1, (int(co[-1]), 128), "bf16"), _randn(2, (1, int(qo[-1]), 4, 128), "bf16")
    w = [torch.zeros(int(co[-1]), device="cuda") for _ in range(2)]
    pool.key_weights(co, prefix, qo, Q, ck, w[0])
    for _ in range(40):
        pool.key_weights(co, prefix, qo, Q, ck, w[1])
        assert torch.equal(w[0], w[1])
    # every query row's probabilities sum to one
    for b in range(n):
        got = float(w[0][int(co[b]):int(co[b + 1])].double().sum())
        assert abs(got - 4 * q[b]) <= 4 * q[b] * 2.0 ** -16
