"""The paged operators at the edges of what their documentation allows: stops, overflowing steps,
counts updated in place by many CTAs, widely spread scales, long sums of small weights."""
import math
import time

import numpy as np
import pytest
import torch

from paged_helpers import BF16_ROWS
from test_gpu_paged import Pool, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__
    __graft_entry__.build()
    import compressed_decode_attention_kvk_b200 as p
    assert torch.cuda.is_available()
    return p


@pytest.mark.parametrize("b,G,d", [(8, 0, 512), (16, 0, 512), (BF16_ROWS, 0, 512), (4, 32, 128),
                                   (8, 0, 128), (BF16_ROWS, 0, 192)])
def test_a_stop_at_any_moment_ends_soon(pkg, oracle_mod, b, G, d):
    """Wait limits that run out at different steps of the expanded-rows kernel: the two CTAs of a
    pair stop at different loads, the call ends without waiting for loads that never come (well
    under the two seconds that the kernel grants its own loads), and the next call is right."""
    q_lens, H = [40, 30], 40
    pool = Pool(pkg, oracle_mod, [1500, 700], d, 64, b, G, 64, 3)
    lay = pool.lay
    try:
        sigma = 1 / math.sqrt(d + 64)
        ql, qr = pool.queries(q_lens, H, torch.bfloat16, 1)
        _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, sigma, torch.bfloat16)
        stops = 0
        for limit in (1, 100, 300, 600, 1000, 1500, 2500, 4000, 8000, 16000):
            for _ in range(3):
                lay.set_wait_limit(limit)
                torch.cuda.synchronize()
                t0 = time.perf_counter()
                _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, sigma, torch.bfloat16)
                took = time.perf_counter() - t0
                status = lay.read_status(clear=True)
                assert status in (0, pkg.kvk.KVK_FLAG_TIMEOUT), limit
                stops += status != 0
                assert took < 1.0, f"limit {limit} ns: {took:.2f} s"
        assert stops >= 3
        lay.set_wait_limit(0)
        out, lse = _run(pool, pkg, pkg.KVK_PATH_TENSOR, q_lens, ql, qr, sigma, torch.bfloat16)
        pool.check(q_lens, ql, qr, out, lse, torch.bfloat16, sigma, True)
        assert lay.read_status() == 0
    finally:
        lay.close()
