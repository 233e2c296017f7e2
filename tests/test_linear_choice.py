"""Which kernel of qmoe_linear_fp8 takes which sizes (CPU; the query is pure host code)."""
import os
import re

import pytest

from tests import test_gpu_linear_paths as P

SMS = 152                                            # of a GB300


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_mixture_experts_f32_gb300 as q
    return q


def test_the_tested_sizes_go_where_they_say(q):
    for T, K, N, want in [P.T128, P.T256, P.SHARED, P.FEW] + [p[:4] for p in P.PATHS]:
        assert q.qmoe_debug_linear_choice(SMS, T, K, N) == want, (T, K, N)


def test_every_choice_can_be_launched(q):
    """At any size and on smaller GPUs: a tile that exists, k shared only by tiles of 128, each pair with a group of its own."""
    for sms in (2, 76, 132, SMS, 160):
        for T in (1, 16, 17, 100, 256, 257, 5000, 1 << 20, 1 << 24):
            for K in (16, 128, 144, 512, 528, 2048, 20000, 1 << 20):
                for N in (1, 16, 130, 2048, 151936, 1 << 24):
                    tile, parts = q.qmoe_debug_linear_choice(sms, T, K, N)
                    assert tile in (0, 128, 256) and 1 <= parts <= (4 if tile == 128 else 1)
                    assert parts == 1 or -(-(-(-K // 128)) // 4) >= parts
                    assert tile or -(-T // (8 if T <= 8 else 16 if T <= 32 else 32)) <= 65535
                    if parts > 1:                        # all clusters at once
                        assert -(-T // 256) * -(-N // 128) * parts * 2 <= sms


def test_choice_refusals(q):
    for bad in ((1, 1, 16, 1), (SMS, 0, 16, 1), (SMS, 1, 8, 1), (SMS, 1, 24, 1), (SMS, 1, 16, 0), (SMS, 1, (1 << 20) + 16, 1),
                (SMS, (1 << 24) + 1, 16, 1), (SMS, 1, 16, (1 << 24) + 1)):
        with pytest.raises(q.QmoeError) as e:
            q.qmoe_debug_linear_choice(*bad)
        assert e.value.status == 1
    assert q.lib.qmoe_debug_linear_choice(SMS, 1, 16, 1, None, None) == 1


def test_a_context_sets_up_no_kernels_of_products():
    """There are 36 on pairs of CTAs: each is set up by its first call, not by every qmoe_create."""
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_mixture_experts_f32_gb300", "csrc")
    api = open(os.path.join(csrc, "qmoe_api.cu")).read()
    create = re.search(r"^qmoe_status qmoe_create\(.*?^}", api, flags=re.S | re.M).group(0)
    assert "_prepare(" in create and "linear" not in create
    assert not re.search(r"linear\w*prepare", "".join(open(os.path.join(csrc, f)).read() for f in os.listdir(csrc)))
