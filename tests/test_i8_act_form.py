"""The kernel that a product with an activation and a residual runs on, as
q8v_i8_act_form names it (on the host, without a GPU)."""
import pytest

import moe_expert_ffn_q8_amd as q
from test_gpu_i8_act import SIZES
from test_i8_abi import SHAPE, UNSUP

K_HALVES = 6
form, plain = q.raw.q8v_i8_act_form, q.raw.q8v_i8_form


@pytest.mark.parametrize("m,k,n", [(300, 1024, 4100), (300, 1056, 4100), (130, 2080, 6000), (97, 1312, 8200),
                                   (512, 4128, 3001), (320, 14336, 4096), (65, 1024, 16384), (700, 2048, 2000)])
def test_few_outputs_and_a_long_k(m, k, n):
    assert form(n, k, m) == K_HALVES and plain(n, k, m, 0) == 2


def test_others_are_those_of_the_plain_product():
    """A shorter k, more outputs, fewer tokens, larger tiles."""
    for m, k, n in SIZES + [(300, 992, 4100), (129, 1024, 16384), (64, 2048, 4096), (2048, 2048, 8192), (97, 1312, 8192)]:
        assert form(n, k, m) == plain(n, k, m, 0) != K_HALVES, (m, k, n)


def test_every_kernel_has_a_tested_size():
    from test_gpu_i8_act_forms import SIZES as more
    assert {form(n, k, m) for m, k, n in SIZES + more} >= {0, 1, 2, 3, 4, K_HALVES}


def test_refused_sizes():
    assert form(8, 33, 4) == SHAPE and form(0, 64, 4) == SHAPE and form(8, 64, 0) == SHAPE
    assert form(8, 1 << 17, 4) == UNSUP and form((1 << 27) + 1, 64, 4) == UNSUP
