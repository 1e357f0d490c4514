"""GPU tests of the backward pass with several heads per preparing CTA (the preparation computes
a row's angles once for a group of heads), the last group short; bounds as in
``tests/test_gpu_backward.py``."""
import pytest

import oracle
import pose_retrieved_kv_b200 as P
from tests._gpu import need_gpu
from tests.test_gpu_backward import backward, case, check, forward, inputs

pytestmark = pytest.mark.gpu


def prep_heads(cfg, n_sm=148):
    """Heads per CTA as the launch chooses them: as many as leave eight CTAs per SM."""
    s = oracle.layout_sizes(cfg)
    rows = 256 // (cfg["head_dim"] // 8)
    row_ctas = -(-s["T"] // rows) + -(-s["L_blk"] // 128) * 128 // rows
    most = row_ctas * cfg["n_heads"] // (8 * n_sm)
    groups = cfg["n_heads"] if most < 1 else -(-cfg["n_heads"] // most)
    return -(-cfg["n_heads"] // groups)


GROUPED = [(case("grid", n_heads=53, grid_h=12, grid_w=12), 3),
           (case("grid", n_heads=11, head_dim=128, grid_h=16, grid_w=16), 2)]


@pytest.mark.parametrize("cfg,heads", GROUPED)
@pytest.mark.parametrize("mask", [0xFF, 0b011011])
def test_several_heads_per_preparing_cta(cfg, heads, mask):
    need_gpu()
    assert prep_heads(cfg) == heads and cfg["n_heads"] % heads
    cfg = dict(cfg, valid_mask=mask, block_index=7 if mask == 0xFF else 1)
    q, k, v, do = inputs(cfg, 71)
    out, lse = forward(cfg, q, k, v)
    got = backward(cfg, q, k, v, do, out, lse)
    assert P.prsink_sync_status() == P.PRSINK_OK
    check(cfg, got, q, k, v, do)
