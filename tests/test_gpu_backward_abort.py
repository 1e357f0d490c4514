"""GPU tests of a backward pass whose waits give up (the first commit is withheld): zeros in the
rows that were asked for, nothing anywhere else, and the next call is as if nothing had been."""
import pytest
import torch

import oracle
import pose_retrieved_kv_b200 as P
from tests._gpu import need_gpu
from tests.test_gpu_backward import backward, case, forward, inputs

pytestmark = pytest.mark.gpu
GUARD = 1 << 16                                      # elements on both sides of a gradient


@pytest.mark.parametrize("kw", [dict(head_dim=128), dict(n_heads=5), dict(head_dim=128, grid_h=9, grid_w=11),
                                dict(valid_mask=0b001001, block_index=0, head_dim=128)])
@pytest.mark.parametrize("mask", [0xFF, 0b101000])
@pytest.mark.parametrize("limit_ns", [10_000, 60_000])
def test_a_pass_that_gives_up_writes_no_row_that_is_not_its_own(kw, mask, limit_ns):
    need_gpu()
    cfg = case("grid", **kw)
    q, k, v, do = inputs(cfg, 81)
    out, lse = forward(cfg, q, k, v)
    want = backward(cfg, q, k, v, do, out, lse)
    lay = P.make_layout(**cfg)
    scratch = torch.full((P.prsink_attention_backward_scratch_bytes(lay),), 255,
                         dtype=torch.uint8, device="cuda")
    dev = [x.cuda() for x in (q, k, v, out, lse, do)]
    room = [torch.full((2 * GUARD + x.numel(),), 7.0, dtype=torch.bfloat16, device="cuda")
            for x in want]
    grads = [r[GUARD:-GUARD].view(x.shape) for r, x in zip(room, want)]
    assert P.prsink_sync_status() == P.PRSINK_OK
    P.prsink_debug_attention_stall(limit_ns)
    P.prsink_attention_backward(lay, *dev, *grads, scratch, grad_mask=mask)
    assert P.prsink_sync_status() == P.PRSINK_ERR_TIMEOUT
    for r in room:
        assert torch.all(r[:GUARD] == 7.0) and torch.all(r[-GUARD:] == 7.0)
    assert not grads[0].any()
    for s, (a, e) in enumerate(oracle.slot_ranges(cfg)):
        for g in grads[1:]:
            assert torch.all(g[:, a:e] == (0.0 if (mask >> s) & 1 else 7.0)), s
    again = backward(cfg, q, k, v, do, out, lse)
    assert P.prsink_sync_status() == P.PRSINK_OK
    assert all(torch.equal(a, b) for a, b in zip(want, again))
