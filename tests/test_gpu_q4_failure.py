"""The bounded waits of the 4-bit attention kernel, made to run out on purpose without any fault: the test entry point
holds back every warp's first stage until its wait has given up.  The call must report ZF_DEV_TIMEOUT and
return; the context and the stream stay usable, and the next ordinary call gives what it gave before."""
import pytest
import torch

from tests import helpers as H
from tests.test_gpu_q4 import bits, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    return H.zf_module()


# (group, T): up to 4 columns, 5 to 8, 16, 24, 32 and two passes, with one and several new tokens
@pytest.mark.parametrize("group,T", [(4, 1), (2, 2), (7, 1), (3, 2), (8, 2), (7, 3), (7, 4), (8, 5)])
def test_a_wait_that_runs_out_reports_timeout_and_the_next_call_is_right(zf, group, T):
    lens = [900, 3, 0, 130]
    c, _, table, sl = build(zf, lens, 2, 16, 70)
    args = (bits(torch.randn(4, T, 2 * group, 128, generator=torch.Generator().manual_seed(71))).cuda(), table.cuda(), sl.cuda())
    want = zf.q4_decode_attn(c, *args)
    assert c.status_word() == 0
    for limit in (1000, 200_000):
        zf.q4_decode_attn_wait_test(c, *args, wait_limit_ns=limit)
        got = zf.q4_decode_attn(c, *args)                      # right behind it, on the same stream
        torch.cuda.synchronize()
        assert c.status_word() == zf.DEV_TIMEOUT
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        c.status.zero_()
    # one bad page as a warp's first records: its next wait runs out instead
    bad = table.clone()
    bad[0, :3] = -1
    zf.q4_decode_attn_wait_test(c, args[0], bad.cuda(), args[2], wait_limit_ns=1000)
    assert c.status_word() == zf.DEV_TIMEOUT | zf.DEV_BAD_PAGE_ID
    c.status.zero_()
    got = zf.q4_decode_attn(c, *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and c.status_word() == 0


def test_wait_limits_out_of_range_are_rejected(zf):
    c, _, table, sl = build(zf, [40], 1, 16, 72)
    args = (c, bits(torch.randn(1, 1, 4, 128)).cuda(), table.cuda(), sl.cuda())
    for limit in (0, 999, 2_000_000_001):
        with pytest.raises(zf.ZfError, match="invalid argument"):
            zf.q4_decode_attn_wait_test(*args, wait_limit_ns=limit)
    assert c.status_word() == 0
