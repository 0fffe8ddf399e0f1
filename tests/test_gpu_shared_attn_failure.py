"""The bounded waits of the shared-prefix attention's tcgen05 kernel, run out one by one from the host
(a barrier that wants one arrival more than come): the call returns, sets TIMEOUT, and the next one is
bit for bit right."""
import pytest
import torch

from pe_helpers import pk
from test_gpu_shared_attn import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wait", range(6))
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("shape", ["pairs", "long", "many"])
def test_a_wait_that_runs_out(shape, hd, wait):
    m = pk()
    if wait == 5 and hd == 128:
        pytest.skip("scores are read before their weights are stored over them: no wait of its own")
    if shape == "pairs":
        c = Call("bf16", 9, 8, 16, 2, hd, 100000, [10 * i for i in range(9)])
    elif shape == "long":
        c = Call("bf16", 2, 1, 4, 1, hd, 200000, [10, 3])
    else:
        c = Call("bf16", 200, 2, 16, 8, hd, 500, [i * 7 % 900 for i in range(200)])
    want, wlse = c.run()
    assert c.errors.item() == 0
    try:
        m.peagle_set_wait_limit_shared(1000000, wait)
        c.run()
        torch.cuda.synchronize()
        assert c.errors.item() == m.PEAGLE_DEV_TIMEOUT
    finally:
        m.peagle_set_wait_limit_shared(0, -1)
    c.errors.zero_()
    got, lse = c.run()
    assert c.errors.item() == 0 and torch.equal(got, want) and torch.equal(lse, wlse)
