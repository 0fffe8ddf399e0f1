"""Failure detection of the tcgen05 attention over the 8-bit cache without a GPU fault.

peagle_set_wait_limit_quant shortens the bound of the kernel's waits to 1 ms and gives one kind of
barrier an arrival more than come, so the waits on it run out: the kernel must set
PEAGLE_DEV_TIMEOUT, leave in every role, let its copies and tensor operations finish, free its
tensor memory and return.  The next call, with the default bound, must match the fp64 oracle.
Every wait that runs out is an ordinary bounded spin."""
import time

import pytest
import torch

from pe_helpers import pk
from test_gpu_kv_quant import Cache, attend, check_result, ints, queries

pytestmark = pytest.mark.gpu

# a few long heads in pieces, and more heads than SMs (both have CTAs of more than one head and of
# more tiles than the ring of copied codes holds)
CASES = [(64, 16, 4, [98000, 60000], 98304), (128, 8, 5, [98000, 60000], 98304),
         (64, 16, 8, [300 + 7 * (i % 100) for i in range(300)], 1024),
         (128, 16, 8, [300 + 7 * (i % 100) for i in range(300)], 1024)]


@pytest.fixture(scope="module", params=range(len(CASES)))
def case(request):
    hd, G, K, lens, cap = CASES[request.param]
    c = Cache(1, len(lens), 1, cap, hd, 32, 3, spread=2)
    q = queries(len(lens), K, G, hd, "bf16", 4)
    m = pk()
    work = torch.zeros(m.peagle_decode_attention_quant_workspace(c.kv, len(lens), K, G),
                       dtype=torch.uint8, device="cuda")
    want, wl = attend(c, 0, q, lens, K, work=work)
    assert c.err() == 0
    if cap == 1024:
        check_result(c, 0, q, lens, K, True, 0, None, want, wl)
    return c, q, lens, K, work, want, wl


@pytest.mark.parametrize("wait", range(9))
def test_a_wait_that_cannot_end_times_out_and_the_next_call_is_right(case, wait):
    m = pk()
    c, q, lens, K, work, want, wl = case
    sl, out = ints(lens), torch.empty_like(want)
    torch.cuda.synchronize()
    m.peagle_set_wait_limit_quant(1_000_000, wait)
    try:
        t0 = time.perf_counter()
        m.peagle_decode_attention_quant(c.kv, 0, len(lens), K, q.shape[1], q, sl, out, work)
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        m.peagle_set_wait_limit_quant(0, -1)
    assert c.err() == m.PEAGLE_DEV_TIMEOUT
    assert dt < 1.5, f"the drilled call took {dt:.2f} s"
    got, lse = attend(c, 0, q, lens, K, work=work)
    assert c.err() == 0 and torch.equal(got, want) and torch.equal(lse, wl)


def test_a_short_limit_alone_changes_nothing(case):
    """1 ms is far more than any wait of these calls takes."""
    m = pk()
    c, q, lens, K, work, want, wl = case
    m.peagle_set_wait_limit_quant(1_000_000, -1)
    try:
        got, lse = attend(c, 0, q, lens, K, work=work)
        torch.cuda.synchronize()
    finally:
        m.peagle_set_wait_limit_quant(0, -1)
    assert c.err() == 0 and torch.equal(got, want) and torch.equal(lse, wl)
