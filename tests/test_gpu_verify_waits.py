"""csa_verify_drafts: waits that run out."""
import numpy as np
import pytest

from test_gpu_verify_drafts import call, make

pytestmark = pytest.mark.gpu


def test_waits_that_expire_are_reported(cuda_lib):
    """A limit of one nanosecond, shorter than any exchange between CTAs: the calls end with the status, what they
    leave is in range, and the next call is right."""
    csd = cuda_lib
    x = make(20, 5, 40000, "chain", "bf16", "bf16", seed=12)
    want = call(csd, x)
    csd.csa_debug_set_wait_limit_ns(1)
    try:
        path, accepted, nxt = call(csd, x)
    finally:
        csd.csa_debug_set_wait_limit_ns(0)
    assert csd.csa_read_device_error() == csd.ERR_TIMEOUT
    gave_up = nxt == -1
    assert gave_up.any() and np.all((accepted >= 1) & (accepted <= 5)) and np.all((nxt >= -1) & (nxt < 40000))
    for b in range(20):
        n = int(accepted[b])
        assert path[b, 0] == 0 and np.all(path[b, n:] == -1)
        assert np.array_equal(path[b, :n], want[0][b, :n])  # (a walk that ended early is the right one's beginning)
        if not gave_up[b]:
            assert n == want[1][b] and nxt[b] == want[2][b]
    assert all(np.array_equal(a, b) for a, b in zip(call(csd, x), want))
    assert csd.csa_read_device_error() == 0
