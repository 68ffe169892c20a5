"""Item ids and decay attention where a caller can go wrong, as far as it needs no GPU."""
import numpy as np
import pytest

import shared_prefix_behavior_b200 as R
from tests.conftest import gpu_available
from tests.test_history_boundary import NO_DEVICE, WORKSPACE, _pass


def test_decay_heads_keep_the_arrays_that_the_calls_read():
    heads = R.DecayHeads((0, 64), (-0.1, -0.2), 16)
    at = heads.decay
    for name in ("taus", "log_decay"):
        with pytest.raises(AttributeError):
            setattr(heads, name, np.zeros(2))
    heads.log_decay[0] = -0.5
    heads.taus[1] = 0
    assert heads.decay == at == heads.log_decay.ctypes.data and not heads.timed


BATCHES = [[4096], [16384] * 2, [4096] * 8, [4096] * 16, [4096] * 64, [64], [0], [1, 0, 200], [300] * 200,
           [100 * (i % 37) for i in range(150)], [5] * 1000]


def _cu(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


# the calls have addresses of no memory: with a GPU they would be launched
@pytest.mark.skipif(gpu_available(), reason="needs a machine without a GPU")
@pytest.mark.parametrize("dt", [R.REST_BF16, R.REST_F32])
@pytest.mark.parametrize("taus,hd", [((0,) * 8, 64), ((0, 64), 16)])
def test_a_workspace_for_one_batch_serves_every_batch_of_no_more_users(dt, taus, hd):
    decay = (-0.1,) * len(taus)
    heads = R.DecayHeads(taus, decay, hd)
    size = {i: R.decay_attn_workspace_size(dt, heads, _cu(b)) for i, b in enumerate(BATCHES)}
    for i, big in enumerate(BATCHES):
        for small in BATCHES:
            if len(small) > len(big) or sum(small) == 0:
                continue
            for back in (False, True):
                got = _pass(back, dt=dt, taus=taus, hd=hd, decay=decay, cu=_cu(small), ws_bytes=size[i])
                assert got == NO_DEVICE, (big[:3], small[:3], back)


@pytest.mark.skipif(gpu_available(), reason="needs a machine without a GPU")
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("lengths", [b for b in BATCHES if sum(b)])
def test_the_smallest_workspace(lengths, back):
    """Below what the users' items take the call is refused, from there on it is not."""
    n, taus = len(lengths), (0, 64)
    item, user = 56, 24                              # bytes of what the kernels read of each
    least = (n * item + 255) // 256 * 256 + (n * user + 255) // 256 * 256
    kw = dict(taus=taus, hd=32, decay=(-0.1, -0.1), cu=_cu(lengths))
    assert _pass(back, ws_bytes=least, **kw) == NO_DEVICE
    assert _pass(back, ws_bytes=least - 256, **kw) == WORKSPACE
    heads = R.DecayHeads(taus, (-0.1, -0.1), 32)
    assert R.decay_attn_workspace_size(R.REST_BF16, heads, _cu(lengths)) >= least


def test_the_step_self_test_refuses_its_limits():
    import ctypes
    from tests.test_history_boundary import FAKE, INVALID, _heads, _state
    t, hs = _heads((0, 64), 16)
    g = np.asarray((-0.1, 0.0))
    st = _state()

    def call(limit=2_000_000, err=FAKE):
        return R.library().rest_selftest_decay_step_timeout(R.REST_F32, ctypes.byref(hs), g.ctypes.data, 0, None, None, None,
                                                            FAKE, ctypes.byref(st), FAKE, None, limit, err, None)
    assert call(limit=10) == call(limit=5_000_000_000) == call(err=None) == INVALID
    if not gpu_available():
        assert call() == NO_DEVICE
