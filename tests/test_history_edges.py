"""Item ids and decay attention where a caller can go wrong, as far as it needs no GPU."""
import numpy as np
import pytest

import shared_prefix_behavior_b200 as R


def test_decay_heads_keep_the_arrays_that_the_calls_read():
    heads = R.DecayHeads((0, 64), (-0.1, -0.2), 16)
    at = heads.decay
    for name in ("taus", "log_decay"):
        with pytest.raises(AttributeError):
            setattr(heads, name, np.zeros(2))
    heads.log_decay[0] = -0.5
    heads.taus[1] = 0
    assert heads.decay == at == heads.log_decay.ctypes.data and not heads.timed
