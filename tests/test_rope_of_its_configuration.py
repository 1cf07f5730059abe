"""A rotation table belongs to its configuration's rope_theta: with another one
the queries would turn by other frequencies than the block keys."""
import ctypes

import pytest

from sparse_attention_long_qsa_gb300 import build as qbuild
from sparse_attention_long_qsa_gb300 import qsa

F = 0x10000   # an aligned address that is never read


def test_another_theta_is_refused():
    qbuild.build()
    c = qsa.config(rope_theta=1e4)

    def call(rope, cfg, n, q_idx=True):
        idx = (F, F, 512, F, F) if q_idx else (None, None, 0, None, None)
        return qsa.lib().qsa_qk_norm_rope(ctypes.byref(cfg), ctypes.byref(rope), n, 1, F, F, 5120, F, 5120, F, F, F, F,
                                          *idx, None)
    other = qsa.rope_config((64,))                          # of the default configuration
    assert other.rope_theta == 1e6
    assert call(other, c, 4) == -1 and call(other, c, 4, q_idx=False) == -1 and call(other, c, 0) == -1
    own = qsa.rope_config((64,), cfg=c)
    assert own.rope_theta == 1e4
    assert call(own, c, 0) == 0                             # (no tokens: nothing is launched)
    assert call(own, qsa.config(), 4) == -1
    # what else differs between two configurations does not matter
    assert call(other, qsa.config(kv_type="q4_0", rms_eps=1e-5), 0) == 0
    with pytest.raises(qsa.QSAError, match="INVALID_ARG"):
        qsa._check(call(other, c, 4), "qsa_qk_norm_rope")
