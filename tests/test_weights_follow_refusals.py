"""Refusals of qsa_weight_trim and of block weights in qsa_seq_fork_weighed: no GPU is needed."""
import ctypes

import pytest
import torch

from sparse_attention_long_qsa_gb300 import build as qbuild
from sparse_attention_long_qsa_gb300 import qsa

F = 0x10000   # an aligned address that is never read


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qsa.lib()


def test_weight_trim_host_checks(L):
    c = qsa.config()
    base = [ctypes.byref(c), F, F, 2, 300, F, None]

    def call(**kw):
        args = list(base)
        for i, v in kw.items():
            args[int(i[1:])] = v
        return L.qsa_weight_trim(*args)
    assert call(a3=0, a1=None) == 0                          # nothing to do
    for i in (1, 2, 5):
        assert call(**{f"a{i}": None}) == -1, i
    assert call(a1=F + 2) == -1 and call(a2=F + 4) == -1 and call(a5=F + 2) == -1
    assert call(a3=-1) == -1 and call(a4=-1) == -1 and call(a4=1 << 31) == -3
    assert call(a0=None) == -1 and call(a0=ctypes.byref(qsa.config(head_dim=128))) == -3


def test_fork_weights_host_checks(L):
    c = qsa.config()
    #        0               1  2  3  4  5  6  7  8  9  10   11 12 13   14    15  16 17 18 19
    base = [ctypes.byref(c), 3, F, F, F, F, F, F, F, 4, 300, F, F, 200, 1000, 50, F, F, F, None]

    def call(**kw):
        args = list(base)
        for i, v in kw.items():
            args[int(i[1:])] = v
        return L.qsa_seq_fork_weighed(*args)
    assert call(a1=0, a2=None) == 0
    assert call(a18=F + 2) == -1 and call(a8=None) == -1 and call(a1=65_536) == -3


def test_binding_refuses_weights_of_another_length():
    c = qsa.config()
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_weight must hold"):
        qsa.seq_fork(c, i, i, i, i, torch.zeros((3, 4), dtype=torch.int32), torch.zeros(4, dtype=torch.int64), i,
                     torch.zeros((5, 4), dtype=torch.int32), torch.zeros(5, dtype=torch.int32), 4,
                     torch.zeros((3, 4), dtype=torch.int32), torch.zeros((3, 4), dtype=torch.int32),
                     block_weight=torch.zeros(4))
    with pytest.raises(ValueError, match="seq_len must hold"):
        qsa.weight_trim(c, i, torch.zeros(3, dtype=torch.int64), torch.zeros(4))
    with pytest.raises(ValueError, match="required"):
        qsa.weight_trim(c, None, torch.zeros(3, dtype=torch.int64), torch.zeros(4))
