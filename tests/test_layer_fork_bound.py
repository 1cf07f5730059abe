"""QSALayer.fork bounds a fork's blocks by what one sequence can have, not by
all sequences' lists together (the bound sizes the launch)."""
import numpy as np
import torch

from qsa_workload import make_workload
from sparse_attention_long_qsa_gb300 import build as qbuild
from sparse_attention_long_qsa_gb300 import qsa
from sparse_attention_long_qsa_gb300.layer import QSALayer


def test_the_bound_is_a_sequences(monkeypatch):
    qbuild.build()
    wl = make_workload(n_seq=3, prompt_len=[900, 400, 40], n_steps=1, seed=3)
    L = QSALayer.from_workload(wl, 0, device="cpu")
    got = []

    def seq_fork(cfg, src, dst, n_pos, slot, cells, off, lists, table, block, max_blocks, *rest):
        got.append(max_blocks)
    monkeypatch.setattr(qsa, "seq_fork", seq_fork)
    monkeypatch.setattr(qsa, "cells_copy", lambda *a, **k: None)
    one = torch.zeros(1, dtype=torch.int32)
    L.fork(one, one + 1, one + 396, one, torch.zeros((1, 4), dtype=torch.int32))
    assert got == [L.max_blocks]
    assert 900 // 4 <= L.max_blocks < int(np.diff(wl.seq_blk_off).sum())
