"""qsa_seq_fork of a sequence that an eviction has shortened: its partial block's
keys turn by the positions they had, which slot_block_idx says, not by the block's
place in the list; so does the private copy's."""
import numpy as np
import pytest
import torch

from sparse_attention_long_qsa_gb300 import qsa

pytestmark = pytest.mark.gpu
R, D = 4, 128


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("evicted", [0, 1, 37])
def test_the_private_tail_block_keeps_its_index(evicted):
    rng = np.random.default_rng(evicted)
    nb, tail, cells = 20, 3, 200
    off = torch.tensor([0, 24, 48], dtype=torch.int64, device="cuda")
    lists = np.full(48, -1)
    lists[:nb + 1] = np.arange(nb + 1)
    table = np.full((30, R), -1)
    table[:nb] = np.arange(nb * R).reshape(nb, R)
    table[nb, :tail] = nb * R + np.arange(tail)
    block = np.zeros(30)
    block[:nb + 1] = np.arange(nb + 1) + evicted            # the places the blocks had
    d_lists, d_table, d_block = _i32(lists), _i32(table), _i32(block)
    cfg = qsa.config(compress_ratio=R)
    cs, cd = _i32(np.zeros((1, R))), _i32(np.zeros((1, R)))
    fresh = np.array([[150, 151, 152, 153]])
    qsa.seq_fork(cfg, _i32([0]), _i32([1]), _i32([nb * R + tail]), _i32([25]), _i32(fresh), off, d_lists, d_table, d_block, nb,
                 cs, cd, cells)
    assert int(d_block[25]) == nb + evicted
    assert torch.equal(d_lists[24:24 + nb], d_lists[:nb]) and int(d_lists[24 + nb]) == 25
    # the same keys in the copy, one position more in each: the pooled keys agree bit for bit
    idx_k = torch.from_numpy(rng.standard_normal((cells, D)).astype(np.float16)).cuda()
    idx_k[cd[0, :tail].long()] = idx_k[cs[0, :tail].long()]
    idx_k[153] = idx_k[nb * R + tail]
    d_table[nb, tail], d_table[25, tail] = nb * R + tail, 153
    pooled = torch.zeros((30, D), device="cuda")
    qsa.pool_update(cfg, idx_k, d_table, d_block, _i32([nb, 25, -1, -1]), torch.ones(D, device="cuda"), pooled)
    torch.cuda.synchronize()
    assert qsa.debug_check() == (0, 0)
    assert bool(pooled[25].any()) and torch.equal(pooled[nb], pooled[25])
