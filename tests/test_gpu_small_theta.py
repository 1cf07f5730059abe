"""Frequencies of more than a turn a position (rope_theta below 1 / 2 pi): block
keys turn by them as the indexer queries do."""
import numpy as np
import pytest
import torch

from oracle import qsa_oracle as O
from qsa_workload import default_cfg
from sparse_attention_long_qsa_gb300 import qsa

from gpu_util import assert_no_device_errors, check_pooled, to_np

pytestmark = pytest.mark.gpu


THETAS = [0.5, 0.125, 2.0 ** -10]


@pytest.mark.parametrize("theta", THETAS)
def test_pooled_keys_of_small_thetas(theta):
    r, n_slots = 4, 40
    cfg = default_cfg(rope_theta=theta)
    rng = np.random.default_rng(7)
    idx_k = rng.standard_normal((n_slots * r, 128)).astype(np.float16)
    table = rng.permutation(n_slots * r).reshape(n_slots, r).astype(np.int32)
    block = rng.integers(0, 5000, n_slots).astype(np.int32)
    w = (1.0 + 0.1 * rng.standard_normal(128)).astype(np.float32)
    dev = [torch.from_numpy(x).cuda() for x in (idx_k, table, block)]
    pooled = torch.zeros((n_slots, 128), device="cuda")
    qsa.pool_update(qsa.config(rope_theta=theta), *dev, torch.arange(n_slots, dtype=torch.int32, device="cuda"),
                    torch.from_numpy(w).cuda(), pooled)
    want = np.stack([O.pool_block(cfg, idx_k[table[s]], int(block[s]), w) for s in range(n_slots)])
    check_pooled(to_np(pooled), want)
    assert_no_device_errors()


@pytest.mark.parametrize("theta", THETAS + [1e6])
def test_queries_and_keys_turn_alike(theta):
    """A query and a block's only member, the same row at the same position, come out as the same row: both
    take angles from one table (the query's to 2^-32 of a turn), and each is off by at most 2^-20 of its pair."""
    cfg, n = qsa.config(rope_theta=theta, compress_ratio=1, top_k=512), 30
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.standard_normal((n, 128)).astype(np.float16)).cuda()
    w = torch.from_numpy((1.0 + 0.1 * rng.standard_normal(128)).astype(np.float32)).cuda()
    pos = torch.from_numpy(rng.integers(0, 200_000, n).astype(np.int32)).cuda()
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    pooled, q = torch.zeros((n, 128), device="cuda"), torch.zeros((n, 4, 128), device="cuda")
    qsa.pool_update(cfg, x, at.view(n, 1), pos, at, w, pooled)
    rope = qsa.rope_config((8,), cfg=cfg)
    qsa.qk_norm_rope(cfg, rope, None, None, None, None, None, None, None, x.unsqueeze(1).expand(n, 4, 128).contiguous(),
                     pos, w, q)
    a, b = to_np(pooled).astype(np.float64), to_np(q).astype(np.float64)
    pair = np.tile(np.abs(a[:, :64]) + np.abs(a[:, 64:]), 2)
    assert np.all(np.abs(a[:, None] - b) <= 2.0 ** -20 * 2 * pair[:, None])
    assert_no_device_errors()
