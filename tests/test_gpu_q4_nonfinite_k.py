"""Non-finite scales of an attended K block, with finite V: every head of the KV
head gives NaN, whatever the sign of its product with the block."""
import numpy as np
import pytest
import torch

from oracle import qsa_oracle as O
from qsa_workload import default_cfg, make_workload, quantize_q4_0
from sparse_attention_long_qsa_gb300 import qsa
from sparse_attention_long_qsa_gb300.layer import QSALayer, step_inputs

from gpu_util import assert_no_device_errors, max_rel, to_np

pytestmark = pytest.mark.gpu
CFG = default_cfg(kv_type="q4_0")
N = 700


def _attend(kc, vc, n, lists, q):
    cfg = qsa.config(kv_type="q4_0")
    T = len(lists)
    cells = np.full((T, qsa.cells_per_token(cfg)), -1, np.int32)
    for t, c in enumerate(lists):
        cells[t, :len(c)] = c
    out = torch.empty((T, 16, 256), device="cuda")
    qsa.sparse_attn(cfg, torch.from_numpy(q).cuda(), kc, vc, n, torch.from_numpy(cells).cuda(),
                    torch.tensor([len(c) for c in lists], dtype=torch.int32, device="cuda"), out)
    return to_np(out)


def _cache(seed):
    codes, d = quantize_q4_0(np.random.default_rng(seed).standard_normal((N, 2, 256)))
    return np.concatenate([codes.reshape(-1), d.reshape(-1).view(np.uint8)])


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("block", [0, 5])
def test_one_bad_scale_of_k(bad, block):
    kc, vc = _cache(1), _cache(2)
    q = np.random.default_rng(3).standard_normal((4, 16, 256)).astype(np.float16)
    q[2] = -q[1]                                  # both signs of every head's product
    clean = [O.attend(CFG, q[1], kc, vc, N, np.arange(N))]
    kc[N * 256:].view(np.float16).reshape(N, 2, 8)[333, 0, block] = bad
    k, v = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()
    # long lists, the cell alone, and a list without it
    out = _attend(k, v, N, [[333], np.arange(N), np.arange(N), np.delete(np.arange(N), 333)], q)
    assert np.all(np.isnan(out[:3, :8]))
    assert np.all(np.isfinite(out[:3, 8:])) and np.all(np.isfinite(out[3]))
    assert max_rel(out[1, 8:], clean[0][8:]) <= 2e-5    # the other KV head as before
    assert_no_device_errors()


def test_an_appended_key_with_one_infinity():
    """(its block decodes to an infinity among NaN)"""
    wl = make_workload(n_seq=1, prompt_len=300, n_steps=1, seed=4, kv_type="q4_0")
    L, st = QSALayer.from_workload(wl, 0), wl.steps[0]
    i = step_inputs(st, new_cells=True)
    k_new = i["k_new"].clone()
    k_new[0, 1, 70] = float("inf")
    L.kv_append(i["tok_seq"], i["tok_pos"], i["cells"], k_new, i["v_new"], i["idx_new"])
    q = np.random.default_rng(5).standard_normal((2, 16, 256)).astype(np.float16)
    q[1] = -q[0]
    cells = wl.seq_cells[0][:301]
    for lists in ([cells, cells], [st.cells, st.cells]):
        out = _attend(L.k_cache, L.v_cache, wl.n_cells, lists, q)
        assert np.all(np.isnan(out[:, 8:])) and np.all(np.isfinite(out[:, :8]))
