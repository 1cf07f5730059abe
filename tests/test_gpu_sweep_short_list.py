"""A list that ends before the offsets say: what the sequences would hold past
it is not there, and is flagged, not freed in silence."""
import numpy as np
import pytest
import torch

from sparse_attention_long_qsa_gb300 import qsa

from gpu_util import to_np

pytestmark = pytest.mark.gpu
BLOCK_LIST = 4      # qsa_debug_check's bit of a list shorter than its sequence needs


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("scale", [1, 200])       # one cluster, and kernels of their own
@pytest.mark.parametrize("compact", [False, True])
@pytest.mark.parametrize("lens,short,flagged", [([400, 300], 1, True), ([400, 300], 80, True), ([400, 0], 60, False),
                                                ([400, 296], 1, False), ([400, 0], 80, True)])
def test_offsets_past_the_list(scale, compact, lens, short, flagged):
    lens, short = [scale * x for x in lens], scale * short
    n_slots, n = 175 * scale, 700 * scale
    off = torch.tensor([0, 100 * scale, 175 * scale], device="cuda")
    table = np.arange(n).reshape(n_slots, 4)
    lists = np.arange(n_slots)[:n_slots - short]
    cfg, counts = qsa.config(), _i32(np.zeros(4))
    out, cell_map = _i32(np.zeros((n_slots, 4))), _i32(np.zeros(n))
    ws = torch.empty(qsa.cache_sweep_workspace_size(cfg, n, n_slots), dtype=torch.uint8, device="cuda")
    qsa.debug_check()
    qsa.cache_sweep(cfg, _i32(lens), off, _i32(lists), _i32(table), out, n, counts, ws, compact, cell_map=cell_map,
                    move_src=_i32(np.zeros(n // 2)), move_dst=_i32(np.zeros(n // 2)))
    st, flags = qsa.debug_check()
    assert (st, flags) == ((-6, BLOCK_LIST) if flagged else (0, 0))
    held = sum(min(x, 4 * max(0, min(e, len(lists)) - b)) for x, b, e in
               zip(lens, (0, 100 * scale), (100 * scale, 175 * scale)))
    assert to_np(counts)[0] == held
