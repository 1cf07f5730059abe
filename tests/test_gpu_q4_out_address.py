"""The attention over a q4_0 cache writes its output at any float address, as
the other cache types do, whatever cluster size the call gets."""
import numpy as np
import pytest
import torch

from qsa_workload import quantize_q4_0
from sparse_attention_long_qsa_gb300 import qsa

from gpu_util import assert_no_device_errors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 40, 200, 400])
def test_output_at_any_float_address(T):
    n, cfg = 3000, qsa.config(kv_type="q4_0")
    rng = np.random.default_rng(T)
    cache = []
    for _ in range(2):
        codes, d = quantize_q4_0(rng.standard_normal((n, 2, 256)))
        cache.append(torch.from_numpy(np.concatenate([codes.reshape(-1), d.reshape(-1).view(np.uint8)])).cuda())
    cells = torch.from_numpy(rng.integers(0, n, (T, qsa.cells_per_token(cfg))).astype(np.int32)).cuda()
    count = torch.from_numpy(rng.integers(0, 700, T).astype(np.int32)).cuda()
    q = torch.from_numpy(rng.standard_normal((T, 16, 256)).astype(np.float16)).cuda()
    want = torch.full((T, 16, 256), 3.0, device="cuda")
    qsa.sparse_attn(cfg, q, *cache, n, cells, count, want)
    for off in (1, 2, 3):
        buf = torch.full((T * 4096 + 8,), 7.0, device="cuda")
        qsa.sparse_attn(cfg, q, *cache, n, cells, count, buf[off:off + T * 4096].view(T, 16, 256))
        assert torch.equal(buf[off:off + T * 4096].view(T, 16, 256), want)
        assert bool((buf[:off] == 7).all()) and bool((buf[off + T * 4096:] == 7).all())
    assert_no_device_errors()
