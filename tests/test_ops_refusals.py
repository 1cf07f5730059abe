"""Refusals of the calls around the step (head norms, cache rows, forks,
sweeps) and of the q4_0 configuration, made on the host before any launch: no
GPU is needed.  Also the q4_0 encoders of the oracle and of the input
generator, pinned by hand and against each other."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import qsa_oracle as O
from qsa_workload import default_cfg, quantize_q4_0
from sparse_attention_long_qsa_gb300 import build as qbuild
from sparse_attention_long_qsa_gb300 import qsa

F = 0x10000   # an aligned address that is never read


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return qsa.lib()


def _call(fn, base, **kw):
    args = list(base)
    for i, v in kw.items():
        args[int(i[1:])] = v
    return fn(*args)


def test_rope_init(L):
    c = qsa.config()
    r = qsa.rope_config((16, 8, 8), interleaved=False)
    assert (r.n_rot, r.n_axes) == (64, 3)
    assert list(r.axis[:32]) == [0] * 16 + [1] * 8 + [2] * 8
    r = qsa.rope_config((16, 8, 8), interleaved=True)
    assert list(r.axis[:32]) == [i % 3 if i // 3 < (16, 8, 8)[i % 3] else 0 for i in range(32)]
    assert sorted(r.axis[:32]).count(1) == 8 and sorted(r.axis[:32]).count(2) == 8
    # theta^(-2i/64) / 2 pi as a 64-bit fraction: rounded to a whole unit (half of one), from doubles of 53 bits
    for i in (0, 1, 17, 31):
        want = 1e6 ** (-2.0 * i / 64) / (2 * np.pi) * 2.0 ** 64
        assert abs(r.turns[i] - want) <= 0.5 + want * 2.0 ** -50
    assert qsa.rope_config(()[:0] + (0,)).n_rot == 0

    def init(sections, interleaved=0, n=None, cfg=c):
        out = qsa.Rope()
        arr = (ctypes.c_int32 * max(len(sections), 1))(*sections)
        return L.qsa_rope_init(ctypes.byref(cfg), len(sections) if n is None else n, arr, interleaved, ctypes.byref(out))
    assert init((8, 8, 8, 8)) == 0
    assert init((), n=0) == -1
    assert init((8,) * 5) == -3                  # more than four axes
    assert init((8, -8, 16)) == -1
    assert init((136,)) == -2                    # more pairs than a head has
    assert init((12,)) == -3                     # not a multiple of 8
    assert init((8, 8), interleaved=2) == -1
    assert init((0, 16), interleaved=1) == -2    # axis 1 would get every other pair only
    assert init((8,), cfg=qsa.config(head_dim=128)) == -3
    assert L.qsa_rope_init(ctypes.byref(c), 1, None, 0, ctypes.byref(qsa.Rope())) == -1
    assert L.qsa_rope_init(ctypes.byref(c), 1, (ctypes.c_int32 * 1)(8), 0, None) == -1


@pytest.mark.parametrize("theta", [0.5, 0.1, 1e-3])
def test_rope_frequencies_of_several_turns(theta):
    """Whole turns of a frequency above 2 pi do not count.  The frequency is a double (the power to an ulp or two:
    2^-51 of it), so its turns are off by at most 2^-51 of them; the rounding to a whole unit adds half of one."""
    r = qsa.rope_config((64,), cfg=qsa.config(rope_theta=theta))
    th = float(np.float32(theta))
    for table, m in ((r.turns, 64), (r.idx_turns, 64)):
        for i in (0, 1, 31, 63):
            turns = th ** (-i / m) / (2 * np.pi)
            got = table[i] / 2.0 ** 64
            err = abs(got - turns % 1.0)
            assert min(err, 1.0 - err) <= 2.0 ** -50 * (1.0 + turns)


def test_norm_rope_host_checks(L):
    c, r = qsa.config(), qsa.rope_config((64,))
    #       0                1                2  3  4  5  6     7  8    9  10 11 12 13 14 15   16 17 18
    base = [ctypes.byref(c), ctypes.byref(r), 4, 1, F, F, 5120, F, 5120, F, F, F, F, F, F, 512, F, F, None]
    call = lambda **kw: _call(L.qsa_qk_norm_rope, base, **kw)  # noqa: E731
    assert call(a2=0) == 0                       # nothing to do
    assert call(a5=None, a11=None, a7=None, a12=None, a13=None, a14=None, a17=None) == 0
    assert call(a2=-1) == -1
    assert call(a3=3) == -1                      # unknown element type
    assert call(a1=None) == -1
    assert call(a1=ctypes.byref(qsa.Rope())) == -1          # not made by qsa_rope_init
    assert call(a4=None) == -1                   # no positions
    assert call(a13=None) == -1                  # no cache positions for the indexer queries
    assert call(a5=None) == -1                   # an output without its input
    assert call(a11=None) == -1                  # an input without its output
    assert call(a9=None) == -1                   # no weight
    assert call(a5=F + 2) == -1
    assert call(a6=5121) == -1                   # rows not 16-byte aligned
    assert call(a6=4088) == -2                   # tokens would overlap
    assert call(a8=504) == -2
    assert call(a15=508) == -2
    assert call(a15=513) == -1
    assert call(a3=2, a6=5122) == -1
    assert call(a0=ctypes.byref(qsa.config(head_dim=128))) == -3
    bad = qsa.rope_config((64,))
    bad.axis[5] = 1                              # an axis that pos does not have
    assert call(a1=ctypes.byref(bad)) == -1


def test_kv_read_and_cells_copy_host_checks(L):
    c = qsa.config(kv_type="q4_0")
    base = [ctypes.byref(c), 4, F, F, F, 1000, F, F, None]
    call = lambda **kw: _call(L.qsa_kv_read, base, **kw)  # noqa: E731
    assert call(a1=0, a2=None, a6=None) == 0
    assert call(a1=-1) == -1 and call(a5=-1) == -1 and call(a5=1 << 31) == -3
    assert call(a2=None) == -1 and call(a3=F + 8) == -1 and call(a6=F + 8) == -1 and call(a7=None) == -1
    base = [ctypes.byref(c), 4, None, F, F, F, F, F, 1000, None]
    call = lambda **kw: _call(L.qsa_cells_copy, base, **kw)  # noqa: E731
    assert call(a1=0, a3=None) == 0
    assert call(a1=-1) == -1 and call(a8=-1) == -1 and call(a8=1 << 31) == -3
    assert call(a3=None) == -1 and call(a4=None) == -1 and call(a5=F + 4) == -1 and call(a7=F + 4) == -1
    assert call(a0=ctypes.byref(qsa.config(kv_type=3))) == -1


def test_seq_fork_host_checks(L):
    c = qsa.config()
    base = [ctypes.byref(c), 2, F, F, F, F, F, F, F, 3, 100, F, F, 100, 1000, 50, F, F, None]
    call = lambda **kw: _call(L.qsa_seq_fork, base, **kw)  # noqa: E731
    assert call(a1=0, a2=None) == 0
    assert call(a1=-1) == -1 and call(a1=65_536) == -3
    for i in (2, 3, 4, 5, 6, 7, 8, 11, 12, 16, 17):
        assert call(**{f"a{i}": None}) == -1
    assert call(a9=0) == -1 and call(a15=-1) == -1 and call(a10=-1) == -1
    assert call(a13=1 << 31) == -3 and call(a15=1 << 31) == -3


def test_cache_sweep_host_checks(L):
    c = qsa.config()
    need = L.qsa_cache_sweep_workspace_size(ctypes.byref(c), 100_000, 30_000)
    assert need >= 100_000 // 8 + 30_000 // 8
    assert L.qsa_cache_sweep_workspace_size(ctypes.byref(c), -1, 5) == 0
    base = [ctypes.byref(c), 1, F, F, F, 3, 30_000, F, F, 30_000, 100_000, F, F, F, F, F, F, F, need, None]
    call = lambda **kw: _call(L.qsa_cache_sweep, base, **kw)  # noqa: E731
    for i in (2, 3, 4, 7, 8, 11, 12, 15, 16):
        assert call(**{f"a{i}": None}) == -1, i
    assert call(a1=2) == -1 and call(a5=0) == -1 and call(a6=-1) == -1 and call(a10=1 << 31) == -3
    assert call(a17=None) == -4 and call(a17=F + 16) == -4 and call(a18=need - 1) == -4


def test_q4_0_refuses_the_union(L):
    c = qsa.config(kv_type="q4_0")
    assert L.qsa_sparse_attn_union(ctypes.byref(c), 2, F, F, F, 100, F, F, F, None, 0, None) == -3
    need = L.qsa_index_topk_workspace_size(ctypes.byref(c), 5, 1000)
    args = [ctypes.byref(c), 5, 5] + [F] * 6 + [100, F, F, 1, 1000, F, F, F, 1000, F, F, F, None, 0]
    assert L.qsa_index_attn(*args, 2, F, need, None) == -3
    assert L.qsa_index_attn_kernels(ctypes.byref(c), 5, 1, 1000, 2) == 0
    # the selection inside the attention clusters is not offered for q4_0: the separate kernels run
    assert qsa.index_attn_kernels(c, 5, 1, 1000, in_cluster=True) == ["score", "select", "attn"]


def test_binding_refusals(L):
    c = qsa.config(kv_type="q4_0")
    t = torch.zeros((1, 16, 256), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.kv_read(c, torch.zeros(1, dtype=torch.int32), torch.zeros(288, dtype=torch.uint8),
                    torch.zeros(288, dtype=torch.uint8), 1, torch.zeros((1, 2, 256)), torch.zeros((1, 2, 256)))
    with pytest.raises(ValueError, match="bytes"):
        qsa.kv_read(c, torch.zeros(1, dtype=torch.int32), torch.zeros(287, dtype=torch.uint8),
                    torch.zeros(288, dtype=torch.uint8), 1, torch.zeros((1, 2, 256)), torch.zeros((1, 2, 256)))
    r = qsa.rope_config((64,))
    with pytest.raises(ValueError, match="contiguous"):
        qsa.qk_norm_rope(c, r, None, torch.zeros((1, 16, 512))[:, :, ::2], None, None, None, t, None)
    with pytest.raises(TypeError):
        qsa.qk_norm_rope(c, r, None, torch.zeros((1, 16, 256), dtype=torch.float64), None, None, None, t, None)
    with pytest.raises(ValueError, match="same length"):
        i = torch.zeros(3, dtype=torch.int32)
        qsa.cells_copy(c, i, i[:2], t, t, None, 1)
    with pytest.raises(ValueError, match="must hold"):
        i = torch.zeros(3, dtype=torch.int32)
        qsa.seq_fork(c, i, i, i, i, i, i.long(), i, i.view(3, 1), i, 4, i, i)


def test_an_empty_pair_count_is_refused(L):
    """(an empty tensor has no address, and no address would mean that all pairs count)"""
    i, c = torch.zeros(3, dtype=torch.int32), qsa.config()
    rows = torch.zeros((1, 2, 256), dtype=torch.float16)
    with pytest.raises(ValueError, match="n_pairs must hold one value"):
        qsa.cells_copy(c, i, i, rows, rows, None, 1, n_pairs=i[:0])


# ------------------------------------------------------------------ q4_0
def test_q4_0_block_closed_forms():
    x = np.zeros(32, dtype=np.float32)
    codes, d = O.q4_0_block(x)
    assert d == 0 and np.all(codes == 8)
    x[3], x[20] = -8.0, 7.0                       # d = 1: codes are the values + 8
    codes, d = O.q4_0_block(x)
    assert d == 1 and codes[3] == 0 and codes[20] == 15 and np.all(np.delete(codes, [3, 20]) == 8)
    x[:] = 0
    x[0], x[1], x[2] = 4.0, -4.0, 0.25            # the first of equal magnitudes sets the sign: d = -0.5
    codes, d = O.q4_0_block(x)
    assert d == -0.5 and codes[0] == 0 and codes[1] == 15 and codes[2] == 8   # 0.25 / -0.5 + 8.5 = 8.0
    x[:] = 0
    x[31], x[0] = 8.0, -7.5                       # 7.5 + 8.5 = 16 is clamped to 15
    codes, d = O.q4_0_block(x)
    assert d == -1 and codes[31] == 0 and codes[0] == 15


def test_q4_0_encoders_agree_and_bound():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 64)).astype(np.float16).astype(np.float32)
    x[:4] *= 1e-5
    x[4:8] *= 1e4
    codes, d = quantize_q4_0(x)
    cfg = default_cfg(kv_type="q4_0", n_kv_heads=1, head_dim=64)
    raw = np.concatenate([codes.reshape(-1), d.reshape(-1).view(np.uint8)])
    got = O.kv_rows(cfg, raw, 40, range(40), 0)
    for i in range(40):
        for b in range(2):
            blk = x[i, 32 * b:32 * b + 32]
            c, db = O.q4_0_block(blk)
            assert db.view(np.uint16) == d[i, b].view(np.uint16)
            np.testing.assert_array_equal(got[i, 32 * b:32 * b + 32], (c - 8) * np.float64(db))
            # a step of d: half of it by rounding, up to a whole one where the top code is clamped;
            # d itself is off by fp16's 2^-11 (subnormals: 2^-25) times at most 8 codes
            dd = np.abs(blk).max() / 8
            assert np.all(np.abs(got[i, 32 * b:32 * b + 32] - blk) <= dd * (1 + 2.0 ** -8) + 2.0 ** -22)
