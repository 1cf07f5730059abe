"""Attention over q4_0 caches whose scales lie far apart, each 32-dim block of
an output measured by its own size.

Tolerance 2e-5 of a block's norm: as for rows of equal scales, a cell's score is
off by the rounding of some 270 fp32 additions, so its probability by a relative
1.6e-5 at four standard deviations, and the errors of different cells are
independent; the weights behind it lose at most 2^-18 (4e-6) of what a chunk of
cells adds to a block.  A block's norm over 32 dims and the sum over cells average these
errors, and the values of different cells are independent, so that a block's
norm is not the remainder of a cancellation."""
import numpy as np
import pytest
import torch

from oracle import qsa_oracle as O
from qsa_workload import default_cfg, quantize_q4_0
from sparse_attention_long_qsa_gb300 import qsa

from gpu_util import assert_no_device_errors, to_np

pytestmark = pytest.mark.gpu
TOL = 2e-5


def _pack(x):
    codes, d = quantize_q4_0(x)
    return np.concatenate([codes.reshape(-1), d.reshape(-1).view(np.uint8)])


def _check(k, v, q, lists, scale=1.0 / 16.0):
    """k, v: fp32 rows [n][2][256]; q fp16 [T][16][256]."""
    n, T = len(k), len(lists)
    kc, vc, cfg = _pack(k), _pack(v), qsa.config(kv_type="q4_0", attn_scale=scale)
    plain = default_cfg(kv_type="q4_0", attn_scale=scale)
    cells = np.full((T, qsa.cells_per_token(cfg)), -1, np.int32)
    for t, c in enumerate(lists):
        cells[t, :len(c)] = c
    out = torch.empty((T, 16, 256), device="cuda")
    qsa.sparse_attn(cfg, torch.from_numpy(q).cuda(), torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), n,
                    torch.from_numpy(cells).cuda(), torch.tensor([len(c) for c in lists], dtype=torch.int32, device="cuda"),
                    out)
    ref = np.stack([O.attend(plain, q[t], kc, vc, n, np.asarray(lists[t])) for t in range(T)])
    err = np.linalg.norm((to_np(out) - ref).reshape(T, 16, 8, 32), axis=-1)
    size = np.linalg.norm(ref.reshape(T, 16, 8, 32), axis=-1)
    tol = TOL * max(1.0, 16 * abs(scale))   # a score's error grows with the scale
    assert np.all(err <= tol * size), np.max(err / size, axis=(0, 1))
    assert_no_device_errors()


def _rows(seed, n=2051):
    rng = np.random.default_rng(seed)
    return rng, rng.standard_normal((n, 2, 256)), rng.standard_normal((n, 2, 256))


def _alike(rng, T=1):
    """Queries of one direction per KV head, and that direction: keys along it
    raise or lower the scores of all its heads together (by 16 a unit)."""
    u = rng.standard_normal((2, 256))
    q = np.repeat(u, 8, axis=0)[None] + 0.3 * rng.standard_normal((T, 16, 256))
    return q.astype(np.float16), u


# one token in a cluster of 16 CTAs, and 200 in single CTAs
@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("ratio,base", [(100.0, 1.0), (3e3, 1.0), (1e6, 2e-3)])
def test_one_block_larger_in_every_cell(T, ratio, base):
    rng, k, v = _rows(int(ratio) + T, 1000)
    v *= base
    v[:, :, 64:96] *= ratio
    q = rng.standard_normal((T, 16, 256)).astype(np.float16)
    _check(k, v, q, [rng.permutation(1000)[:700] for _ in range(T)])


@pytest.mark.parametrize("ratio", [1e3, 3e3, 1e4])
def test_unlikely_cells_of_large_values(ratio):
    """64 of 2,051 cells, likely 2^-30 as much, with values `ratio` times as large."""
    rng, k, v = _rows(int(ratio))
    q, u = _alike(rng)
    far = rng.permutation(2051)[:64]
    k[far] = -1.3 * u[None]
    v[far] *= ratio
    for order in (np.arange(2051), np.concatenate([far, np.setdiff1d(np.arange(2051), far)])):
        _check(k, v, q, [order])


@pytest.mark.parametrize("small", [0.0, 2.0 ** -12, 2.0 ** -20])
@pytest.mark.parametrize("up", [0.5, 1.1])
def test_a_likely_cell_with_a_small_block(small, up):
    """A cell 2^11 or 2^25 times as likely as the others, with one block of (almost) zeros: there the
    others are the output."""
    rng, k, v = _rows(int(up * 10))
    q, u = _alike(rng)
    k[77] = up * u
    v[77, :, 96:128] *= small
    _check(k, v, q, [np.arange(2051)])
    v[78:90, :, 32:64] = 0          # and zero blocks among the others
    _check(k, v, q, [np.arange(2051)])


@pytest.mark.parametrize("T", [1, 200])
def test_scales_over_the_whole_range(T):
    """Every cell's and block's scale drawn from the normal and subnormal halves."""
    rng, k, v = _rows(9 + T, 1000)
    v *= np.exp2(rng.uniform(-19, 13, (1000, 2, 8))).repeat(32, axis=-1)
    q = rng.standard_normal((T, 16, 256)).astype(np.float16)
    _check(k, v, q, [rng.permutation(1000)[:700] for _ in range(T)])
    v = rng.standard_normal((1000, 2, 256)) * 1e-6     # subnormal scales only
    _check(k, v, q, [rng.permutation(1000)[:700] for _ in range(T)])


@pytest.mark.parametrize("down", [12, 16, 20])
def test_queries_of_large_and_small_dims(down):
    """One block of a head's queries 2^down times as large as the others, the keys the other way round: both
    parts count alike in the scores.  With the largest query brought to 2^14 the others lie, divided by 16,
    around 2^(10 - down) or above: at down = 20 some 4 % of them are subnormal halves, off by at most 2^-25,
    2^-15 of their deviation, which moves a score by less than 2e-6."""
    rng, k, v = _rows(down, 1500)
    big = np.s_[..., 160:192]
    q = rng.standard_normal((2, 16, 256)) * 2.0 ** (14 - down)
    q[big] = rng.standard_normal((2, 16, 32)) * 2.0 ** 13
    k *= 2.0 ** (down - 14)
    k[big] = rng.standard_normal((1500, 2, 32)) * 2.0 ** -13
    _check(k, v, q.astype(np.float16), [np.arange(1500), rng.permutation(1500)[:33]])


@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("blocks", [[0], [6, 7], list(range(8))])
def test_blocks_of_zeros_in_every_cell(T, blocks):
    """Dims of padding: exact zeros there, the other blocks as without them; and one cell of the list that is
    zero throughout."""
    rng, k, v = _rows(17 + T, 1000)
    v.reshape(1000, 2, 8, 32)[:, :, blocks] = 0
    v[500] = 0
    q = rng.standard_normal((T, 16, 256)).astype(np.float16)
    _check(k, v, q, [rng.permutation(1000)[:701] for _ in range(T)])


@pytest.mark.parametrize("top", [1.0, 2.0 ** -8, 2.0 ** -11, 2.0 ** -13, 2.0 ** -14, 2.0 ** -15, 2.0 ** -18])
@pytest.mark.parametrize("ratio", [2.0 ** 5, 2.0 ** 9, 2.0 ** 11, 2.0 ** 13])
def test_scales_around_the_forms_limits(top, ratio):
    """Scales spread over a ratio below a largest one, normal and subnormal, with the likely cells at either end."""
    rng, k, v = _rows(23, 640)
    q, u = _alike(rng)
    f = np.exp2(-rng.uniform(0, np.log2(ratio), (640, 2, 8)))
    f[::16], f[5::16] = 1.0, 1.0 / ratio             # both ends in every chunk
    v *= (f * top * 3).repeat(32, axis=-1)
    for sign in (-0.5, 0.5):
        kk = k.copy()
        kk[5::16] += sign * u
        _check(kk, v, q, [np.arange(640)])


@pytest.mark.parametrize("scale", [0.0, -1.0 / 16.0, 1.0 / 256.0, 0.5])
@pytest.mark.parametrize("T", [1, 200])
def test_attention_scales(T, scale):
    """From all cells alike to one or two that count (a chunk's likeliest cells 2^100 apart)."""
    rng, k, v = _rows(31 + T, 900)
    q = rng.standard_normal((T, 16, 256)).astype(np.float16)
    _check(k, v, q, [rng.permutation(900)[:650 + t % 50] for t in range(T)], scale)
