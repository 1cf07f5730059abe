"""qsa_qk_norm_rope against the 64-bit definition.

Tolerance of one output (derived from the fp32 steps, u = 2^-24):
  a lane's 8 squares in two chains of four, their sum and 5 shuffle levels:
  relative 10u, halved by the root; eps 0.5u; rsqrtf's 2 ulp: 4u; the products
  with weight, partner and root: 4u.  In all 13.5u of |y_i cos| + |y_p sin|.
  Sine and cosine of |x| <= pi/4, a Taylor series to below 2e-9: x is off by 3u
  of itself (conversion, constant, product) and the angle by 2^-32 of a turn,
  the last steps by 1u: 2.7u at pi/4, where the first part is 0.71 of its
  largest, and 0.5u at 0.  In all below 15u < 2^-20 of |y_i| + |y_p|.  fp16
  outputs add half a step: 2^-11 of the value, or 2^-25 where fp16 is subnormal."""
import numpy as np
import pytest
import torch

from sparse_attention_long_qsa_gb300 import qsa
from gpu_util import to_np

pytestmark = pytest.mark.gpu
EPS, THETA = 1e-6, 1e6


def _axes(sections, interleaved):
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    i, n = np.arange(sum(sections)), len(sections)
    return np.where(i // n < np.array(sections)[i % n], i % n, 0)


def _ref(x, w, ang):
    """x [T][H][n] float64, ang [T][m]: (value, bound on |y_i| + |y_partner|)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
    m = ang.shape[1]
    a, b = y[..., :m], y[..., m:2 * m]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    out = np.concatenate([a * c - b * s, b * c + a * s, y[..., 2 * m:]], -1)
    mag = np.abs(a) + np.abs(b)
    return out, np.concatenate([mag, mag, np.abs(y[..., 2 * m:])], -1)


def _check(got, ref, mag, half):
    bound = 2.0 ** -20 * mag
    if half:
        bound = bound + np.maximum(2.0 ** -11 * np.abs(ref), 2.0 ** -25) * (1 + 2.0 ** -8)
    err = np.abs(to_np(got).astype(np.float64) - ref)
    assert np.all(err <= bound), (np.max(err / bound), np.argwhere(err > bound)[:4])


def _make(T, dtype, fused=True, scale=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = (torch.randn((T, 20 * 256), generator=g, device="cuda") * scale).to(dtype)
    if fused:
        q, k = qkv[:, :4096].unflatten(1, (16, 256)), qkv[:, 4096:4608].unflatten(1, (2, 256))
    else:
        q, k = qkv[:, :4096].reshape(T, 16, 256).contiguous(), qkv[:, 4096:4608].reshape(T, 2, 256).contiguous()
    qi = (torch.randn((T, 4, 128), generator=g, device="cuda") * scale).to(dtype)
    w = [1.0 + 0.3 * torch.randn(n, generator=g, device="cuda") for n in (256, 256, 128)]
    outs = [torch.full((T, 16, 256), 7.0, dtype=torch.float16, device="cuda"),
            torch.full((T, 2, 256), 7.0, dtype=torch.float16, device="cuda"),
            torch.full((T, 4, 128), 7.0, dtype=torch.float32, device="cuda")]
    return q, k, qi, w, outs


def _run_and_check(T, dtype, sections, interleaved, pos, idx_pos, **kw):
    q, k, qi, w, (qo, ko, io) = _make(T, dtype, **kw)
    rope = qsa.rope_config(sections, interleaved)
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    ip = torch.from_numpy(idx_pos.astype(np.int32)).cuda()
    qsa.qk_norm_rope(qsa.config(), rope, p, q, k, w[0], w[1], qo, ko, qi, ip, w[2], io)
    m = sum(sections)
    f = THETA ** (-np.arange(m) / m) if m else np.zeros(0)
    ang = pos.astype(np.float64)[_axes(sections, interleaved)].T * f if m else np.zeros((T, 0))
    iang = idx_pos.astype(np.float64)[:, None] * THETA ** (-np.arange(64) / 64.0)
    for got, x, wt, a, half in ((qo, q, w[0], ang, True), (ko, k, w[1], ang, True), (io, qi, w[2], iang, False)):
        ref, mag = _ref(x.double().cpu().numpy(), wt.double().cpu().numpy(), a)
        # cos and sin of angles up to 2^31 in float64: the product pos * f is off by 2^-53 of it
        _check(got, ref, mag * (1 + 2.0 ** 20 * 2.0 ** -53 * (np.abs(a).max() if a.size else 0)), half)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 7, 130])
@pytest.mark.parametrize("sections,interleaved", [((128,), False), ((0,), False), ((8,), False), ((32,), False),
                                                  ((48, 40, 40), False), ((24, 20, 20), True), ((8, 8, 8, 8), True),
                                                  ((0, 40, 24), False)])
def test_matches_the_definition(dtype, T, sections, interleaved):
    rng = np.random.default_rng(T + sum(sections))
    pos = rng.integers(0, 1_000_000, (len(sections), T))
    _run_and_check(T, dtype, sections, interleaved, pos, rng.integers(0, 1_000_000, T), fused=T != 7)


def test_far_and_negative_positions_and_small_rows():
    pos = np.array([[0, 1, -1, -250_000, 2**31 - 1, -2**31, 123_456_789]])
    _run_and_check(7, torch.float32, (128,), False, pos, pos[0][::-1].copy())
    _run_and_check(7, torch.float16, (128,), False, pos, pos[0], scale=1e-4)   # eps counts
    _run_and_check(7, torch.float32, (64,), False, pos, pos[0], scale=1e4)


def test_long_prompt():
    T = 4099
    pos = np.stack([np.arange(T), np.arange(T) // 64, np.arange(T) % 64])
    _run_and_check(T, torch.bfloat16, (24, 20, 20), True, pos, np.arange(T))


def test_zero_rows_nan_and_inf_stay_in_their_rows():
    q, k, qi, w, (qo, ko, io) = _make(3, torch.float16, fused=False)
    q[0, 3] = 0
    q[1, 5, 17] = float("nan")
    k[2, 1, 200] = float("inf")
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    qsa.qk_norm_rope(qsa.config(), qsa.rope_config((128,)), pos, q, k, w[0], w[1], qo, ko, qi, pos, w[2], io)
    assert bool((qo[0, 3] == 0).all())
    assert bool(qo[1, 5].isnan().all()) and bool(torch.isfinite(qo[1, :5]).all()) and bool(torch.isfinite(qo[2]).all())
    assert bool(ko[2, 1].isnan().any()) and bool(torch.isfinite(ko[2, 0]).all()) and bool(torch.isfinite(io).all())


def test_parts_in_place_other_stream_and_capture():
    q, k, qi, w, (qo, ko, io) = _make(33, torch.float16, fused=False)
    cfg, rope = qsa.config(), qsa.rope_config((64,))
    pos = torch.arange(33, dtype=torch.int32, device="cuda") * 77
    qsa.qk_norm_rope(cfg, rope, pos, q, k, w[0], w[1], qo, ko, qi, pos, w[2], io)
    only = torch.empty_like(ko)
    qsa.qk_norm_rope(cfg, rope, pos, None, k, None, w[1], None, only)
    assert torch.equal(only, ko)
    ionly = torch.empty_like(io)
    qsa.qk_norm_rope(cfg, rope, None, None, None, None, None, None, None, qi, pos, w[2], ionly)
    assert torch.equal(ionly, io)
    # in place, on another stream, and captured
    q2, s = q.clone(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qsa.qk_norm_rope(cfg, rope, pos, q2, None, w[0], None, q2, None, stream=s)
    s.synchronize()
    assert torch.equal(q2, qo)
    g, out = torch.cuda.CUDAGraph(), torch.zeros_like(qo)
    with torch.cuda.graph(g):
        qsa.qk_norm_rope(cfg, rope, pos, q, None, w[0], None, out, None)
    q.mul_(2.0)
    qsa.qk_norm_rope(cfg, rope, pos, q, None, w[0], None, qo, None)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, qo)


def test_pinned_inputs_and_outputs():
    q, k, qi, w, (qo, ko, io) = _make(2, torch.bfloat16, fused=False)
    cfg, rope = qsa.config(), qsa.rope_config((128,))
    pos = torch.tensor([5, 99_999], dtype=torch.int32, device="cuda")
    qsa.qk_norm_rope(cfg, rope, pos, q, k, w[0], w[1], qo, ko, qi, pos, w[2], io)
    pin = lambda t: t.cpu().pin_memory()  # noqa: E731
    po = torch.zeros((2, 16, 256), dtype=torch.float16).pin_memory()
    qsa.qk_norm_rope(cfg, rope, pin(pos), pin(q), None, w[0], None, po, None)
    torch.cuda.synchronize()
    assert torch.equal(po, qo.cpu())


def test_binding_checks_positions():
    q, k, qi, w, (qo, ko, io) = _make(3, torch.float16)
    cfg, rope = qsa.config(), qsa.rope_config((64, 64))
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (None, pos):                       # two axes want six positions
        with pytest.raises(ValueError, match="pos must hold"):
            qsa.qk_norm_rope(cfg, rope, bad, q, None, w[0], None, qo, None)
    with pytest.raises(ValueError, match="idx_pos must hold"):
        qsa.qk_norm_rope(cfg, rope, None, None, None, None, None, None, None, qi, None, w[2], io)
    with pytest.raises(TypeError):                # one element type for all inputs
        qsa.qk_norm_rope(cfg, rope, pos.repeat(2), q, k.float(), w[0], w[1], qo, ko)
    with pytest.raises(ValueError, match="contiguous"):
        qsa.qk_norm_rope(cfg, rope, pos.repeat(2), q.transpose(0, 1).contiguous().transpose(0, 1), None, w[0], None, qo, None)
