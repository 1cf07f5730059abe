"""paged_attn of scores so large that their last place is more than the softmax's range:
nearly all weight goes to the largest (which of close ones, rounding decides), the
output stays a mean of values, and no probability leaves its type's range."""
import pytest
import torch

from paged_util import Paged, no_errors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("scale,k_mul,q_mul", [(1 / 16, 100.0, 600.0), (1 / 16, 300.0, 2000.0), (1.0, 300.0, 2000.0), (-30.0, 1000.0, 2000.0),
                                               (5e3, 3000.0, 8000.0)])
def test_outputs_stay_means_of_values(kv, T, scale, k_mul, q_mul):
    n = 900
    P = Paged(kv, (n,), seed=T, scale=scale, k_mul=k_mul)
    q, s, p = P.tokens([0] * T, list(range(n - T, n)), q_mul=q_mul)
    w = torch.zeros(P.slots.numel(), device="cuda") if T != 40 else None
    out = P.attend(q, s, p, weight=w)
    no_errors()
    P.check(out, q, s, p)                                     # (a bound of thousands where rounding decides)
    assert out.isfinite().all()
    V = P.V[P.visible(0, n - 1)[1]]
    top = V.abs().amax((0, 2)).repeat_interleave(8).view(1, 16, 1)
    assert torch.all(out.double().abs() <= top * (1 + 1e-3))
    if w is not None:
        assert abs(float(w.double().sum()) - 16 * T) <= 1e-3 * 16 * T
    # where one cell is far ahead of all others, the output is its values
    for t in range(T):
        j, c = P.visible(0, int(p[t]))
        x = q[t].double().view(2, 8, 256)
        raw = torch.einsum("ghd,cgd->ghc", x, P.K[c]) * scale
        mag = torch.einsum("ghd,cgd->ghc", x.abs(), P.K[c].abs()).amax(-1) * abs(scale)
        two = raw.topk(2, dim=-1)
        sure = two.values[..., 0] - two.values[..., 1] > 64 * 2.0 ** -23 * mag + 50
        best = P.V[c][two.indices[..., 0], torch.arange(2, device="cuda").unsqueeze(1)]
        err = (out[t].view(2, 8, 256).double() - best).abs().amax(-1)
        assert torch.all(err[sure] <= 1e-3 * V.abs().max()), t
