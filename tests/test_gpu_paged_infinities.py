"""paged_attn over fp16 rows whose values are infinite: a token that sees one gets
that infinity in its dim (two of opposite signs, or NaN: NaN), as the sum of the
definition does, whatever kernel a call goes to; all other dims keep their bits."""
import pytest
import torch

from paged_util import D, Paged, no_errors

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


# (one token: whole, and joined from many parts; a few tokens; a chunk of a prompt, alone and with a window and sinks)
@pytest.mark.parametrize("n,T,window,sinks", [(1, 1, 0, 0), (300, 1, 0, 0), (20_011, 1, 0, 0), (20_011, 5, 0, 0), (900, 40, 0, 0),
                                              (20_011, 40, 0, 0), (9_000, 70, 6_000, 5)])
def test_an_infinite_value_is_one_of_the_output(n, T, window, sinks):
    P = Paged("f16", (n,), seed=n + T)
    q, s, p = P.tokens([0] * T, list(range(n - T, n)))
    clean = P.attend(q, s, p, window, sinks)
    _, cells = P.visible(0, n - T, window, sinks)          # what all tokens see, but for the window's first T
    cells = cells[cells.numel() // 3:]
    at = lambda f: int(cells[int(f * (cells.numel() - 1))])   # noqa: E731
    want = {3: INF, 100: -INF, 131: NAN, 200: NAN, 255: INF}
    P.v[at(0.0), 1, 3] = INF
    P.v[at(0.5), 1, 100] = -INF
    P.v[at(0.9), 1, 100] = -INF
    P.v[at(0.2), 1, 131] = NAN
    P.v[at(0.0), 1, 200] = INF
    P.v[at(1.0), 1, 200] = -INF
    P.v[at(0.7), 1, 255] = INF
    if cells.numel() == 1:
        want[200] = -INF                                     # (one cell: the second value is the one that is there)
    out = P.attend(q, s, p, window, sinks)
    no_errors()
    assert torch.equal(out[:, :8], clean[:, :8])
    rest = [d for d in range(D) if d not in want]
    assert torch.equal(out[:, 8:, rest], clean[:, 8:, rest])
    for d, x in want.items():
        got = out[:, 8:, d]
        assert torch.all(got.isnan() if x != x else got == x), (d, x, got.flatten()[:8].tolist())
