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


@pytest.mark.parametrize("kv", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("n,T", [(200, 1), (200, 5), (200, 40), (5_000, 1), (5_000, 5), (5_000, 40)])
def test_a_token_whose_scores_are_nan_is_nan(kv, n, T):
    """Beside infinite values of V, too; tokens before the cell, and the other KV head, are as they were."""
    P = Paged(kv, (n,), seed=n + T)
    q, s, p = P.tokens([0] * T, list(range(n - T, n)))
    first = n - 1 - T // 2                                   # the first token to see the cell
    clean = P.attend(q, s, p)
    cells = P.visible(0, n - 1)[1]
    if kv == "f16":
        P.k[cells[first], 1, 17] = NAN
        P.v[cells[n // 2], 1, 40] = INF
        dims = [40]
    else:
        codes = P.n_cells * 2 * (256 if kv == "q8_0" else 128)
        for raw, c, block in ((P.k, cells[first], 0), (P.v, cells[n // 2], 1)):
            raw[codes:].view(torch.float16).view(P.n_cells, 2, 8)[c, 1, block] = INF
        dims = list(range(32, 64))
    out = P.attend(q, s, p)
    no_errors()
    sees = p >= first
    assert sees.any() and out[sees][:, 8:].isnan().all()
    assert torch.equal(out[:, :8], clean[:, :8])
    rest = [d for d in range(D) if d not in dims]
    assert torch.equal(out[~sees][:, 8:][..., rest], clean[~sees][:, 8:][..., rest])
    hit = out[~sees][:, 8:][..., dims]
    assert torch.all(hit == INF if kv == "f16" else hit.isnan())
