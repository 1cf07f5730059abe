"""paged_attn where a few cells take nearly all of the weight and hardly any of the
values (attention sinks): the output is the sum of the small weights, which have to
keep their bits.

Scores are `places` binary places apart: a sink's, and the others', which spread by
one place.  A weight is relative to the largest of the cells that are read together
(at most 128): 2^15 or more there, and its second part ends at 2^-24, half of which
is lost at most, 2^-24 / sqrt(12) on average.  24 places below, a weight is 2^-9, and the
loss 2^-15 / sqrt(12) = 8.8e-6 of it (5.5e-6 of the root mean square of weights that
spread by a place); where other cells are read besides, it is less.  With what
paged_util.py derives for the rest that stays within the 1e-5 of the norm that
Paged.check asks for."""
import pytest
import torch

from paged_util import D, Paged, encode, no_errors

pytestmark = pytest.mark.gpu


def sunk(kv, n, T, places, sinks, v_sink, seed):
    """A cache whose cells `sinks` score `places` above the others for every token and head, their values times v_sink."""
    P = Paged(kv, (n,), seed=seed)
    k = torch.randn((P.n_cells, 2, D), generator=P.g, device="cuda") * 0.693
    v = torch.randn((P.n_cells, 2, D), generator=P.g, device="cuda")
    k[:, :, :32] = 0                                         # (a block of its own, so that codes hold both)
    _, cells = P.visible(0, n - 1)
    for j in sinks:
        k[cells[j]] = 0
        k[cells[j], :, 0] = places / 1.4427
        v[cells[j]] *= v_sink
    P.k, P.K = encode(kv, k)
    P.v, P.V = encode(kv, v)
    q, s, p = P.tokens([0] * T, list(range(n - T, n)), q_mul=1.0)
    q[:, :, 0] = 16
    return P, q, s, p


@pytest.mark.parametrize("kv", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("places", [14, 18, 20, 24])
@pytest.mark.parametrize("n,T", [(3_000, 1), (3_000, 5), (64, 5), (3_000, 40), (40_000, 5), (40_000, 33)])
def test_small_weights_below_a_sink(kv, places, n, T):
    P, q, s, p = sunk(kv, n, T, places, [0], 0.0, seed=n + places)
    out = P.attend(q, s, p)
    no_errors()
    P.check(out, q, s, p, only={0, T // 2, T - 1})


@pytest.mark.parametrize("kv", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("places,v_sink", [(20, 0.01), (40, 0.0), (70, 0.0)])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_sinks_first_and_in_the_middle(kv, places, v_sink, T):
    """Four first sinks and one further on.  Beyond 24 places what is read with a sink loses bits, of 20,000 cells two
    tiles: where nothing else has weight either the others keep theirs."""
    n = 20_000
    P, q, s, p = sunk(kv, n, T, places, [0, 1, 2, 3, 11_111], v_sink, seed=places)
    if places > 24:
        # the cells read with a sink (128 at most, by how the tiles lie) count for nothing
        _, cells = P.visible(0, n - 1)
        gone = torch.cat([cells[:160], cells[11_111 - 160:11_111 + 160]])
        for raw, val in ((P.v, P.V),):
            if kv == "f16":
                raw[gone] = 0
            else:
                codes = P.n_cells * 2 * (256 if kv == "q8_0" else 128)
                raw[codes:].view(torch.float16).view(P.n_cells, 2, 8)[gone] = 0
            val[gone] = 0
    out = P.attend(q, s, p)
    no_errors()
    P.check(out, q, s, p, only={0, T - 1})


@pytest.mark.parametrize("kv", ["f16", "q8_0"])
def test_block_weights_of_small_weights(kv):
    """The weights of blocks beside a sink's, each to its own bits."""
    P, q, s, p = sunk(kv, 5_000, 5, 20, [0, 1], 0.0, seed=3)
    w = torch.zeros(P.slots.numel(), device="cuda")
    before = w.clone()
    out = P.attend(q, s, p, weight=w)
    no_errors()
    P.check(out, q, s, p, weight=w, before=before)
