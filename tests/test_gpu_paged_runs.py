"""paged_attn of calls whose sequences do not all have the same number of tokens, or
that touch few of the lists: single tokens, drafted ones and chunks of prompts side by
side, each checked against the definition in 64 bits; and neighbouring tokens share
their reading whatever the number of lists is."""
import numpy as np
import pytest
import torch

from paged_util import Paged, no_errors
from sparse_attention_long_qsa_gb300 import qsa

pytestmark = pytest.mark.gpu
KV = ["f16", "q8_0", "q4_0"]


def bound(P, T, much):
    """max_len with which reading the rows of T tokens one by one takes `much` bytes: with 1.25e9 of T lists or more a call
    goes to a kernel for single tokens and one for groups, with 2e10 of a few lists to one for groups of 16 and one of 32."""
    row = {"f16": 512, "q8_0": 272, "q4_0": 144}[P.kv]
    return max(max(P.lens), int(1.05 * much / (2 * P.G * row * T)))


def runs(P, spec):
    """Tokens of (sequence, number) in order: each run the last positions of its sequence."""
    seqs = [s for s, n in spec for _ in range(n)]
    poss = [P.lens[s] - n + i for s, n in spec for i in range(n)]
    return P.tokens(seqs, poss)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window,sinks,much", [(0, 0, 0), (77, 3, 0), (0, 0, 1.25e9), (2 ** 31 - 1, 5, 1.25e9), (0, 0, 2e10)])
@pytest.mark.parametrize("spec", [[(3, 1), (0, 5)], [(0, 5), (3, 1)], [(2, 2), (1, 1), (0, 3)], [(0, 40), (1, 1), (2, 2), (3, 16), (4, 17)],
                                  [(i % 5, 1) for i in range(30)], [(0, 64)], [(4, 2), (0, 2), (1, 2)], [(1, 1), (2, 33), (3, 1), (0, 3)]],
                         ids=lambda s: "-".join(str(n) for _, n in s[:6]))
@pytest.mark.parametrize("lists", [5, 300])
def test_runs_of_any_lengths(kv, window, sinks, much, spec, lists):
    P = Paged(kv, (900, 333, 1200, 64, 500) + (1,) * (lists - 5), seed=len(spec))
    q, s, p = runs(P, spec)
    m = bound(P, q.shape[0], much)
    out = P.attend(q, s, p, window, sinks, max_len=m)
    no_errors()
    P.check(out, q, s, p, window, sinks)
    assert torch.equal(out, P.attend(q, s, p, window, sinks, max_len=m, fill=0))   # workspace of other contents


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("much", [0, 1.25e9, 2e10])
@pytest.mark.parametrize("singles,chunk", [(63, 50), (100, 3), (200, 130), (60, 500)])
def test_a_chunk_among_single_tokens(kv, singles, chunk, much):
    """More tokens than parts, too; the chunk in the middle, and a run of two."""
    rng = np.random.default_rng(singles)
    lens = [int(x) for x in rng.integers(1, 400, singles)] + [1500, 70]
    P = Paged(kv, lens, seed=singles)
    half = singles // 2
    q, s, p = runs(P, [(i, 1) for i in range(half)] + [(singles, chunk)] + [(i, 1) for i in range(half, singles)] + [(singles + 1, 2)])
    out = P.attend(q, s, p, max_len=bound(P, q.shape[0], much))
    no_errors()
    P.check(out, q, s, p, only=set(range(half)) | set(range(half, half + chunk, 13)) | set(range(half + chunk, q.shape[0])))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("G,r,lists", [(1, 1, 300), (3, 8, 300), (8, 2, 300), (3, 4, 5), (64, 4, 300)])
def test_heads_of_mixed_calls(kv, G, r, lists):
    P = Paged(kv, (500, 90, 333, 64, 200) + (1,) * (lists - 5), G=G, r=r, seed=G)
    q, s, p = runs(P, [(0, 40), (1, 1), (2, 2), (3, 16), (4, 1), (1, 3)])
    for much in (1.25e9, 2e10):
        out = P.attend(q, s, p, max_len=bound(P, q.shape[0], much))
        no_errors()
        P.check(out, q, s, p)


def test_a_window_over_long_lists():
    P = Paged("f16", (20_000,) + (13_000,) * 70, seed=4)
    q, s, p = runs(P, [(1, 1), (0, 50), (2, 2), (3, 1), (4, 1), (0, 1), (5, 3), (6, 1), (7, 1), (8, 1), (9, 1), (10, 1)])
    out = P.attend(q, s, p, 12_000, 4)
    no_errors()
    P.check(out, q, s, p, 12_000, 4, only={0, 1, 20, 50, 51, 52, 53, 54, 56, 60, 63})


@pytest.mark.parametrize("lists", [3, 400, 5000])
def test_runs_across_launches(lists):
    """4,096 tokens a launch: a chunk that ends in the first with one token of the second, singles behind it.  Groups of 32, of
    16 and one by one on average."""
    P = Paged("f16", (4300, 40, 50) + (1,) * (lists - 3), seed=3)
    q, s, p = runs(P, [(1, 1), (0, 4094), (2, 2), (1, 1), (2, 1), (0, 5)])
    out = P.attend(q, s, p, 90, 2)
    P.check(out, q, s, p, 90, 2, only={0, 1, 50, 4094, 4095, 4096, 4097, 4098, 4099, 4103})
    out = P.attend(q, s, p, 90, 2, max_len=2 ** 20)
    P.check(out, q, s, p, 90, 2, only={0, 1, 50, 4094, 4095, 4096, 4097, 4098, 4099, 4103})
    out = P.attend(q, s, p, 2 ** 31 - 1, 2, max_len=2 ** 20)
    P.check(out, q, s, p, 2 ** 31 - 1, 2, only={0, 1, 50, 4094, 4095, 4096, 4097, 4098, 4099, 4103})
    out = P.attend(q, s, p, 90, 2)
    no_errors()
    P.check(out, q, s, p, 90, 2, only={0, 1, 50, 4094, 4095, 4096, 4097, 4098, 4099, 4103})


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("spec", [[(0, 5), (1, 1), (2, 2), (3, 1)], [(1, 1), (0, 70), (2, 1), (3, 3)], [(i % 4, 1) for i in range(90)]],
                         ids=["few", "over 64", "single"])
@pytest.mark.parametrize("lists", [4, 100])
def test_block_weights_of_mixed_runs(kv, spec, lists):
    P = Paged(kv, (1000, 333, 64, 500) + (1,) * (lists - 4), seed=7)
    q, s, p = runs(P, spec)
    w = torch.rand(P.slots.numel(), device="cuda")
    for window, m in ((400, None), (0, bound(P, min(q.shape[0], 26), 1.25e9))):   # (a launch takes 64 tokens, the last 26)
        before = w.clone()
        out = P.attend(q, s, p, window, 2, weight=w, max_len=m)
        no_errors()
        P.check(out, q, s, p, window, 2, weight=w, before=before)


def test_tokens_of_no_sequence_among_runs():
    P = Paged("q8_0", (300, 200, 100), seed=8)
    q, s, p = runs(P, [(0, 4), (1, 1), (2, 3), (0, 1), (1, 20)])
    s[2], p[6], s[8] = 3, -1, -5
    for m in (300, bound(P, 29, 1.25e9), bound(P, 29, 2e10)):
        out = P.attend(q, s, p, max_len=m)
        torch.cuda.synchronize()
        assert qsa.debug_check() == (-6, 16)
        assert torch.all(out[[2, 6, 8]] == 0)
        P.check(out, q, s, p, only=set(range(29)) - {2, 6, 8})


def test_mixed_runs_in_two_graphs():
    P = Paged("f16", (900, 300, 50) + (1,) * 60, seed=9)
    calls = [runs(P, [(0, 40), (1, 1), (2, 1)]), runs(P, [(1, 1), (2, 1), (0, 1)])]   # both kinds; only one
    n, m = max(q.shape[0] for q, _, _ in calls), bound(P, 3, 1.25e9)
    ws = torch.empty(qsa.paged_attn_workspace_size(P.cfg, n, m, False), dtype=torch.uint8, device="cuda")
    want = [P.attend(*c, max_len=m) for c in calls]
    outs = [torch.empty_like(x) for x in want]
    side, graphs = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, o in zip(calls, outs):
            P.attend(*c, out=o, ws=ws, max_len=m)
        side.synchronize()
    for c, o in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            P.attend(*c, out=o, ws=ws, max_len=m)
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    no_errors()


def _us(P, q, s, p):
    out = torch.empty_like(q, dtype=torch.float32)
    ws = torch.empty(qsa.paged_attn_workspace_size(P.cfg, q.shape[0], max(P.lens), False), dtype=torch.uint8, device="cuda")
    best = float("inf")
    for _ in range(5):
        P.attend(q, s, p, ws=ws, out=out)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            P.attend(q, s, p, ws=ws, out=out)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 5 * 1e3)
    no_errors()
    return best


@pytest.mark.parametrize("kv,n,T", [("q8_0", 250_000, 5), ("f16", 30_000, 64), ("f16", 30_000, 512)])
def test_neighbours_share_their_reading_among_many_lists(kv, n, T):
    """Tokens of one sequence take about as long beside 63 short lists, or beside 63 single tokens of their sequences, as
    alone; one by one they would read the rows T times, in groups of 16 512 tokens 32 times in place of 16.  (The other
    launch, and the short sequences, take some microseconds.)"""
    alone, among = Paged(kv, (n,), seed=1), Paged(kv, (n,) + (40,) * 63, seed=1)
    one = _us(alone, *runs(alone, [(0, T)]))
    many = _us(among, *runs(among, [(0, T)]))
    mixed = _us(among, *runs(among, [(i, 1) for i in range(1, 64)] + [(0, T)]))
    assert many <= 1.25 * one + 12, (one, many, mixed)
    assert mixed <= 1.25 * one + 40, (one, many, mixed)
