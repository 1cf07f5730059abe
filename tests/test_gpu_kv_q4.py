"""The q4_0 cache: appends and reads against the oracle bit for bit, attention
over it against the oracle in 64 bits, and the whole step.

Attention tolerance 2e-5 of a row's largest value, derived: codes, queries and
their products are exact, so a cell's score is off by the rounding of some 270
fp32 additions, each at most 2^-23 of a block's running sum.  For N(0,1) rows
that sum, scaled, is at most 3.4 (32 x 0.8 x 7.5 code units x d = 0.28 / 16), so
four standard deviations of the score error are 4 x sqrt(270) x 2^-23 x 3.4 /
sqrt(3) = 1.6e-5, which is also the relative error of that cell's probability;
exp2f and the split of p * d_V into two halves add 2^-21.  The errors of
different cells are independent, as their values are, so the sum's relative
error is no larger than a single cell's.  Rows whose cells' values cancel have
no such bound and are not used."""
import numpy as np
import pytest
import torch

from oracle import qsa_oracle as O
from qsa_workload import default_cfg, make_workload, quantize_q4_0
from sparse_attention_long_qsa_gb300 import qsa
from sparse_attention_long_qsa_gb300.layer import QSALayer, append_rows, step_inputs

from gpu_util import (Runner, assert_no_device_errors, check_pooled, max_rel, run_lists, to_np)

pytestmark = pytest.mark.gpu
TOL = 2e-5


def _cache(n, G, seed, scale=1.0, zero_blocks=False):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((n, G, 256)) * scale).astype(np.float16).astype(np.float32)
    if zero_blocks:
        x.reshape(n, G, 8, 32)[rng.random((n, G, 8)) < 0.3] = 0
    codes, d = quantize_q4_0(x)
    return np.concatenate([codes.reshape(-1), d.reshape(-1).view(np.uint8)])


class _Case:
    """A bare q4_0 cache with explicit cell lists."""

    def __init__(self, n=3000, G=2, top_k=2048, seed=0, **kw):
        self.cfg = default_cfg(kv_type="q4_0", n_kv_heads=G, n_q_heads=8 * G, top_k=top_k)
        self.c = qsa.config_from_dict(self.cfg)
        self.c.kv_type = qsa.QSA_KV_Q4_0
        self.n = n
        self.kc, self.vc = _cache(n, G, seed, **kw), _cache(n, G, seed + 1, **kw)
        self.k, self.v = (torch.from_numpy(x).cuda() for x in (self.kc, self.vc))
        self.pitch = qsa.cells_per_token(self.c)

    def run(self, lists, q, counts=None, stream=None):
        T = len(lists)
        cells = np.full((T, self.pitch), -1, dtype=np.int32)
        count = np.zeros(T, dtype=np.int32)
        for t, c in enumerate(lists):
            cells[t, :len(c)] = c
            count[t] = len(c) if counts is None else counts[t]
        out = torch.full((T, self.cfg["n_q_heads"], 256), float("nan"), device="cuda")
        qsa.sparse_attn(self.c, torch.from_numpy(q).cuda(), self.k, self.v, self.n, torch.from_numpy(cells).cuda(),
                        torch.from_numpy(count).cuda(), out, None, stream=stream)
        torch.cuda.synchronize()
        return to_np(out)

    def ref(self, lists, q):
        return np.stack([O.attend(self.cfg, q[t], self.kc, self.vc, self.n, np.asarray(c))
                         for t, c in enumerate(lists)])


def _q(T, H, seed):
    return np.random.default_rng(seed).standard_normal((T, H, 256)).astype(np.float16)


@pytest.mark.parametrize("count", [1, 2, 15, 16, 17, 63, 64, 65, 129, 1000, 2047, 2048, 2051])
def test_every_list_length(count):
    C = _Case(seed=count)
    rng = np.random.default_rng(count)
    lists = [rng.permutation(C.n)[:count] for _ in range(2)]
    q = _q(2, 16, count)
    out = C.run(lists, q)
    assert max_rel(out, C.ref(lists, q)) <= TOL
    assert_no_device_errors()


@pytest.mark.parametrize("T", [1, 3, 5, 16, 40, 80, 200])
def test_token_counts_and_mixed_lengths(T):
    """Every cluster size; lists of different lengths in one call, some empty."""
    C = _Case(n=4000, seed=T)
    rng = np.random.default_rng(T)
    lists = [rng.permutation(C.n)[:int(n)] for n in rng.integers(0, 2052, T)]
    if T > 2:
        lists[1] = lists[1][:0]
    q = _q(T, 16, T)
    out = C.run(lists, q)
    ref = C.ref(lists, q)
    for t in range(T):
        if len(lists[t]) == 0:
            assert np.all(out[t] == 0)
        else:
            assert max_rel(out[t], ref[t]) <= TOL, (t, len(lists[t]))
    np.testing.assert_array_equal(out, C.run(lists, q))   # the same bits again


@pytest.mark.parametrize("G,top_k", [(1, 2048), (3, 16), (2, 8), (8, 256), (2, 4096)])
def test_head_counts_and_budgets(G, top_k):
    C = _Case(n=max(6000, 2 * top_k), G=G, top_k=top_k, seed=G)
    rng = np.random.default_rng(G)
    lists = [rng.permutation(C.n)[:C.pitch - i] for i in range(3)]
    q = _q(3, 8 * G, G)
    assert max_rel(C.run(lists, q), C.ref(lists, q)) <= TOL


@pytest.mark.parametrize("scale", [3e-6, 1e-3, 1.0, 300.0])
def test_value_magnitudes(scale):
    """Scales from fp16's subnormals up: the weights' common exponent follows
    them.  Queries shrink as keys grow, so that the scores stay of order one."""
    C = _Case(n=1200, seed=7, scale=scale, zero_blocks=True)
    rng = np.random.default_rng(8)
    lists = [rng.permutation(C.n)[:900], rng.permutation(C.n)[:3]]
    q = (_q(2, 16, 9).astype(np.float32) / max(scale, 1.0)).astype(np.float16)
    assert max_rel(C.run(lists, q), C.ref(lists, q)) <= TOL


def test_growing_scales_and_scores_along_the_list():
    """Cells in order of rising value scale and of rising score: the running
    maximum and the exponent move many times."""
    n = 2048
    rng = np.random.default_rng(11)
    grow = np.exp(np.linspace(-8, 5, n))[:, None, None]
    C = _Case(n=n, seed=12)
    v = (rng.standard_normal((n, 2, 256)) * grow).astype(np.float16).astype(np.float32)
    codes, d = quantize_q4_0(v)
    C.vc = np.concatenate([codes.reshape(-1), d.reshape(-1).view(np.uint8)])
    C.v = torch.from_numpy(C.vc).cuda()
    q = _q(1, 16, 13)
    score = O.kv_rows(C.cfg, C.kc, n, range(n), 0) @ q[0, 0].astype(np.float64)
    for order in (np.arange(n), np.argsort(score), np.argsort(-score)):
        assert max_rel(C.run([order], q), C.ref([order], q)) <= TOL


def test_one_dominant_cell_and_equal_cells():
    C = _Case(n=500, seed=21)
    q = _q(1, 16, 22) * np.float16(30)
    lists = [np.arange(500)]
    # scores reach +-200: their error grows with the queries' factor of 30
    assert max_rel(C.run(lists, q), C.ref(lists, q)) <= 30 * TOL
    same = [np.full(777, 13)]
    assert max_rel(C.run(same, _q(1, 16, 23)), C.ref(same, _q(1, 16, 23))) <= TOL


def test_bad_cells_are_masked_and_flagged():
    C = _Case(n=3000, seed=31)
    rng = np.random.default_rng(32)
    good = rng.permutation(C.n)[:700]
    q = _q(3, 16, 33)
    bad = good.astype(np.int64).copy()
    bad[::7] = C.n + 5
    bad[3::7] = -4
    keep = good[(np.arange(700) % 7 != 0) & (np.arange(700) % 7 != 3)]
    qsa.debug_check()
    out = C.run([bad, good, np.full(40, C.n)], q)
    st, flags = qsa.debug_check()
    assert st == -6 and flags == 2
    assert max_rel(out[:2], C.ref([keep, good], q[:2])) <= TOL
    assert np.all(out[2] == 0)
    # a count outside the list is clamped
    out = C.run([good, good], q[:2], counts=[-5, 10**6])
    st, flags = qsa.debug_check()      # the entries past the list are -1
    assert np.all(out[0] == 0) and st == -6 and flags == 2
    assert max_rel(out[1], C.ref([good], q[:1] * 0 + q[1:2])[0]) <= TOL


def test_infinities_and_nan_outside_the_list_do_not_reach_it():
    C = _Case(n=1000, seed=41)
    nq = C.n * 2 * 128
    for x in (C.kc, C.vc):
        x[nq:].view(np.float16).reshape(C.n, 16)[500:] = np.inf
        x[nq:].view(np.float16).reshape(C.n, 16)[0] = np.nan
    C.k, C.v = (torch.from_numpy(x).cuda() for x in (C.kc, C.vc))
    lists = [np.arange(1, 500), np.array([7]), np.array([], dtype=np.int64)]
    q = _q(3, 16, 42)
    out = C.run(lists, q)
    assert max_rel(out[:2], C.ref(lists[:2], q)) <= TOL and np.all(out[2] == 0)
    assert np.all(np.isnan(C.run([np.arange(495, 510)], q[:1])))


def test_an_infinite_value_scale_spoils_its_own_dims_only():
    C = _Case(n=1000, seed=43)
    nq = C.n * 2 * 128
    d = C.vc[nq:].view(np.float16).reshape(C.n, 2, 8)
    keep = d[[100, 200], 0, [3, 5]].copy()
    q = _q(1, 16, 44)
    lists = [np.arange(900)]
    ref = C.ref(lists, q)
    d[100, 0, 3], d[200, 0, 5] = np.inf, np.nan
    C.v = torch.from_numpy(C.vc).cuda()
    out = C.run(lists, q)
    assert np.all(np.isnan(out[0, :8, 96:128])) and np.all(np.isnan(out[0, :8, 160:192]))
    assert np.all(np.isfinite(np.delete(out[0, :8], np.r_[96:128, 160:192], axis=1))) and np.all(np.isfinite(out[0, 8:]))
    d[[100, 200], 0, [3, 5]] = keep
    out[np.isnan(out)] = ref[np.isnan(out)]
    assert max_rel(out, ref) <= TOL


def test_append_and_read_match_the_oracle_bit_for_bit():
    for kw in (dict(n_seq=1, prompt_len=301, n_steps=3), dict(n_seq=3, prompt_len=[101, 202, 303], n_steps=2,
               tokens_per_step=5, shuffled=True), dict(n_seq=1, prompt_len=50, n_steps=1, tokens_per_step=96)):
        wl = make_workload(seed=51, kv_type="q4_0", **kw)
        L = QSALayer.from_workload(wl, 0)
        L.warm(torch.from_numpy(wl.prompt_dirty()).cuda())
        new = np.unique(np.concatenate([st.cells for st in wl.steps]))
        for x in (L.k_cache, L.v_cache):   # poison the new cells
            x[:wl.n_cells * 256].view(wl.n_cells, 256)[new] = 0xAB
            x[wl.n_cells * 256:].view(wl.n_cells, 32)[new] = 0xCD
        for st in wl.steps:
            i = step_inputs(st, new_cells=True)
            L.kv_append(i["tok_seq"], i["tok_pos"], i["cells"], i["k_new"], i["v_new"], i["idx_new"], pool=True)
        np.testing.assert_array_equal(to_np(L.k_cache), wl.k_cache)   # the generator's own encoding
        np.testing.assert_array_equal(to_np(L.v_cache), wl.v_cache)
        kc, vc = np.zeros_like(wl.k_cache), np.zeros_like(wl.v_cache)
        tbl = wl.blk_cells_state(0)
        for st in wl.steps:
            kc, vc, _, tbl, _ = O.kv_append(wl.cfg, st.tok_seq, st.tok_pos, st.cells, st.k_new, st.v_new, st.idx_new,
                                            kc, vc, wl.idx_k, wl.n_cells, tbl, wl.seq_blk_off, wl.seq_blk_slots, 1024)
        np.testing.assert_array_equal(to_np(L.blk_cells), tbl)
        c = torch.from_numpy(new.astype(np.int32)).cuda()
        k, v = L.kv_read(c)
        for g in range(2):
            np.testing.assert_array_equal(to_np(k)[:, g], O.kv_rows(wl.cfg, kc, wl.n_cells, new, g).astype(np.float16))
            np.testing.assert_array_equal(to_np(v)[:, g], O.kv_rows(wl.cfg, vc, wl.n_cells, new, g).astype(np.float16))
    assert_no_device_errors()


def test_append_of_special_blocks():
    """Zeros, ties of magnitude, subnormals, the largest halves, infinities and
    NaN in an encoded block."""
    wl = make_workload(n_seq=1, prompt_len=40, n_steps=1, seed=52, kv_type="q4_0")
    st = wl.steps[0]
    rows = np.random.default_rng(1).standard_normal((2, 256)).astype(np.float16)
    rows[0, :32] = 0
    rows[0, 32:64] = np.where(np.arange(32) % 2, -1.5, 1.5)
    rows[0, 64:96] = np.arange(32) * 6e-8
    rows[0, 96:128] = 65504 * np.linspace(-1, 1, 32)
    rows[0, 128:160] = -np.arange(32)
    k_new = rows[None].copy()
    v_new = k_new.copy()
    v_new[0, 1, 5] = np.inf
    v_new[0, 1, 40] = np.nan
    L = QSALayer.from_workload(wl, 0)
    i = step_inputs(st, new_cells=True)
    L.kv_append(i["tok_seq"], i["tok_pos"], i["cells"], torch.from_numpy(k_new).cuda(), torch.from_numpy(v_new).cuda(),
                i["idx_new"])
    kc = np.zeros_like(wl.k_cache)
    kc, _, _, _, _ = O.kv_append(wl.cfg, st.tok_seq, st.tok_pos, st.cells, k_new, k_new, st.idx_new, kc, kc.copy(),
                                 wl.idx_k, wl.n_cells, wl.blk_cells_state(0), wl.seq_blk_off, wl.seq_blk_slots, 4)
    k, v = (to_np(x)[0] for x in L.kv_read(i["cells"]))
    for g in range(2):
        np.testing.assert_array_equal(k[g], O.kv_rows(wl.cfg, kc, wl.n_cells, st.cells, g)[0].astype(np.float16))
    assert np.isposinf(v[1, 5]) and np.all(np.isnan(np.delete(v[1, :32], 5))) and np.all(np.isnan(v[1, 32:64]))
    np.testing.assert_array_equal(v[1, 64:], k[1, 64:])


@pytest.mark.parametrize("kv_type", ["f16", "q8_0", "q4_0"])
def test_read_skips_and_flags(kv_type):
    wl = make_workload(n_seq=1, prompt_len=100, n_steps=1, seed=53, kv_type=kv_type)
    L = QSALayer.from_workload(wl, 0)
    cells = np.array([5, -1, 99, 10_000, 0, 5], dtype=np.int32)
    out = [torch.full((6, 2, 256), 3.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    qsa.debug_check()
    qsa.kv_read(L.cfg, torch.from_numpy(cells).cuda(), L.k_cache, L.v_cache, L.n_cells, *out)
    st, flags = qsa.debug_check()
    assert st == -6 and flags == 2
    for got, cache in zip(out, (wl.k_cache, wl.v_cache)):
        got = to_np(got)
        for i, c in enumerate(cells):
            for g in range(2):
                want = O.kv_rows(wl.cfg, cache, wl.n_cells, [c], g)[0].astype(np.float16) if 0 <= c < 100 else 3.0
                np.testing.assert_array_equal(got[i, g], want if 0 <= c < 100 else np.full(256, 3.0, np.float16))


@pytest.mark.parametrize("kw", [dict(n_seq=1, prompt_len=3001, n_steps=2),
                                dict(n_seq=2, prompt_len=[9001, 700], n_steps=2, tokens_per_step=6, shuffled=True)])
@pytest.mark.parametrize("mode", ["calls", "index_attn", "in_cluster", "full"])
def test_whole_step(kw, mode):
    wl = make_workload(seed=61, kv_type="q4_0", **kw)
    run = Runner(wl, mode="calls" if mode == "full" else mode)
    L = run.layer
    for i, st in enumerate(wl.steps):
        if mode == "full":
            out = to_np(L.full_step(**step_inputs(st, new_cells=True)))
            cells, count = to_np(L.cells), to_np(L.count)
        else:
            res = run.run_step(i)
            out, cells, count = res["out"], res["cells"], res["count"]
        for t in range(len(st.tok_pos)):
            ref = O.attend(wl.cfg, st.q[t], wl.k_cache, wl.v_cache, wl.n_cells, cells[t, :count[t]])
            assert max_rel(out[t], ref) <= TOL
        sel = to_np(L.pooled)[wl.steps[i].dirty[wl.steps[i].dirty >= 0]]
        assert np.all(np.isfinite(sel))
    assert_no_device_errors()


def test_streams_and_captured_graphs():
    """Two captured calls replayed in turn and an eager call on another stream
    give the eager results."""
    C = _Case(n=2500, seed=71)
    rng = np.random.default_rng(72)
    lists = [[rng.permutation(C.n)[:n] for n in ns] for ns in ((2051, 5), (900,))]
    qs = [_q(2, 16, 73), _q(1, 16, 74)]
    want = [C.run(l, q) for l, q in zip(lists, qs)]
    s = torch.cuda.Stream()
    np.testing.assert_array_equal(C.run(lists[0], qs[0], stream=s), want[0])
    graphs, outs, keep = [], [], []
    for l, q in zip(lists, qs):
        cells = torch.full((len(l), C.pitch), -1, dtype=torch.int32)
        for t, c in enumerate(l):
            cells[t, :len(c)] = torch.from_numpy(c.astype(np.int32))
        args = (torch.from_numpy(q).cuda(), C.k, C.v, C.n, cells.cuda(),
                torch.tensor([len(c) for c in l], dtype=torch.int32, device="cuda"))
        out = torch.zeros((len(l), 16, 256), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qsa.sparse_attn(C.c, *args, out, None)
        graphs.append(g), outs.append(out), keep.append(args)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        np.testing.assert_array_equal(to_np(o), w)


def test_offsets_past_32_bits():
    """A cell whose codes lie past 2^32 bytes (n_cells * 256 bytes of codes)."""
    n = (1 << 24) + 40_000
    cfg = qsa.config(kv_type="q4_0")
    rows = _cache(64, 2, 81)
    where = torch.cat([torch.arange(8), torch.arange(n - 56, n)])
    cache = torch.zeros(n * 288, dtype=torch.uint8, device="cuda")
    cache[:n * 256].view(n, 256)[where.cuda()] = torch.from_numpy(rows[:64 * 256]).cuda().view(64, 256)
    cache[n * 256:].view(n, 32)[where.cuda()] = torch.from_numpy(rows[64 * 256:]).cuda().view(64, 32)
    q = _q(1, 16, 82)
    cells = torch.full((1, 2051), -1, dtype=torch.int32)
    cells[0, :64] = where.int()
    out = torch.empty((1, 16, 256), device="cuda")
    qsa.sparse_attn(cfg, torch.from_numpy(q).cuda(), cache, cache, n, cells.cuda(),
                    torch.tensor([64], dtype=torch.int32, device="cuda"), out, None)
    ref = O.attend(default_cfg(kv_type="q4_0"), q[0], rows, rows, 64, np.arange(64))
    assert max_rel(to_np(out)[0], ref) <= TOL
    k, v = (torch.zeros((64, 2, 256), dtype=torch.float16, device="cuda") for _ in range(2))
    qsa.kv_read(cfg, where.int().cuda(), cache, cache, n, k, v)
    np.testing.assert_array_equal(to_np(k)[:, 1], O.kv_rows(default_cfg(kv_type="q4_0"), rows, 64, range(64), 1)
                                  .astype(np.float16))
    # copies between the ends
    qsa.cells_copy(cfg, torch.tensor([n - 1], dtype=torch.int32, device="cuda"),
                   torch.tensor([100], dtype=torch.int32, device="cuda"), cache, cache, None, n)
    assert torch.equal(cache[100 * 256:101 * 256], cache[(n - 1) * 256:n * 256])
    assert torch.equal(cache[n * 256 + 3200:n * 256 + 3232], cache[n * 288 - 32:])
    assert_no_device_errors()
