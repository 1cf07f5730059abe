"""Cells and blocks of a cache: qsa_cells_copy, qsa_seq_fork and
qsa_cache_sweep against plain NumPy, all integers (or bytes) exact; and a run
of the calls together as a server makes them."""
import numpy as np
import pytest
import torch

from oracle import qsa_oracle as O
from qsa_workload import default_cfg, make_workload
from sparse_attention_long_qsa_gb300 import qsa
from sparse_attention_long_qsa_gb300.layer import QSALayer, step_inputs

from gpu_util import assert_no_device_errors, max_rel, to_np

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


# ------------------------------------------------------------ cells_copy
@pytest.mark.parametrize("kv_type", ["f16", "q8_0", "q4_0"])
@pytest.mark.parametrize("G", [1, 2, 5])
@pytest.mark.parametrize("n_pairs", [0, 1, 7, 300])
def test_copy_moves_whole_cells(kv_type, G, n_pairs):
    cfg = qsa.config(kv_type=kv_type, n_kv_heads=G, n_q_heads=8 * G)
    n = 800
    rng = np.random.default_rng(G + n_pairs)
    caches = [torch.from_numpy(rng.integers(0, 256, qsa.cache_bytes(cfg, n), dtype=np.uint8)).cuda() for _ in range(2)]
    idx = torch.from_numpy(rng.integers(0, 60000, (n, 128)).astype(np.uint16).view(np.float16)).cuda()
    at = rng.permutation(n)[:2 * n_pairs]
    src, dst = at[:n_pairs].copy(), at[n_pairs:].copy()
    if n_pairs > 6:
        src[2], dst[4], dst[5] = -1, -3, src[5]          # skipped; onto itself
    want = [to_np(c).copy() for c in caches]
    widx = to_np(idx).copy().view(np.uint16)
    codes = {"f16": 512, "q8_0": 256, "q4_0": 128}[kv_type] * G
    scales = 0 if kv_type == "f16" else 16 * G
    for s, d in zip(src, dst):
        if s < 0 or d < 0:
            continue
        for w in want:
            a, b = w[:n * codes].reshape(n, codes), w[n * codes:].reshape(n, scales) if scales else None
            a[d] = a[s]
            if scales:
                b[d] = b[s]
        widx[d] = widx[s]
    before = idx.clone()
    qsa.cells_copy(cfg, _i32(src), _i32(dst), caches[0], caches[1], None, n)
    assert torch.equal(idx.view(torch.int16), before.view(torch.int16))   # no indexer keys given: none moved
    qsa.cells_copy(cfg, _i32(src), _i32(dst), caches[0], caches[1], idx, n)
    for c, w in zip(caches, want):
        np.testing.assert_array_equal(to_np(c), w)
    np.testing.assert_array_equal(to_np(idx).view(np.uint16), widx)
    assert_no_device_errors()


def test_copy_device_count_and_flags():
    cfg, n = qsa.config(), 64
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((n, 2, 256), generator=g, device="cuda").half()
    v, idx = k * 2, k[:, 0, :128].contiguous()
    for count, done in ((3, 3), (0, 0), (-7, 0), (99, 8)):
        k2, v2, i2 = k.clone(), v.clone(), idx.clone()
        src, dst = torch.arange(8, dtype=torch.int32, device="cuda"), torch.arange(40, 48, dtype=torch.int32, device="cuda")
        qsa.cells_copy(cfg, src, dst, k2, v2, i2, n, n_pairs=_i32([count]))
        for got, was in ((k2, k), (v2, v), (i2, idx)):
            want = was.clone()
            want[40:40 + done] = was[:done]
            assert torch.equal(got, want)
    qsa.debug_check()
    k2 = k.clone()
    qsa.cells_copy(cfg, _i32([1, 64, 2]), _i32([50, 51, 70]), k2, v.clone(), None, n)
    st, flags = qsa.debug_check()
    assert st == -6 and flags == 2
    want = k.clone()
    want[50] = k[1]
    assert torch.equal(k2, want)


# -------------------------------------------------------------- seq_fork
def _tables(rng, lens, cap, r, spare_slots, spare_cells):
    S = len(lens)
    off = np.concatenate([[0], np.cumsum(cap)]).astype(np.int64)
    used_slots = sum(-(-int(x) // r) for x in lens)
    n_slots, n_cells = used_slots + spare_slots, sum(lens) + spare_cells
    order, cell = rng.permutation(n_slots), rng.permutation(n_cells)
    lists = rng.integers(0, n_slots, int(off[-1])).astype(np.int32)     # stale entries past each length
    table = np.full((n_slots, r), -1, dtype=np.int32)
    block = np.zeros(n_slots, dtype=np.int32)
    ks = kc = 0
    for s in range(S):
        nb = -(-int(lens[s]) // r)
        sl = order[ks:ks + nb]
        lists[off[s]:off[s] + nb] = sl
        flat = np.full(nb * r, -1)
        flat[:lens[s]] = cell[kc:kc + lens[s]]
        table[sl] = flat.reshape(nb, r)
        block[sl] = np.arange(nb)
        ks, kc = ks + nb, kc + int(lens[s])
    return off, lists, table, block, order[ks:], cell[kc:], n_cells


def _fork_ref(src, dst, n_pos, tslot, tcells, off, lists, table, block, r, skip=()):
    lists, table, block = lists.copy(), table.copy(), block.copy()
    cs, cd = np.full((len(src), r), -1, np.int32), np.full((len(src), r), -1, np.int32)
    old = lists.copy()
    for f in range(len(src)):
        if f in skip:
            continue
        nb, t = divmod(int(n_pos[f]), r)
        a, b = int(off[src[f]]), int(off[dst[f]])
        lists[b:b + nb] = old[a:a + nb]
        if t:
            cs[f, :t], cd[f, :t] = table[old[a + nb], :t], tcells[f, :t]
            table[tslot[f]] = -1
            table[tslot[f], :t] = tcells[f, :t]
            block[tslot[f]] = nb
            lists[b + nb] = tslot[f]
    return lists, table, block, cs, cd


@pytest.mark.parametrize("r", [1, 4, 8])
@pytest.mark.parametrize("lens", [[1], [9, 4003], [8, 0, 30_001], [5000] * 4])
def test_fork_matches_plain(r, lens):
    rng = np.random.default_rng(r * 100 + len(lens))
    S, F = len(lens), 3
    cap = [-(-x // r) + 5 for x in lens] + [max(lens) // r + 7] * F
    off, lists, table, block, fs, fc, n_cells = _tables(rng, lens + [0] * F, cap, r, F + 2, F * r)
    src = rng.integers(0, S, F)
    dst = S + rng.permutation(F)
    n_pos = np.array([rng.integers(0, lens[s] + 1) for s in src])
    n_pos[0] = lens[src[0]]
    tcells = fc[:F * r].reshape(F, r)
    want = _fork_ref(src, dst, n_pos, fs, tcells, off, lists, table, block, r)
    cfg = qsa.config(compress_ratio=r)
    d_lists, d_table, d_block = _i32(lists), _i32(table), _i32(block)
    cs, cd = _i32(np.full((F, r), 9)), _i32(np.full((F, r), 9))
    mb = int(n_pos.max()) // r
    qsa.seq_fork(cfg, _i32(src), _i32(dst), _i32(n_pos), _i32(fs[:F]), _i32(tcells), torch.from_numpy(off).cuda(),
                 d_lists, d_table, d_block, mb, cs, cd, n_cells)
    for got, w in zip((d_lists, d_table, d_block, cs, cd), want):
        np.testing.assert_array_equal(to_np(got), w)
    assert_no_device_errors()


def test_fork_onto_itself_gets_a_tail_of_its_own():
    rng = np.random.default_rng(3)
    off, lists, table, block, fs, fc, n_cells = _tables(rng, [2051], [600], 4, 2, 4)
    want = _fork_ref([0], [0], [2051], fs, fc[:4].reshape(1, 4), off, lists, table, block, 4)
    d = [_i32(lists), _i32(table), _i32(block), _i32(np.zeros((1, 4))), _i32(np.zeros((1, 4)))]
    qsa.seq_fork(qsa.config(), _i32([0]), _i32([0]), _i32([2051]), _i32(fs[:1]), _i32(fc[:4].reshape(1, 4)),
                 torch.from_numpy(off).cuda(), d[0], d[1], d[2], 512, d[3], d[4], n_cells)
    for got, w in zip(d, want):
        np.testing.assert_array_equal(to_np(got), w)


def test_fork_refuses_on_the_device():
    """One good fork among bad ones: only it is carried out."""
    rng = np.random.default_rng(4)
    lens = [4001, 10]
    cap = [1010, 10, 1010, 3, 1010, 1010, 1010, 1010, 1010, 1010]
    off, lists, table, block, fs, fc, n_cells = _tables(rng, lens + [0] * 8, cap, 4, 12, 40)
    src = np.array([0, 0, 7777, 0, 0, 0, 0, 1, 0])
    dst = np.array([2, 3, 4, -1, 5, 6, 7, 8, 9])
    n_pos = np.array([4001, 4001, 3, 3, -5, 4001, 4001, 4001, 4001])   # 1: no room; 7: more than the list holds
    tslot = fs[:9].copy()
    tslot[5] = 10**6
    tcells = fc[:36].reshape(9, 4).copy()
    tcells[6, 0] = n_cells
    tslot[8] = lists[1000]                                             # the source's own tail slot
    want = _fork_ref(src, dst, n_pos, tslot, tcells, off, lists, table, block, 4, skip=range(1, 9))
    d = [_i32(lists), _i32(table), _i32(block), _i32(np.zeros((9, 4))), _i32(np.zeros((9, 4)))]
    qsa.debug_check()
    args = (_i32(src), _i32(dst), _i32(n_pos), _i32(tslot), _i32(tcells), torch.from_numpy(off).cuda())
    qsa.seq_fork(qsa.config(), *args, d[0], d[1], d[2], 1000, d[3], d[4], n_cells)
    st, flags = qsa.debug_check()
    assert st == -6 and flags == (1 | 2 | 4 | 16)
    for got, w in zip(d, want):
        np.testing.assert_array_equal(to_np(got), w)
    qsa.seq_fork(qsa.config(), *args, d[0], d[1], d[2], 999, d[3], d[4], n_cells)
    st, flags = qsa.debug_check()
    assert flags & 8 and np.all(to_np(d[3]) == -1)


# ----------------------------------------------------------- cache_sweep
def _sweep_ref(lens, off, lists, table, n_cells, compact):
    n_slots, r = table.shape
    cell, slot = np.zeros(n_cells, bool), np.zeros(n_slots, bool)
    for s in range(len(lens)):
        for j in range(min(-(-max(int(lens[s]), 0) // r), int(off[s + 1] - off[s]))):
            sl = int(lists[off[s] + j])
            if not 0 <= sl < n_slots:
                continue
            slot[sl] = True
            for i in range(min(r, int(lens[s]) - j * r)):
                if 0 <= table[sl, i] < n_cells:
                    cell[table[sl, i]] = True
    held = int(cell.sum())
    new = np.where(cell, np.arange(n_cells), -1)
    src = dst = np.zeros(0, int)
    if compact:
        src = np.where(cell & (np.arange(n_cells) >= held))[0]
        dst = np.where(~cell & (np.arange(n_cells) < held))[0]
        new[src] = dst
    out = np.full_like(table, -1)
    for sl in np.where(slot)[0]:
        for i in range(r):
            if 0 <= table[sl, i] < n_cells:
                out[sl, i] = new[table[sl, i]]
    free = np.arange(held, n_cells) if compact else np.where(~cell)[0]
    return out, np.array([held, n_cells - held, int((~slot).sum()), len(src)]), new, free, np.where(~slot)[0], src, dst


def _sweep(cfg, lens, off, lists, table, n_cells, compact, in_place=False, **drop):
    n_slots = table.shape[0]
    t_in = _i32(table)
    out = t_in if in_place else _i32(np.full(table.shape, 77))
    a = dict(cell_map=_i32(np.full(n_cells, 77)), free_cells=_i32(np.full(n_cells, 77)),
             free_slots=_i32(np.full(n_slots, 77)), move_src=_i32(np.full(n_cells // 2, 77)),
             move_dst=_i32(np.full(n_cells // 2, 77)))
    a.update(drop)
    ws = torch.randint(0, 256, (qsa.cache_sweep_workspace_size(cfg, n_cells, n_slots),), dtype=torch.uint8, device="cuda")
    counts = _i32(np.zeros(4))
    qsa.cache_sweep(cfg, _i32(lens), torch.from_numpy(np.ascontiguousarray(off)).cuda(), _i32(lists), t_in, out, n_cells,
                    counts, ws, compact, **a)
    return out, counts, a


def _check_sweep(cfg, lens, off, lists, table, n_cells, compact, **kw):
    want = _sweep_ref(lens, off, lists, table, n_cells, compact)
    out, counts, a = _sweep(cfg, lens, off, lists, table, n_cells, compact, **kw)
    np.testing.assert_array_equal(to_np(out), want[0])
    np.testing.assert_array_equal(to_np(counts), want[1])
    for name, w in zip(("cell_map", "free_cells", "free_slots", "move_src", "move_dst"), want[2:]):
        if a[name] is None:
            continue
        got = to_np(a[name])
        np.testing.assert_array_equal(got[:len(w)], w, err_msg=name)
        assert np.all(got[len(w):] == 77), name      # entries past the count are left as they were


@pytest.mark.parametrize("compact", [False, True])
@pytest.mark.parametrize("r", [1, 4, 7])
@pytest.mark.parametrize("lens,keep", [([1], [1]), ([1], [0]), ([40], [40]), ([9, 5, 13], [9, 0, 6]),
                                       ([8000, 193, 20_001], [7999, -3, 12_345]), ([1000] * 40, list(range(40))),
                                       ([30_000, 10, 60_000], [0, 10, 60_000])])
def test_sweep_matches_plain(compact, r, lens, keep):
    rng = np.random.default_rng(len(lens) * 10 + r)
    cap = [-(-x // r) + int(rng.integers(0, 4)) for x in lens]
    off, lists, table, _, _, _, n_cells = _tables(rng, lens, cap, r, 5, int(rng.integers(0, 50)))
    cfg = qsa.config(compress_ratio=r, top_k=r * 512)
    _check_sweep(cfg, keep, off, lists, table, n_cells, compact)
    _check_sweep(cfg, keep, off, lists, table, n_cells, compact, in_place=True)
    if not compact:
        _check_sweep(cfg, keep, off, lists, table, n_cells, compact, cell_map=None, free_cells=None, free_slots=None,
                     move_src=None, move_dst=None)
    assert_no_device_errors()


@pytest.mark.parametrize("compact", [False, True])
def test_sweep_of_shared_blocks_and_aliased_cells(compact):
    """Blocks shared by sequences of different lengths stay for the longest
    holder; a cell named twice is one cell; holes inside rows are skipped."""
    rng = np.random.default_rng(9)
    off, lists, table, _, _, _, n_cells = _tables(rng, [4000, 0, 0, 900], [1000, 1000, 1000, 300], 4, 3, 100)
    lists[1000:2000] = lists[:1000]
    lists[2000:3000] = lists[:1000]
    table[lists[5], 2] = table[lists[900], 1]       # the same cell in two blocks
    table[lists[7], 1] = -1                         # a position without a cell
    for keep in ([0, 2001, 37, 900], [4000, 1, 0, 0], [0, 0, 0, 0]):
        _check_sweep(qsa.config(), keep, off, lists, table, n_cells, compact)
    assert_no_device_errors()


def test_sweep_flags_bad_indices():
    rng = np.random.default_rng(10)
    off, lists, table, _, _, _, n_cells = _tables(rng, [400, 300], [101, 75], 4, 3, 40)
    lists[3], lists[102] = -2, 10**6
    table[lists[9], 1] = n_cells + 3
    for compact in (False, True):
        qsa.debug_check()
        _check_sweep(qsa.config(), [10_000, 300], off, lists, table, n_cells, compact)
        st, flags = qsa.debug_check()
        assert st == -6 and flags == (1 | 2 | 4)


def test_sweep_of_one_cell_and_of_a_cache_at_the_cluster_limit():
    for n_cells in (1, 2, 4_097, 65_536, 65_537):
        off = np.array([0, n_cells], np.int64)
        lists = np.arange(n_cells)[::-1].copy()
        table = np.random.default_rng(n_cells).permutation(n_cells).reshape(n_cells, 1).astype(np.int32)
        cfg = qsa.config(compress_ratio=1, top_k=512)
        for keep in (0, 1, n_cells // 2, n_cells):
            for compact in (False, True):
                _check_sweep(cfg, [keep], off, lists, table, n_cells, compact)


def test_sweep_captured_and_replayed_on_a_used_workspace():
    """One workspace, dirty from a call of other sizes, shared by two captured
    sweeps replayed in turn."""
    rng = np.random.default_rng(14)
    cfg = qsa.config()
    ws = torch.full((qsa.cache_sweep_workspace_size(cfg, 200_000, 60_000),), 0xEE, dtype=torch.uint8, device="cuda")
    runs = []
    for lens, keep in (([5000, 90_000], [0, 70_000]), ([3000, 40], [2999, 0])):
        cap = [-(-x // 4) + 1 for x in lens]
        off, lists, table, _, _, _, n_cells = _tables(rng, lens, cap, 4, 3, 20)
        want = _sweep_ref(keep, off, lists, table, n_cells, True)
        bufs = dict(cell_map=_i32(np.zeros(n_cells)), move_src=_i32(np.zeros(n_cells // 2)),
                    move_dst=_i32(np.zeros(n_cells // 2)))
        out, counts = _i32(np.zeros(table.shape)), _i32(np.zeros(4))
        args = (_i32(keep), torch.from_numpy(off).cuda(), _i32(lists), _i32(table), out, n_cells, counts, ws)
        qsa.cache_sweep(cfg, *args, compact=True, **bufs)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qsa.cache_sweep(cfg, *args, compact=True, **bufs)
        runs.append((g, args, bufs, want, out, counts))
    for _ in range(2):
        for g, _, bufs, want, out, counts in runs:
            out.fill_(5), counts.fill_(5), bufs["cell_map"].fill_(5)
            g.replay()
            torch.cuda.synchronize()
            np.testing.assert_array_equal(to_np(out), want[0])
            np.testing.assert_array_equal(to_np(counts), want[1])
            np.testing.assert_array_equal(to_np(bufs["cell_map"]), want[2])


def test_sweep_large_cache():
    """Many tiles of cells; compaction of a random half, checked as sets."""
    rng = np.random.default_rng(12)
    n = 1_250_003
    lens = rng.multinomial(n - 7, np.full(30, 1 / 30))
    cap = -(-lens // 4)
    off, lists, table, _, _, _, n_cells = _tables(rng, list(lens), list(cap), 4, 3, 7)
    keep = np.where(rng.random(30) < 0.5, 0, lens)
    out, counts, a = _sweep(qsa.config(), keep, off, lists, table, n_cells, True)
    held = int(keep.sum())
    c = to_np(counts)
    assert c[0] == held and c[1] == n_cells - held
    m, cm = int(c[3]), to_np(a["cell_map"])
    src, dst = to_np(a["move_src"])[:m], to_np(a["move_dst"])[:m]
    live = np.zeros(n_cells, bool)
    for s in range(30):
        sl = lists[off[s]:off[s] + -(-keep[s] // 4)]
        live[table[sl].reshape(-1)[:keep[s]]] = True
    np.testing.assert_array_equal(src, np.where(live[held:])[0] + held)
    np.testing.assert_array_equal(dst, np.where(~live[:held])[0])
    want = np.where(live, np.arange(n_cells), -1)
    want[src] = dst
    np.testing.assert_array_equal(cm, want)
    o = to_np(out)
    np.testing.assert_array_equal(np.sort(o[o >= 0]), np.arange(held))


# ------------------------------------------------------- the calls together
@pytest.mark.parametrize("kv_type", ["f16", "q4_0"])
def test_a_served_run(kv_type):
    """Projections -> head norms -> steps of two sequences; one is forked and
    both go on; one finishes, the cache is compacted, and the others' next steps
    give what the oracle gives on the values read back."""
    wl = make_workload(n_seq=2, prompt_len=[2603, 801], n_steps=3, seed=91, kv_type=kv_type, shuffled=True)
    r, spare_cells, room = 4, 60, 20
    n_cells = wl.n_cells + spare_cells
    # a third sequence and room to go on; spare cells and slots at the end
    nb = [len(wl.seq_blk_slots[wl.seq_blk_off[s]:wl.seq_blk_off[s + 1]]) for s in range(2)]
    n_slots = wl.n_slots + 2 * room
    off = np.cumsum([0, nb[0] + room, nb[1] + room, nb[0] + room]).astype(np.int64)
    lists = np.zeros(off[-1], np.int32)
    for s in range(2):
        lists[off[s]:off[s] + nb[s]] = wl.seq_blk_slots[wl.seq_blk_off[s]:wl.seq_blk_off[s + 1]]
    table = np.concatenate([wl.blk_cells_state(0), np.full((2 * room, r), -1, np.int32)])
    block = np.concatenate([wl.slot_block_idx, np.zeros(2 * room, np.int32)])
    idx = np.concatenate([wl.idx_k, np.zeros((spare_cells, 128), np.float16)])
    if kv_type == "f16":
        grow = lambda x: np.concatenate([x, np.zeros((spare_cells, 2, 256), np.float16)])  # noqa: E731
    else:
        def grow(x):
            z = np.zeros(n_cells * 288, np.uint8)
            z[:wl.n_cells * 256], z[n_cells * 256:n_cells * 256 + wl.n_cells * 32] = (x[:wl.n_cells * 256],
                                                                                     x[wl.n_cells * 256:])
            return z
    L = QSALayer(wl.cfg, idx, grow(wl.k_cache), grow(wl.v_cache), n_cells, table, block, off, lists, wl.norm_w,
                 nb[0] + room, 8)
    L.warm(torch.from_numpy(wl.prompt_dirty()).cuda())
    rope, g = qsa.rope_config((64,)), torch.Generator(device="cuda").manual_seed(5)
    w = [torch.ones(n, device="cuda") for n in (256, 256, 128)]

    def step(seqs, poss, cells):
        """One token of each sequence, from its projection; checks the outputs
        against the oracle on the layer's own tables and rows."""
        T = len(seqs)
        qkv = torch.randn((T, 20 * 256), generator=g, device="cuda").bfloat16()
        qi = torch.randn((T, 4, 128), generator=g, device="cuda").bfloat16()
        pos = _i32(poss)
        q, k, q_idx = L.norm_rope(rope, pos, qkv[:, :4096].unflatten(1, (16, 256)),
                                  qkv[:, 4096:4608].unflatten(1, (2, 256)), w[0], w[1], qi, pos, w[2])
        v = qkv[:, 4608:].reshape(T, 2, 256).half()
        idx_new = torch.randn((T, 128), generator=g, device="cuda").half()
        w_idx = torch.rand((T, 4), generator=g, device="cuda")
        out = to_np(L.full_step(_i32(seqs), pos, q, q_idx, w_idx, _i32(cells), k, v, idx_new))
        got, cnt = to_np(L.cells), to_np(L.count)
        every = _i32(np.arange(n_cells))
        K, V = (to_np(x) for x in L.kv_read(every))
        plain = default_cfg(kv_type="f16")
        tol = 2e-3 if kv_type == "f16" else 1e-3   # q4_0 rows read back are rounded to fp16: 2^-11 a value
        for t in range(T):
            c = got[t, :cnt[t]]
            assert len(np.unique(c)) == len(c) == min(2048, (poss[t] + 1) // 4 * 4) + (poss[t] + 1) % 4
            ref = O.attend(plain, to_np(q)[t], K, V, n_cells, c)
            assert max_rel(out[t], ref) <= tol
        return out, got[:T].copy(), cnt[:T].copy()

    step([0, 1], [2603, 801], [wl.seq_cells[0][2603], wl.seq_cells[1][801]])
    # sequence 2: the first 2603 positions of sequence 0 (three of its tail block's cells are its own copies)
    extra = np.arange(wl.n_cells, n_cells)
    cs, cd = L.fork(_i32([0]), _i32([2]), _i32([2603]), _i32([wl.n_slots]), _i32(extra[:4].reshape(1, 4)))
    assert int((cs >= 0).sum()) == 3
    rows = [x for x in L.kv_read(cs.flatten()[:3])]
    for a, b in zip(rows, L.kv_read(cd.flatten()[:3])):
        assert torch.equal(a, b)
    assert torch.equal(L.idx_k[cs.flatten()[:3].long()], L.idx_k[cd.flatten()[:3].long()])
    # all three go on; sequence 2's block 651 starts at position 2604
    L.seq_blk_slots[int(off[2]) + 651] = wl.n_slots + 1
    L.slot_block_idx[wl.n_slots + 1] = 651
    step([0, 1, 2], [2604, 802, 2603], [wl.seq_cells[0][2604], wl.seq_cells[1][802], extra[3]])
    _, c2, n2 = step([2], [2604], [extra[4]])
    # sequence 0 finishes; the rest moves together
    every = _i32(np.arange(n_cells))
    K0, V0 = (x.clone() for x in L.kv_read(every))
    idx0 = L.idx_k.clone()
    s = L.release(_i32([0, 803, 2605]), compact=True)
    held, free, _, moves = to_np(s["counts"]).tolist()
    assert held == 803 + 2605 and free == n_cells - held and moves > 0
    cm = to_np(s["cell_map"])
    K1, V1 = L.kv_read(every)
    old = np.where(cm >= 0)[0]
    at, to = torch.from_numpy(old).cuda(), torch.from_numpy(cm[old]).cuda().long()
    assert torch.equal(K1[to], K0[at]) and torch.equal(V1[to], V0[at]) and torch.equal(L.idx_k[to], idx0[at])
    tb = to_np(L.blk_cells)
    assert np.array_equal(np.sort(tb[tb >= 0]), np.arange(held))
    # and on with cells from the free list
    fcells = to_np(s["free_cells"])
    step([1, 2], [803, 2605], fcells[:2])
    assert_no_device_errors()


def test_outputs_that_the_next_call_reads_early():
    """The step's kernels read their inputs (queries, new rows, block lists,
    cells) before they wait for their predecessor.  Calls that write such inputs
    are followed at once by the calls that read them, 40 times with new data;
    every result is that of the same calls with a synchronisation between."""
    wl = make_workload(n_seq=2, prompt_len=[3000, 900], n_steps=1, seed=95, kv_type="q4_0")
    A, B = QSALayer.from_workload(wl, 0, max_tokens=8), QSALayer.from_workload(wl, 0, max_tokens=8)
    rope, cfg = qsa.rope_config((128,)), A.cfg
    g = torch.Generator(device="cuda").manual_seed(6)
    w = [torch.ones(n, device="cuda") for n in (256, 256, 128)]
    st = step_inputs(wl.steps[0], new_cells=True)
    for it in range(40):
        T = 2
        q_in = torch.randn((T, 16, 256), generator=g, device="cuda").bfloat16()
        k_in = torch.randn((T, 2, 256), generator=g, device="cuda").bfloat16()
        qi = torch.randn((T, 4, 128), generator=g, device="cuda").bfloat16()
        w_idx, idx_new = torch.rand((T, 4), generator=g, device="cuda"), torch.randn((T, 128), generator=g, device="cuda").half()
        v = torch.randn((T, 2, 256), generator=g, device="cuda").half()
        pos = st["tok_pos"]
        outs = []
        for L, sync in ((A, False), (B, True)):
            wait = torch.cuda.synchronize if sync else (lambda: None)
            torch.cuda.synchronize()
            q, k, q_idx = L.norm_rope(rope, pos, q_in, k_in, w[0], w[1], qi, pos, w[2])
            wait()
            out = L.full_step(st["tok_seq"], pos, q, q_idx, w_idx, st["cells"], k, v, idx_new).clone()
            wait()
            q2, _, _ = L.norm_rope(rope, pos, q_in * 2, k_in, w[1], w[1], qi, pos, w[2])
            wait()
            L.sparse_attn(q2, T)               # reads the queries first thing
            out2 = L.out[:T].clone()
            wait()
            kr, vr = L.kv_read(st["cells"])    # and an append of rows just read back
            wait()
            L.kv_append(st["tok_seq"], pos, st["cells"], kr, vr, idx_new)
            wait()
            torch.cuda.synchronize()
            outs.append((out, out2, kr, vr, L.k_cache.clone(), L.v_cache.clone(), L.cells.clone()))
        for a, b in zip(*outs):
            assert torch.equal(a, b), it
    assert_no_device_errors()


@pytest.mark.parametrize("handle", [False, True])
def test_layer_calls_on_a_stream_that_is_ahead(handle):
    """A layer's calls on another stream than the current one, which is busy: what they allocate and fill must be
    ordered on their own stream."""
    wl = make_workload(n_seq=2, prompt_len=[3000, 902], n_steps=1, seed=97, kv_type="q4_0")
    cells, length = _i32(wl.seq_cells[0][:500]), _i32([3000, 900])
    # sequence 1's block 225 (positions 900, 901) is freed first; then it is forked from sequence 0 with that block
    tail = [int(c) for c in wl.seq_cells[1][900:902]] + [-1, -1]
    slot = int(wl.seq_blk_slots[wl.seq_blk_off[1] + 225])
    fork = [_i32(x) for x in ([0], [1], [802], [slot], [tail])]
    got = []
    for ahead in (False, True):
        L = QSALayer.from_workload(wl, 0)
        other = torch.cuda.Stream()
        stream = None if not ahead else other.cuda_stream if handle else other
        torch.cuda.synchronize()
        if ahead:
            torch.cuda._sleep(40_000_000)          # some 20 ms on the current stream
        k, v = L.kv_read(cells, stream=stream)
        swept = L.release(length, stream=stream)
        swept = {n: t for n, t in swept.items() if not n.startswith("move")}
        pairs = L.fork(*fork, stream=stream)
        torch.cuda.synchronize()
        got.append([k, v, *swept.values(), *pairs, L.blk_cells, L.k_cache])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert_no_device_errors()


def test_norm_rope_of_more_tokens_leaves_the_layers_buffers():
    """A captured call writes the layer's buffers; a larger eager call in between does not move them."""
    wl = make_workload(n_seq=1, prompt_len=[400], n_steps=1, seed=98)
    L, rope = QSALayer.from_workload(wl, 0, max_tokens=4), qsa.rope_config((64,))
    g = torch.Generator(device="cuda").manual_seed(3)
    w = [torch.ones(n, device="cuda") for n in (256, 256, 128)]

    def rows(T):
        return [torch.randn((T, h, d), generator=g, device="cuda") for h, d in ((16, 256), (2, 256), (4, 128))]

    small, large = rows(2), rows(9)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    call = lambda x: L.norm_rope(rope, pos[:len(x[0])], x[0], x[1], w[0], w[1], x[2], pos[:len(x[0])], w[2])  # noqa: E731
    first = call(small)
    want = [t.clone() for t in first]
    at = [t.data_ptr() for t in first]
    big = [t.clone() for t in call(large)]
    again = call(small)
    assert [t.data_ptr() for t in again] == at
    for a, b in zip(again, want):
        assert torch.equal(a, b)
    for a, b in zip(call(large), big):
        assert torch.equal(a, b)
    assert_no_device_errors()
