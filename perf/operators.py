"""Timed cases of the operators around a QSA layer's K/V cache.

Head norms with the position rotation in one pass (qk_norm_rope), a cache held
in 4 bits (kv_append and kv_read on it, and the sparse attention that reads
it), and the upkeep of a cache's cells and blocks (cells_copy, seq_fork,
cache_sweep).  Head shapes are the layer's: 16 query heads over 2 KV heads of
256 dims, 4 indexer heads of 128, 4 cells per block, 2048 + 3 cells per token.

`run` computes the plain form (elementary torch operations) or, with `own`
set, makes the library's calls on the same state.  `exact` is the definition
in 64 bits.
"""
import numpy as np
import torch

own = False

HQ, G, D = 16, 2, 256          # query heads, KV heads, head dim
HI, DI = 4, 128                # indexer heads and dims
R, TOP_K = 4, 2048             # cells per block, selected cells per token
PITCH = TOP_K + R - 1
THETA, EPS, SCALE = 1.0e6, 1.0e-6, 1.0 / 16.0
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
# pairs of each position axis (time; time, height, width) for the rotated dims
SECTIONS = {(1, 256): (128,), (1, 128): (64,), (1, 64): (32,), (3, 256): (48, 40, 40), (3, 128): (24, 20, 20),
            (3, 64): (12, 10, 10)}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token out of a fused bf16 projection
        dict(name="norm_rope decode", op="norm_rope", tokens=1, dtype="bf16", axes=1, n_rot=256, interleaved=False,
             far=250_000),
        # a prompt with images: three position axes, half of each head rotated
        dict(name="norm_rope prompt 3 axes", op="norm_rope", tokens=8192, dtype="fp16", axes=3, n_rot=128,
             interleaved=True, far=8192),
        # five sequences decode one token each into a 4-bit cache
        dict(name="q4 append 5", op="append", tokens=5, seqs=5, cells=65_536),
        # the largest chunk an append takes, two sequences
        dict(name="q4 append 1024", op="append", tokens=1024, seqs=2, cells=65_536),
        # one token's attention at 50k
        dict(name="q4 attention decode", op="attention", tokens=1, cells=50_003, count=2051),
        # a 512-token prompt chunk at 250k
        dict(name="q4 attention prompt", op="attention", tokens=512, cells=250_000, count=2051),
        # the tail cells of four forked sequences
        dict(name="copy fork tails", op="copy", pairs=12, cells=50_000),
        # the moves of a large compaction
        dict(name="copy compaction", op="copy", pairs=100_000, cells=250_000),
        # a second answer to one 50k prompt
        dict(name="fork one", op="fork", forks=1, pos=50_003),
        # eight answers to one 250k prompt
        dict(name="fork eight", op="fork", forks=8, pos=250_001),
        # a finished session's cells are freed
        dict(name="sweep free", op="sweep", cells=50_000, seqs=3, compact=False),
        # a cache of five long sessions is made dense again
        dict(name="sweep compact", op="sweep", cells=1_250_000, seqs=12, compact=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attention", "attention", "copy", "fork", "sweep"])
    if op == "norm_rope":
        axes, n_rot = rng.choice(sorted(SECTIONS))
        return dict(op=op, tokens=_log(rng, 1, 8191), dtype=rng.choice(["fp16", "bf16"]), axes=axes, n_rot=n_rot,
                    interleaved=axes > 1 and rng.random() < 0.5, far=_log(rng, 10, 1_000_000))
    if op == "append":
        tokens = _log(rng, 1, 1023)
        return dict(op=op, tokens=tokens, seqs=_log(rng, 1, min(tokens, 64)), cells=_log(rng, 8192, 65_535))
    if op == "attention":
        tokens = _log(rng, 1, 400)
        return dict(op=op, tokens=tokens, cells=_log(rng, 2100, 249_999), count=_log(rng, 1, PITCH))
    if op == "copy":
        pairs = _log(rng, 1, 99_999)
        return dict(op=op, pairs=pairs, cells=max(2 * pairs + 1, _log(rng, 10_000, 249_999)))
    if op == "fork":
        return dict(op=op, forks=_log(rng, 1, 8), pos=_log(rng, 1, 249_999))
    return dict(op=op, cells=_log(rng, 1000, 1_249_999), seqs=_log(rng, 1, 64), compact=rng.random() < 0.6)


# ------------------------------------------------------------- their inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _encode_q4(x):
    """q4_0 blocks of the last axis (fp32): codes uint8 (two per byte: value i
    of a block low, value i + 16 high) and fp16 scales."""
    b = x.unflatten(-1, (-1, 32))
    at = torch.arange(32, device=b.device).expand_as(b)      # the first value of largest magnitude
    at = at.masked_fill(b.abs() < b.abs().amax(-1, keepdim=True), 32).amin(-1, keepdim=True)
    d = b.gather(-1, at) * -0.125
    inv = torch.where(d != 0, torch.ones_like(d) / d, torch.zeros_like(d))
    n = torch.floor(b * inv + 8.5).clamp(0, 15).to(torch.uint8)
    return (n[..., :16] | (n[..., 16:] << 4)).flatten(-2), d.squeeze(-1).to(torch.float16)


def _q4_values(codes, d):
    """fp32 values of q4_0 codes [..., D / 2] and scales [..., D / 32]."""
    b = codes.unflatten(-1, (-1, 16))
    n = torch.cat([b & 15, b >> 4], dim=-1).float() - 8.0
    return (n * d.float().unsqueeze(-1)).flatten(-2)


def _q4_parts(cache, n_cells):
    """Views of a q4_0 cache's codes [n][G][D/2] and scales [n][G][D/32]."""
    nq = n_cells * G * D // 2
    return cache[:nq].view(n_cells, G, D // 2), cache[nq:].view(torch.float16).view(n_cells, G, D // 32)


def _q4_cache(g, n_cells):
    cache = torch.empty(n_cells * G * (D // 2 + D // 16), dtype=torch.uint8, device="cuda")
    codes, d = _q4_parts(cache, n_cells)
    codes[...], d[...] = _encode_q4(_randn(g, n_cells, G, D).float())
    return cache


def _prepare_norm_rope(c, g, rng):
    T, H = c["tokens"], HQ + 2 * G
    qkv = _randn(g, T, H * D, dtype=DTYPES[c["dtype"]])      # a fused projection: q, k and v of a token in one row
    start = int(rng.integers(0, max(1, c["far"] - T + 1)))
    pos = start + np.arange(T)
    axes = [pos] + [pos[0] + rng.integers(0, 64, T) for _ in range(c["axes"] - 1)]
    return dict(q_in=qkv[:, :HQ * D].unflatten(1, (HQ, D)), k_in=qkv[:, HQ * D:(HQ + G) * D].unflatten(1, (G, D)),
                qi_in=_randn(g, T, HI, DI, dtype=DTYPES[c["dtype"]]), pos=_ints(np.stack(axes)), idx_pos=_ints(pos),
                q_w=1.0 + 0.1 * _randn(g, D, dtype=torch.float32), k_w=1.0 + 0.1 * _randn(g, D, dtype=torch.float32),
                qi_w=1.0 + 0.1 * _randn(g, DI, dtype=torch.float32),
                q=torch.empty((T, HQ, D), dtype=torch.float16, device="cuda"),
                k=torch.empty((T, G, D), dtype=torch.float16, device="cuda"),
                qi=torch.empty((T, HI, DI), dtype=torch.float32, device="cuda"))


def _prepare_append(c, g, rng):
    T, S, n = c["tokens"], c["seqs"], c["cells"]
    per = np.full(S, T // S)
    per[:T % S] += 1
    have = rng.integers(0, max(1, (n - T) // S - 8), S)      # positions each sequence holds already
    cap = -(-(have + per) // R)
    off = np.concatenate([[0], np.cumsum(cap)])
    n_slots = n // R + S                                     # the cache's blocks, more than the lists name
    slots = rng.permutation(n_slots)[:off[-1]]
    tok_seq = np.repeat(np.arange(S), per)
    tok_pos = np.concatenate([h + np.arange(p) for h, p in zip(have, per)])
    cells = rng.permutation(n)[:T]
    return dict(tok_seq=_ints(tok_seq), tok_pos=_ints(tok_pos), cells=_ints(cells), k_new=_randn(g, T, G, D),
                v_new=_randn(g, T, G, D), idx_new=_randn(g, T, DI),
                k_cache=torch.zeros(n * G * (D // 2 + D // 16), dtype=torch.uint8, device="cuda"),
                v_cache=torch.zeros(n * G * (D // 2 + D // 16), dtype=torch.uint8, device="cuda"),
                idx_k=torch.zeros((n, DI), dtype=torch.float16, device="cuda"),
                blk_cells=torch.full((n_slots, R), -1, dtype=torch.int32, device="cuda"),
                off=torch.from_numpy(off.astype(np.int64)).cuda(), slots=_ints(slots),
                dirty=torch.full((T,), -1, dtype=torch.int32, device="cuda"),
                k_out=torch.empty((T, G, D), dtype=torch.float16, device="cuda"),
                v_out=torch.empty((T, G, D), dtype=torch.float16, device="cuda"))


def _prepare_attention(c, g, rng):
    T, n, count = c["tokens"], c["cells"], c["count"]
    nb = n // R - 1                                          # whole blocks to choose from, the last one is the tail's
    sel = min(count // R, nb, TOP_K // R)
    tail = count - count // R * R
    if sel:
        pick = torch.rand((T, nb), generator=g, device="cuda").topk(sel, dim=1).indices.sort(dim=1).values
        cells = (pick.unsqueeze(-1) * R + torch.arange(R, device="cuda")).flatten(1)
    else:
        cells = torch.empty((T, 0), dtype=torch.int64, device="cuda")
    lists = torch.full((T, PITCH), -1, dtype=torch.int32, device="cuda")
    lists[:, :sel * R] = cells.int()
    lists[:, sel * R:sel * R + tail] = (nb * R + torch.arange(tail, device="cuda")).int()
    return dict(q=_randn(g, T, HQ, D), k_cache=_q4_cache(g, n), v_cache=_q4_cache(g, n), cells=lists,
                count=torch.full((T,), sel * R + tail, dtype=torch.int32, device="cuda"),
                out=torch.empty((T, HQ, D), dtype=torch.float32, device="cuda"))


def _prepare_copy(c, g, rng):
    n, m = c["cells"], c["pairs"]
    at = rng.permutation(n)[:2 * m]
    return dict(src=_ints(np.sort(at[:m])), dst=_ints(np.sort(at[m:])), k_cache=_randn(g, n, G, D),
                v_cache=_randn(g, n, G, D), idx_k=_randn(g, n, DI))


def _prepare_fork(c, g, rng):
    F, p = c["forks"], c["pos"]
    n_pos = np.maximum(1, p - rng.integers(0, 8, F))         # the answers start at and just before the prompt's end
    cap = p // R + 64                                        # room to go on
    off = np.arange(F + 2) * cap                             # sequence 0 holds the prompt, 1..F are the forks
    nb = -(-p // R)
    n_slots, n_cells = nb + F, p + F * R
    order, cell = rng.permutation(n_slots), rng.permutation(n_cells)
    lists = np.zeros((F + 1) * cap)
    lists[:nb] = order[:nb]
    table = np.full((n_slots, R), -1)
    flat = np.full(nb * R, -1)
    flat[:p] = cell[:p]
    table[order[:nb]] = flat.reshape(nb, R)
    block = np.zeros(n_slots)
    block[order[:nb]] = np.arange(nb)
    return dict(src_seq=_ints(np.zeros(F)), dst_seq=_ints(1 + np.arange(F)), n_pos=_ints(n_pos),
                tail_slot=_ints(order[nb:]), tail_cells=_ints(cell[p:].reshape(F, R)),
                off=torch.from_numpy(off.astype(np.int64)).cuda(), lists=_ints(lists), table=_ints(table),
                block=_ints(block), max_blocks=nb,
                copy_src=torch.full((F, R), -1, dtype=torch.int32, device="cuda"),
                copy_dst=torch.full((F, R), -1, dtype=torch.int32, device="cuda"))


def _prepare_sweep(c, g, rng):
    n, S = c["cells"], c["seqs"]
    length = rng.multinomial(int(n * 0.9), np.full(S, 1.0 / S))
    share = np.zeros(S, dtype=np.int64)                      # blocks each sequence shares with the one before it
    if S > 2:
        share[1::3] = length[:-1][::3][:len(share[1::3])] // R // 2
    share = np.minimum(share, length // R)
    cap = -(-length // R) + 2
    off = np.concatenate([[0], np.cumsum(cap)])
    n_slots = n // R + 3 * S                                 # the cache's blocks, more than the lists name
    order, cell = rng.permutation(n_slots)[:off[-1]], rng.permutation(n)
    table = np.full((n_slots, R), -1)
    of = np.repeat(np.arange(S), length)                     # sequence and position of each occupied cell
    p = np.arange(len(of)) - np.repeat(np.cumsum(length) - length, length)
    table[order[off[of] + p // R], p % R] = cell[:len(of)]
    of = np.repeat(np.arange(S), cap)                        # sequence and block of each list entry
    j = np.arange(len(order)) - off[of]
    lists = np.where(j < share[of], order[np.minimum(off[np.maximum(of - 1, 0)] + j, len(order) - 1)], order)
    keep = length.copy()
    keep[rng.random(S) < 0.4] = 0                            # finished sessions
    cut = rng.random(S) < 0.3
    keep[cut] = keep[cut] // 2                               # sessions rolled back
    return dict(seq_len=_ints(keep), off=torch.from_numpy(off.astype(np.int64)).cuda(), lists=_ints(lists),
                table=_ints(table), table_out=_ints(np.full((n_slots, R), -7)), ws=None, n_cells=n,
                compact=bool(c["compact"]), counts=_ints(np.zeros(4)), cell_map=_ints(np.full(n, -7)),
                free_cells=_ints(np.full(n, -1)), free_slots=_ints(np.full(n_slots, -1)),
                move_src=_ints(np.full(n // 2 + 1, -1)), move_dst=_ints(np.full(n // 2 + 1, -1)))


def prepare(case, seed):
    make = {"norm_rope": _prepare_norm_rope, "append": _prepare_append, "attention": _prepare_attention,
            "copy": _prepare_copy, "fork": _prepare_fork, "sweep": _prepare_sweep}[case["op"]]
    state = make(case, _gen(seed), np.random.default_rng(seed))
    state["case"] = case
    return state


# ---------------------------------------------------------- the library's calls
def _own(s):
    from sparse_attention_long_qsa_gb300 import qsa

    c, op = s["case"], s["case"]["op"]
    if "cfg" not in s:                                       # the handle a program keeps
        s["cfg"] = qsa.config(kv_type="q4_0" if op in ("append", "attention") else "f16")
        if op == "norm_rope":
            s["rope"] = qsa.rope_config(SECTIONS[c["axes"], c["n_rot"]], interleaved=c["interleaved"])
        if op == "sweep":
            s["ws"] = torch.empty(qsa.cache_sweep_workspace_size(s["cfg"], s["n_cells"], s["table"].shape[0]),
                                  dtype=torch.uint8, device="cuda")
    cfg = s["cfg"]
    if op == "norm_rope":
        qsa.qk_norm_rope(cfg, s["rope"], s["pos"], s["q_in"], s["k_in"], s["q_w"], s["k_w"], s["q"], s["k"],
                         q_idx_in=s["qi_in"], idx_pos=s["idx_pos"], q_idx_norm_w=s["qi_w"], q_idx=s["qi"])
        return s["q"], s["k"], s["qi"]
    if op == "append":
        qsa.kv_append(cfg, s["tok_seq"], s["tok_pos"], s["cells"], s["k_new"], s["v_new"], s["idx_new"],
                      s["k_cache"], s["v_cache"], s["idx_k"], s["blk_cells"], s["off"], s["slots"], s["dirty"])
        qsa.kv_read(cfg, s["cells"], s["k_cache"], s["v_cache"], c["cells"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"], s["idx_k"], s["blk_cells"], s["dirty"]
    if op == "attention":
        qsa.sparse_attn(cfg, s["q"], s["k_cache"], s["v_cache"], c["cells"], s["cells"], s["count"], s["out"])
        return s["out"]
    if op == "copy":
        qsa.cells_copy(cfg, s["src"], s["dst"], s["k_cache"], s["v_cache"], s["idx_k"], c["cells"])
        return s["k_cache"], s["v_cache"], s["idx_k"]
    if op == "fork":
        qsa.seq_fork(cfg, s["src_seq"], s["dst_seq"], s["n_pos"], s["tail_slot"], s["tail_cells"], s["off"],
                     s["lists"], s["table"], s["block"], s["max_blocks"], s["copy_src"], s["copy_dst"])
        return s["lists"], s["table"], s["block"], s["copy_src"], s["copy_dst"]
    qsa.cache_sweep(cfg, s["seq_len"], s["off"], s["lists"], s["table"], s["table_out"], s["n_cells"], s["counts"],
                    s["ws"], compact=s["compact"], cell_map=s["cell_map"], free_cells=s["free_cells"],
                    free_slots=s["free_slots"], move_src=s["move_src"], move_dst=s["move_dst"])
    return (s["table_out"], s["counts"], s["cell_map"], s["free_cells"], s["free_slots"], s["move_src"],
            s["move_dst"])


# ------------------------------------------------------------ the plain forms
def _axis_of_pair(c):
    sec = SECTIONS[c["axes"], c["n_rot"]]
    if not c["interleaved"]:
        return np.repeat(np.arange(len(sec)), sec)
    i = np.arange(sum(sec))
    a = i % len(sec)
    return np.where(i // len(sec) < np.array(sec)[a], a, 0)


def _norm_rotate(x, w, ang):
    """x [T][H][n]: RMS norm, then the pairs (i, i + m) of the first 2m dims
    turned by ang [T][m] (float64)."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    m = ang.shape[1]
    cos, sin = ang.cos().float().unsqueeze(1), ang.sin().float().unsqueeze(1)
    a, b = x[..., :m], x[..., m:2 * m]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * m:]], dim=-1)


def _freqs(n):
    return THETA ** (-2.0 * torch.arange(n // 2, dtype=torch.float64, device="cuda") / n)


def _plain_norm_rope(s, c):
    axis = torch.from_numpy(_axis_of_pair(c)).cuda()
    ang = s["pos"].double()[axis].T * _freqs(c["n_rot"])
    return (_norm_rotate(s["q_in"], s["q_w"], ang).half(), _norm_rotate(s["k_in"], s["k_w"], ang).half(),
            _norm_rotate(s["qi_in"], s["qi_w"], s["idx_pos"].double().unsqueeze(1) * _freqs(DI)))


def _plain_rows(rows, cache, cells, n):
    codes, d = _q4_parts(cache, n)
    codes[cells], d[cells] = _encode_q4(rows.float())
    return _q4_values(codes[cells], d[cells]).half()


def _plain_append(s, c):
    cells = s["cells"].long()
    k_out = _plain_rows(s["k_new"], s["k_cache"], cells, c["cells"])
    v_out = _plain_rows(s["v_new"], s["v_cache"], cells, c["cells"])
    s["idx_k"][cells] = s["idx_new"]
    pos = s["tok_pos"].long()
    slot = s["slots"].long()[s["off"][s["tok_seq"].long()] + pos // R]
    s["blk_cells"][slot, pos % R] = s["cells"]
    order = slot.sort().values
    first = torch.cat([torch.ones_like(order[:1], dtype=torch.bool), order[1:] != order[:-1]])
    at = torch.where(first, first.cumsum(0) - 1, torch.full_like(order, len(order)))
    dirty = torch.full((len(order) + 1,), -1, dtype=torch.int32, device="cuda")
    dirty[at] = order.int()
    return k_out, v_out, s["idx_k"], s["blk_cells"], dirty[:-1]


def _plain_attention(s, c):
    n, T = c["cells"], c["tokens"]
    live = torch.arange(PITCH, device="cuda") < s["count"].unsqueeze(1)
    at = s["cells"].long().clamp(min=0)
    kc, kd = _q4_parts(s["k_cache"], n)
    vc, vd = _q4_parts(s["v_cache"], n)
    K = _q4_values(kc[at], kd[at]).permute(0, 2, 3, 1)                     # [T][G][D][C]
    S = torch.matmul(s["q"].float().view(T, G, HQ // G, D), K) * SCALE
    S = S.masked_fill(~live[:, None, None], float("-inf"))
    E = torch.exp(S - S.amax(-1, keepdim=True))
    V = _q4_values(vc[at], vd[at]).permute(0, 2, 1, 3)                     # [T][G][C][D]
    return (torch.matmul(E, V) / E.sum(-1, keepdim=True)).view(T, HQ, D)


def _plain_copy(s, c):
    src, dst = s["src"].long(), s["dst"].long()
    s["k_cache"][dst] = s["k_cache"][src]
    s["v_cache"][dst] = s["v_cache"][src]
    s["idx_k"][dst] = s["idx_k"][src]
    return s["k_cache"], s["v_cache"], s["idx_k"]


def _plain_fork(s, c):
    lists, off = s["lists"], s["off"]
    nb, tail = s["n_pos"].long() // R, s["n_pos"].long() % R
    a, b = off[s["src_seq"].long()], off[s["dst_seq"].long()]
    j = torch.arange(s["max_blocks"] + 1, device="cuda")
    old = lists[b.unsqueeze(1) + j]
    new = torch.where(j < nb.unsqueeze(1), lists[a.unsqueeze(1) + j], old)
    new = torch.where((j == nb.unsqueeze(1)) & (tail > 0).unsqueeze(1), s["tail_slot"].unsqueeze(1), new)
    lists[b.unsqueeze(1) + j] = new
    i = torch.arange(R, device="cuda")
    has, none = i < tail.unsqueeze(1), torch.full_like(s["tail_cells"], -1)
    from_cells = s["table"][lists[a + nb].long()]
    s["copy_src"][...] = torch.where(has, from_cells, none)
    s["copy_dst"][...] = torch.where(has, s["tail_cells"], none)
    t = s["tail_slot"].long()
    s["table"][t] = torch.where((tail > 0).unsqueeze(1), torch.where(has, s["tail_cells"], none), s["table"][t])
    s["block"][t] = torch.where(tail > 0, nb.int(), s["block"][t])
    return lists, s["table"], s["block"], s["copy_src"], s["copy_dst"]


def _plain_sweep(s, c):
    n, table, lists = s["n_cells"], s["table"], s["lists"].long()
    n_slots, e = table.shape[0], torch.arange(len(lists), device="cuda")
    seq = torch.searchsorted(s["off"], e, right=True) - 1
    held = (s["seq_len"].long()[seq] - (e - s["off"][seq]) * R).clamp(0, R)    # positions held of each listed block
    slot_live = torch.zeros(n_slots, dtype=torch.int32, device="cuda").index_add_(0, lists, (held > 0).int()) > 0
    cell = table[lists].long()
    has = (torch.arange(R, device="cuda") < held.unsqueeze(1)) & (cell >= 0)
    live = torch.zeros(n + 1, dtype=torch.int32, device="cuda").index_add_(
        0, torch.where(has, cell, torch.full_like(cell, n)).flatten(), has.int().flatten())[:n] > 0
    at, n_live = torch.arange(n, device="cuda"), live.sum()
    none = torch.full_like(at, -1)
    new = torch.where(live, at, none)
    m = n // 2 + 1
    src, dst = torch.full((2, m + 1), -1, dtype=torch.int64, device="cuda")
    if s["compact"]:
        goes, hole = live & (at >= n_live), ~live & (at < n_live)
        kg, kh = goes.long().cumsum(0) - 1, hole.long().cumsum(0) - 1
        src[torch.where(goes, kg, torch.full_like(kg, m))] = at
        dst[torch.where(hole, kh, torch.full_like(kh, m))] = at
        new = torch.where(goes, dst[kg.clamp(min=0)], new)
        moves = goes.sum()
    else:
        moves = torch.zeros_like(n_live)
    old = table.long()
    out = torch.where((old >= 0) & slot_live.unsqueeze(1), new[old.clamp(min=0)], torch.full_like(old, -1))
    free = at >= n_live if s["compact"] else ~live
    fc = torch.full((n + 1,), -1, dtype=torch.int32, device="cuda")
    fc[torch.where(free, free.long().cumsum(0) - 1, torch.full_like(at, n))] = at.int()
    fs = torch.full((n_slots + 1,), -1, dtype=torch.int32, device="cuda")
    sl = torch.arange(n_slots, device="cuda")
    fs[torch.where(~slot_live, (~slot_live).long().cumsum(0) - 1, torch.full_like(sl, n_slots))] = sl.int()
    counts = torch.stack([n_live, n - n_live, (~slot_live).sum(), moves]).int()
    return out.int(), counts, new.int(), fc[:-1], fs[:-1], src[:-1].int(), dst[:-1].int()


def run(state):
    if own:
        return _own(state)
    plain = {"norm_rope": _plain_norm_rope, "append": _plain_append, "attention": _plain_attention,
             "copy": _plain_copy, "fork": _plain_fork, "sweep": _plain_sweep}[state["case"]["op"]]
    return plain(state, state["case"])


# ------------------------------------------------------------------- the work
def work(case):
    c, op = case, case["op"]
    row = G * (D // 2 + D // 16)                             # a cell's K (or V) bytes in 4 bits
    if op == "norm_rope":
        size = 4 if c["dtype"] == "fp32" else 2
        heads, idx = (HQ + G) * D, HI * DI
        return dict(bytes=c["tokens"] * (heads * (size + 2) + idx * (size + 4) + 4 * (c["axes"] + 1)) + 4 * (2 * D + DI),
                    flops=c["tokens"] * (heads + idx) * 7)
    if op == "append":
        rows, out = 2 * G * D * 2, c["cells"] * DI * 2
        return dict(bytes=c["tokens"] * (2 * rows + 4 * row + 2 * DI * 2 + 12 + 2 * R * 4), flops=c["tokens"] * 2 * G * D * 6)
    if op == "attention":
        T, n, count = c["tokens"], c["cells"], c["count"]
        touched = n * (1.0 - (1.0 - min(1.0, count / n)) ** T)
        return dict(bytes=T * (HQ * D * (2 + 4) + 4 * count + 4) + touched * 2 * row, flops=4.0 * T * HQ * D * count)
    if op == "copy":
        return dict(bytes=c["pairs"] * (2 * (2 * G * D * 2 + DI * 2) + 8), flops=0)
    if op == "fork":
        return dict(bytes=c["forks"] * (2 * 4 * (c["pos"] // R) + 5 * 4 * R), flops=0)
    n, slots = c["cells"], 0.9 * c["cells"] / R
    return dict(bytes=4 * (2 * n + 2 * slots * R + slots) + (4 * n * 0.3 if c["compact"] else 0), flops=0)


# -------------------------------------------------------- the definitions, in 64 bits
def _exact_rows(x, w, pos, axis, m):
    """RMS norm and rotation of [T][H][n] rows as complex products."""
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    i = torch.arange(m, dtype=torch.float64, device="cuda")
    turn = torch.exp(-(2.0 * i / (2 * m)) * float(np.log(THETA)))
    phase = pos.double().T[:, axis] * turn
    z = torch.complex(x[..., :m].contiguous(), x[..., m:2 * m].contiguous())
    z = z * torch.polar(torch.ones_like(phase), phase).unsqueeze(1)
    return torch.cat([z.real, z.imag, x[..., 2 * m:]], dim=-1)


def _exact_q4(rows):
    """Values of the rows' q4_0 encoding: d = -m / 8 held in fp16, codes by the
    unrounded d."""
    b = rows.double().unflatten(-1, (-1, 32))
    hi, lo = b.amax(-1), b.amin(-1)
    i = torch.arange(32, device="cuda")
    first_hi = torch.where(b == hi.unsqueeze(-1), i, 32).amin(-1) < torch.where(b == lo.unsqueeze(-1), i, 32).amin(-1)
    ext = torch.where((hi > -lo) | ((hi == -lo) & first_hi), hi, lo)
    d = ext / -8.0
    n = torch.where(d.unsqueeze(-1) != 0, torch.floor(b / torch.where(d == 0, torch.ones_like(d), d).unsqueeze(-1) + 8.5),
                    torch.full_like(b, 8.0)).clamp(0, 15)
    return ((n - 8.0) * d.half().double().unsqueeze(-1)).flatten(-2)


def _exact_values(codes, d):
    b = codes.long().unflatten(-1, (-1, 1, 16))
    n = torch.cat([b % 16, b // 16], dim=-2).double() - 8.0
    return (n * d.double()[..., None, None]).flatten(-3)


def _exact_token(q, kc, kd, vc, vd):
    K, V = _exact_values(kc, kd).permute(1, 0, 2), _exact_values(vc, vd).permute(1, 0, 2)   # [G][C][D]
    p = torch.softmax(q.double().view(G, HQ // G, D) @ K.transpose(1, 2) * SCALE, dim=-1)
    return (p @ V).reshape(HQ, D)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "norm_rope":
        axis, m = torch.from_numpy(_axis_of_pair(c)).cuda(), c["n_rot"] // 2
        one = torch.zeros(DI // 2, dtype=torch.int64, device="cuda")
        return (_exact_rows(s["q_in"], s["q_w"], s["pos"], axis, m), _exact_rows(s["k_in"], s["k_w"], s["pos"], axis, m),
                _exact_rows(s["qi_in"], s["qi_w"], s["idx_pos"].unsqueeze(0), one, DI // 2))
    if op == "append":
        idx = s["idx_k"].double()
        idx[s["cells"].long()] = s["idx_new"].double()
        return _exact_q4(s["k_new"]), _exact_q4(s["v_new"]), idx, None, None
    if op == "attention":
        out = torch.zeros((c["tokens"], HQ, D), dtype=torch.float64, device="cuda")
        kc, kd = _q4_parts(s["k_cache"], c["cells"])
        vc, vd = _q4_parts(s["v_cache"], c["cells"])
        for t in range(c["tokens"]):
            at = s["cells"][t, :int(s["count"][t])].long()
            out[t] = _exact_token(s["q"][t], kc[at], kd[at], vc[at], vd[at])
        return out
    if op == "copy":
        got = []
        for name in ("k_cache", "v_cache", "idx_k"):
            x = s[name].double()
            x[s["dst"].long()] = s[name].double()[s["src"].long()]
            got.append(x)
        return tuple(got)
    return None
