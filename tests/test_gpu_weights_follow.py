"""Block weights with the calls around them: a fork's shared blocks weigh what they
weigh in the source, blocks that go leave nothing behind for those that come into
their places, and evictions choose by a sequence's own weights."""
import numpy as np
import pytest
import torch

from sparse_attention_long_qsa_gb300 import qsa
from test_gpu_evict import plain as plain_evict
from test_gpu_paged_layer import _i32, as_paged, layer
from paged_util import no_errors

pytestmark = pytest.mark.gpu
R, G, D = 4, 2, 256


@pytest.mark.parametrize("n_pos", [0, 3, 40, 402, 600, 601])
def test_a_fork_takes_its_sources_weights(n_pos):
    L, wl, cells, slots = layer("f16", [601, 590, 333], seed=5)
    off = L.seq_blk_off.cpu().numpy()
    g = torch.Generator(device="cuda").manual_seed(1)
    L.block_weight = torch.rand(L.seq_blk_slots.numel(), generator=g, device="cuda") + 0.5
    want = L.block_weight.clone()
    # sequence 1's list has room for the fork of at most what is there
    n_pos = min(n_pos, int(off[2] - off[1]) * R)
    L.fork(_i32([0]), _i32([1]), _i32([n_pos]), _i32([slots[0]]), _i32([cells[:R]]))
    nb = n_pos // R
    want[off[1]:off[1] + nb] = want[off[0]:off[0] + nb]
    want[off[1] + nb:off[2]] = 0
    no_errors()
    assert torch.equal(L.block_weight, want)


def test_forks_that_are_refused_leave_the_weights():
    L, wl, cells, slots = layer("f16", [601, 90], seed=6)
    L.block_weight = torch.rand(L.seq_blk_slots.numel(), device="cuda")
    want = L.block_weight.clone()
    # no room in dst's list; a tail slot that does not exist
    L.fork(_i32([0]), _i32([1]), _i32([601]), _i32([slots[0]]), _i32([cells[:R]]))
    assert qsa.debug_check()[0] == -6
    assert torch.equal(L.block_weight, want)
    L.fork(_i32([0]), _i32([1]), _i32([41]), _i32([10 ** 6]), _i32([cells[:R]]))
    assert qsa.debug_check()[0] == -6
    assert torch.equal(L.block_weight, want)


def test_a_sequence_forked_onto_itself():
    L, wl, cells, slots = layer("f16", [601, 90], seed=7)
    off = L.seq_blk_off.cpu().numpy()
    L.block_weight = torch.rand(L.seq_blk_slots.numel(), device="cuda") + 1
    want = L.block_weight.clone()
    L.fork(_i32([0]), _i32([0]), _i32([599]), _i32([slots[0]]), _i32([cells[:R]]))
    want[off[0] + 149:off[1]] = 0
    no_errors()
    assert torch.equal(L.block_weight, want)


@pytest.mark.parametrize("keep", [[601, 90], [600, 0], [1, -3], [0, 89], [597, 10_000]])
def test_release_leaves_no_weight_behind(keep):
    L, wl, cells, slots = layer("f16", [601, 90], seed=8)
    off = L.seq_blk_off.cpu().numpy()
    L.block_weight = torch.rand(L.seq_blk_slots.numel(), device="cuda") + 1
    want = L.block_weight.clone()
    for s, n in enumerate(keep):
        want[min(off[s] + max(0, -(-n // R)), off[s + 1]):off[s + 1]] = 0
    L.release(_i32(keep))
    qsa.debug_check()                                        # (10,000 positions: past the list, flagged by the sweep)
    assert torch.equal(L.block_weight, want)


def test_a_list_past_the_end_is_flagged_and_left():
    c = qsa.config()
    w = torch.ones(10, device="cuda")
    qsa.weight_trim(c, _i32([4, 4]), torch.tensor([0, 5, 11], dtype=torch.int64, device="cuda"), w)
    torch.cuda.synchronize()
    assert qsa.debug_check() == (-6, 4)
    assert w.tolist() == [1, 0, 0, 0, 0, 1, 1, 1, 1, 1]


@pytest.mark.parametrize("kv", ["f16", "q4_0"])
def test_weigh_release_fork_evict(kv):
    """A sequence weighs its blocks, another ends, the first is forked into its place, and both are cut back: each by the
    weights of its own blocks."""
    lens = [602, 590]
    L, wl, cells, slots = layer(kv, lens, seed=9)
    off = L.seq_blk_off.cpu().numpy()
    g = torch.Generator(device="cuda").manual_seed(2)

    def attend(seqs, poss):
        q = (2 * torch.randn((len(seqs), 8 * G, D), generator=g, device="cuda")).half()
        L.paged_attn(_i32(seqs), _i32(poss), q, weigh=True)

    attend([0, 0, 0, 1, 1], [599, 600, 601, 588, 589])
    swept = L.release(_i32([602, 0]))
    n_free, n_slots = int(swept["counts"][1]), int(swept["counts"][2])
    free, slot = swept["free_cells"][:n_free], swept["free_slots"][:n_slots]
    assert not L.block_weight[off[1]:off[2]].any()
    n_pos = 402
    L.fork(_i32([0]), _i32([1]), _i32([n_pos]), slot[:1].clone(), free[:R].clone().view(1, R))
    nb = n_pos // R
    assert torch.equal(L.block_weight[off[1]:off[1] + nb], L.block_weight[off[0]:off[0] + nb])
    attend([1], [n_pos - 1])                                 # the fork goes on by itself
    w, lists = L.block_weight.cpu().numpy(), L.seq_blk_slots.cpu().numpy()
    assert (w[off[1]:off[1] + nb] >= w[off[0]:off[0] + nb]).all() and w[off[1] + nb] > 0
    want = plain_evict(40, 1, 4, np.array([602, n_pos], np.int32), off, lists, w, R)
    new_len, gone = L.evict(_i32([602, n_pos]), 40, n_sink=1, n_recent=4)
    for a, b in zip((new_len, L.seq_blk_slots, L.block_weight, gone), want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    kept = L.block_weight.clone()
    L.release(new_len)
    assert torch.equal(kept, L.block_weight)                 # (an eviction leaves zeros behind the blocks)
    no_errors()
    q = (2 * torch.randn((2, 8 * G, D), generator=g, device="cuda")).half()
    seq, pos = _i32([0, 1]), (new_len - 1).clone()
    out = L.paged_attn(seq, pos, q)
    as_paged(L, kv).check(out, q, seq, pos)
