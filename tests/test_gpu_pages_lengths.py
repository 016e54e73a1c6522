"""Sequences of unusual lengths among the pages of a cache: shorter than the prefix, empty, longer than any table."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import compact_reference, pages_case, rearrange_reference
from test_gpu_pages import run_compact, run_rearrange, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spare", [20, 30000])  # one CTA, a cluster
@pytest.mark.parametrize("room", [None, [0, 3, 0, 25, 0, 8, 10, 41]])
def test_sequences_that_end_within_the_prefix(rope_gpu, spare, room):
    """Padding rows of length 0, and sequences shorter than the prefix: lengths are the parent's and the room's."""
    P, bs = 40, 16
    c = pages_case(51, [20, 0, 33, 0], bs, P=P, spare=spare, share=False)
    c["lens"][1], c["lens"][3] = 30, 0
    parents = [1, 1, 3, 3, 0, 2, -1, 1]
    got = run_rearrange(c, parents, room)
    lens = [int(c["lens"][p]) if p >= 0 else P for p in parents]
    lens = [n + (room[i] if room else 0) for i, n in enumerate(lens)]
    assert got["new_lens"].tolist() == lens
    held = [-(-max(n - P, 0) // bs) for n in lens]
    for row, n in zip(got["new_table"].tolist(), held):
        assert all(0 <= p < c["NB"] for p in row[:n]) and all(p == -77 for p in row[n:])
    mine = [p for row, n in zip(got["new_table"].tolist(), held) for p in row[:n]]
    assert len(set(mine)) == len(mine)
    want = torch.zeros(c["NB"], dtype=torch.int32)
    want[torch.tensor(mine + c["prefix"].tolist())] = 1
    assert torch.equal(got["new_refs"], want)
    assert got["counts"].tolist() == [0, int((want == 0).sum())]


@pytest.mark.parametrize("spare", [9, 30000])  # one CTA, a cluster
@pytest.mark.parametrize("bs", [1, 16])
@pytest.mark.parametrize("P", [0, 40])
@pytest.mark.parametrize("length", [1 << 31, (1 << 62) + 5, (1 << 63) - 1])
def test_lengths_beyond_every_table(rope_gpu, spare, bs, P, length):
    """All of the row's pages are the sequence's then, and the device error says so."""
    c = pages_case(52, [20, 33, 5], bs, P=P, spare=spare, share=False)
    held = -(-33 // bs)
    for j in range(held, c["table"].shape[1]):
        c["table"][1, j] = c["table"][1, 0]
        c["refs"][c["table"][1, 0]] += 1
    c["lens"][1] = length
    got = run_rearrange(c, [0, 2], error=R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
    want = c["refs"].clone()
    want[c["table"][1, :held]] = 0
    assert torch.equal(got["new_refs"], want)
    assert got["new_lens"].tolist() == [P + 20, P + 5]
    got = run_rearrange(c, [1], error=R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
    assert got["new_lens"].tolist() == [P + c["table"].shape[1] * bs]
    assert torch.equal(got["new_table"], c["table"][1:2])
    got = run_compact(c, error=R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
    assert bool((got["new_table"][1] >= 0).all()) and bool((got["new_table"][1] < int(got["counts"][1])).all())


@pytest.mark.parametrize("length", [-1, -(1 << 63)])
def test_negative_lengths(rope_gpu, length):
    """As of an empty sequence."""
    c = pages_case(53, [20, 0, 5], 16, spare=9, share=False)
    want = run_rearrange(c, [0, 1, 2])
    c["lens"][1] = length
    got = run_rearrange(c, [0, 1, 2])
    for k, v in want.items():
        assert torch.equal(got[k], v), k


@pytest.mark.parametrize("P", [0, 40])
@pytest.mark.parametrize("room", [1 << 40, (1 << 63) - 1])
def test_room_beyond_the_table(rope_gpu, P, room):
    """As much as the row's columns hold."""
    c = pages_case(54, [20, 3], 16, P=P, spare=40, share=False)
    got = run_rearrange(c, [0, 1, -1], [room, 5, room], error=R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
    W = c["table"].shape[1]
    assert got["new_lens"].tolist() == [P + 16 * W, P + 8, P + 16 * W]
    assert bool((got["new_table"][[0, 2]] >= 0).all())


@pytest.mark.parametrize("parents", [[0, 1], [1, 0], [1, 1, 0], [1, -1], [0, 0]])
@pytest.mark.parametrize("spare", [9, 30000])  # one CTA, a cluster
def test_a_sequence_cut_short(rope_gpu, parents, spare):
    """Sequence 1 shares whole pages with sequence 0 and was then cut to end inside one: its child may not write on what
    another's child reads."""
    c = pages_case(12, [40, 40], 8, spare=spare, share=False)
    c["refs"][c["table"][1, :4]] = 0
    c["table"][1, :4] = c["table"][0, :4]
    c["refs"][c["table"][0, :4]] = 2
    c["refs"][c["table"][1, 4]] = 0
    c["lens"][1] = 27  # pages 0 to 3, the last with three tokens
    same(run_rearrange(c, parents), rearrange_reference(c, parents))


@pytest.mark.parametrize("n,rows", [(384, 384), (385, 3), (3, 385), (40, 1500), (1500, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_on_both_sides_of_the_choice_of_kernels(rope_gpu, n, rows, in_place):
    """As many as one CTA takes and one more, of old rows and of new ones."""
    g = torch.Generator().manual_seed(55)
    c = pages_case(55, torch.randint(0, 90, (n,), generator=g).tolist(), 16, P=7, spare=12000)
    parents, room = (torch.randint(-1, n, (rows,), generator=g).tolist(), torch.randint(0, 20, (rows,), generator=g).tolist())
    same(run_rearrange(c, parents, room, 20, in_place), rearrange_reference(c, parents, room, 20))
    same(run_compact(c), compact_reference(c, c["NB"] // 2))


@pytest.mark.parametrize("n", [2048, 2049])
def test_compact_on_both_sides_of_the_choice_of_kernels(rope_gpu, n):
    g = torch.Generator().manual_seed(56)
    c = pages_case(56, torch.randint(0, 90, (n,), generator=g).tolist(), 16, P=7, spare=9000)
    assert c["NB"] <= 24576
    same(run_compact(c), compact_reference(c, c["NB"] // 2))
