"""Sequences of unusual lengths among the pages of a cache: shorter than the prefix, empty, longer than any table."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import pages_case
from test_gpu_pages import run_rearrange

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spare_columns", [2, 6000])  # one CTA, a cluster
@pytest.mark.parametrize("room", [None, [0, 3, 0, 25, 0, 8, 10, 41]])
def test_sequences_that_end_within_the_prefix(rope_gpu, spare_columns, room):
    """Padding rows of length 0, and sequences shorter than the prefix: lengths are the parent's and the room's."""
    P, bs = 40, 16
    c = pages_case(51, [20, 0, 33, 0], bs, P=P, spare=20, share=False, spare_columns=spare_columns)
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
