"""Paged attention with a shared prefix, against a float64 reference (bounds: tests/serving_ref.py).

Cache rows that hold no token are NaN in every case, so a row that leaks shows."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from parity import same_bits
from serving_ref import assert_close, attend_case, attend_reference, check_attend, run_attend, widened

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 2), (5, 1), (14, 2), (32, 1)])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 256])
def test_single_tokens(rope_gpu, dtype, hq, hk, D):
    own = [1, 2, 15, 16, 17, 63, 64, 65, 130]
    check_attend(R, attend_case(1, dtype, [1] * len(own), own, hq=hq, hk=hk, D=D), "decode")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [16, 48, 288, 512])
def test_other_head_sizes(rope_gpu, dtype, D):
    if dtype != torch.float32 and D in (16, 48):
        pytest.skip("16-bit heads are multiples of 32")
    check_attend(R, attend_case(2, dtype, [1, 3, 2], [40, 3, 70], P=37, hq=4, hk=2, D=D), "head size")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("P", [0, 1, 16, 37, 128, 129, 300])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [5, 1, 3, 0], [70, 2, 0, 33]])
def test_prefix_and_new_tokens(rope_gpu, dtype, P, new):
    own = [new[0] + 9, new[1], new[2] + 130, new[3] + 64]
    check_attend(R, attend_case(3, dtype, new, own, P=P, hq=8, hk=2, D=64), "prefix")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("bs", [1, 3, 7, 12, 17, 64, 128, 200])
def test_page_sizes(rope_gpu, dtype, bs):
    check_attend(R, attend_case(4, dtype, [1, 4, 20], [260, 4, 77], P=53, hq=4, hk=2, D=128, bs=bs), "pages")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,own,P", [([300], [300], 0), ([129, 257], [400, 257], 0), ([260, 1, 140], [260, 600, 300], 150)])
def test_prompts(rope_gpu, dtype, D, new, own, P):
    check_attend(R, attend_case(5, dtype, new, own, P=P, hq=4, hk=1, D=D, bs=32), "prompt")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_many_short_sequences_behind_a_prefix(rope_gpu, dtype):
    n = 41
    new = [1 + (i % 3 == 0) for i in range(n)]
    own = [new[i] + (i * 37) % 90 for i in range(n)]
    check_attend(R, attend_case(6, dtype, new, own, P=700, hq=8, hk=2, D=64), "many")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_long_keys_for_few_rows(rope_gpu, dtype):
    """The key axis is split over the device and joined."""
    check_attend(R, attend_case(7, dtype, [1, 2], [3000, 1], P=0, hq=2, hk=1, D=64), "long")
    check_attend(R, attend_case(8, dtype, [1, 1], [5, 9], P=2500, hq=2, hk=1, D=128), "long prefix")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("P", [0, 40])
def test_rows_without_keys(rope_gpu, dtype, P):
    """A sequence shorter than its new tokens: the rows at negative positions see nothing (out 0, lse
    -infinity); with a prefix, rows inside it see only its first keys; sequences of no token."""
    c = attend_case(9, dtype, [4, 0, 3, 2], [4, 0, 3, 2], P=P, hq=4, hk=2, D=64)
    c["lens"] = torch.tensor([2, 0, 30 if P else 1, 0])
    out, lse = check_attend(R, c, "empty rows")
    assert torch.equal(lse[:2], torch.full((2, 4), float("-inf"))) and not out[:2].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_spare_rows_and_strided_queries(rope_gpu, dtype):
    c = attend_case(10, dtype, [1, 5, 1], [20, 5, 33], P=18, hq=4, hk=2, D=64, spare_rows=9, stride_pad=64)
    check_attend(R, c, "spare")
    check_attend(R, c, "without lse", lse=False)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_unseen_tokens_of_the_call_have_no_influence(rope_gpu, dtype, bad, D):
    """NaN and infinities in the keys and values of later tokens of the same sequence leave earlier rows alone."""
    for new, own, P in (([6, 40], [50, 40], 0), ([150, 3], [150, 20], 70)):
        c = attend_case(11, dtype, new, own, P=P, hq=4, hk=2, D=D)
        clean = attend_reference(c)
        for b in range(2):
            j = own[b] - 1  # the last token
            c["k"][c["table"][b, j // 16], :, j % 16] = bad
            c["v"][c["table"][b, j // 16], :, j % 16] = bad
        last = {int(c["starts"][1]) - 1, int(c["starts"][2]) - 1}
        rows = [t for t in range(c["T"]) if t not in last]
        for case in (c, widened(c)):
            out, lse = run_attend(R, case)
            assert_close(out[rows], clean[0][rows], clean[2][rows], "out")
            assert_close(lse[rows], clean[1][rows], clean[3][rows], "lse")
            if bad != bad:
                assert torch.isnan(out[list(last)]).all()
            assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_large_scores(rope_gpu, dtype):
    """Scores far apart (the maximum moves by thousands within a row) and a row led by one key."""
    check_attend(R, attend_case(12, dtype, [1, 20, 1], [200, 150, 300], P=140, hq=4, hk=2, D=64, q_scale=60.0), "large")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_lowest_values(rope_gpu, dtype):
    """Queries and keys of the type's extremes: scores at or beyond the ends of binary32 where the type reaches them."""
    c = attend_case(13, dtype, [1, 1], [40, 8], hq=2, hk=1, D=32)
    c["q"][0] = 0
    c["q"][1] = torch.finfo(dtype).tiny
    check_attend(R, c, "tiny")


@pytest.mark.parametrize("new", [[1, 2], [60, 33]])
def test_pages_outside_the_cache_are_unseen(rope_gpu, new):
    for dtype in DTYPES:
        c = attend_case(14, dtype, new, [60, 50], P=40, hq=4, hk=2, D=64)
        c["table"][0, 1] = -3
        c["table"][1, 0] = c["k"].shape[0]
        c["prefix"][1] = 1 << 50
        ro, rl, to, tl = attend_reference(c)
        R.get_device_error()
        for case in (c, widened(c)):
            out, lse = run_attend(R, case)
            assert R.get_device_error() == R.ROPE_DEVICE_SLOT_OUT_OF_RANGE
            assert_close(out, ro, to, "out")
            assert_close(lse, rl, tl, "lse")


def test_sequences_past_their_pages(rope_gpu):
    for dtype in DTYPES:
        c = attend_case(15, dtype, [1, 1], [64, 20], P=0, hq=4, hk=2, D=64, spare_pages=0)
        c["lens"][0] = 64 + 1000
        R.get_device_error()
        out, lse = run_attend(R, c)
        assert R.get_device_error() == R.ROPE_DEVICE_SLOT_OUT_OF_RANGE
        c["lens"][0] = 64
        ro, rl, to, tl = attend_reference(c)
        assert_close(out, ro, to, "out")


def test_repeated_calls_are_bit_identical(rope_gpu):
    for dtype in DTYPES:
        for new in ([1, 1, 7], [20, 33, 7]):
            c = attend_case(16, dtype, new, [900, 33, 200], P=500, hq=8, hk=2, D=128)
            for case in (c, widened(c)):
                a, b = run_attend(R, case), run_attend(R, case)
                assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("bad", [None, float("nan")])
def test_joins_of_many_rows(rope_gpu, dtype, bad):
    """So many rows that a joining warp takes several; the last key of each sequence, which only its last row sees,
    may be NaN."""
    c = attend_case(17, dtype, [700, 0, 1900], [1300, 0, 1900], P=9, hq=8, hk=2, D=64)
    out, lse, tol, ltol = attend_reference(c)
    keep = torch.ones(c["T"], dtype=torch.bool)
    if bad is not None:
        for b, n in ((0, 1300), (2, 1900)):
            c["k"][c["table"][b, (n - 1) // 16], :, (n - 1) % 16] = bad
            keep[int(c["starts"][b + 1]) - 1] = False
    got, got_lse = run_attend(R, c)
    assert_close(got[keep], out[keep], tol[keep], "out")
    assert_close(got_lse[keep], lse[keep], ltol[keep], "lse")
    if bad is not None:
        assert torch.isnan(got[~keep]).all()
    assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("hq,hk,D", [(4, 2, 64), (8, 1, 128), (16, 2, 96)])
def test_units_of_every_length(rope_gpu, dtype, hq, hk, D):
    """Own lengths of one key to several tiles side by side: shares that begin or end within a unit's cost."""
    own = [1 + (i * 61) % 413 for i in range(47)]
    for P in (0, 5):
        check_attend(R, attend_case(18, dtype, [1] * 47, own, P=P, hq=hq, hk=hk, D=D), "lengths")
    new = [min(n, 1 + (i * 5) % 40) for i, n in enumerate(own)]
    check_attend(R, attend_case(19, dtype, new, own, P=0, hq=hq, hk=hk, D=D), "lengths")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prefix_behind_many_rows(rope_gpu, dtype, D):
    """A prefix whose launch takes tall units, ragged own keys after it."""
    n = 50
    new = [1 + (i % 9 == 4) for i in range(n)]
    own = [new[i] + (i * 29) % 70 for i in range(n)]
    check_attend(R, attend_case(20, dtype, new, own, P=2900 if D == 64 else 1500, hq=16, hk=2, D=D, bs=32), "long prefix")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("new,own", [([1, 1, 2], [20, 1, 30]), ([9, 3, 60], [40, 3, 60])])
def test_short_sequences_with_bad_values(rope_gpu, dtype, bad, new, own):
    """Calls that need no joining launch: rows that a NaN or infinite key or value of another row's sight reaches in
    the products are computed again, by the kernel that finished them."""
    for bs, D in ((16, 64), (7, 256)):
        c = attend_case(21, dtype, new, own, P=0, hq=8, hk=2, D=D, bs=bs)
        clean = attend_reference(c)
        last = torch.zeros(c["T"], dtype=torch.bool)
        for b, n in enumerate(own):
            if new[b] > 1:
                c["k"][c["table"][b, (n - 1) // bs], :, (n - 1) % bs] = bad
                c["v"][c["table"][b, (n - 1) // bs], :, (n - 1) % bs] = bad
                last[int(c["starts"][b + 1]) - 1] = True
        for case in (c, widened(c)):
            n = R.launch_count()
            out, lse = run_attend(R, case)
            launches = R.launch_count() - n
            assert_close(out[~last], clean[0][~last], clean[2][~last], "out")
            assert_close(lse[~last], clean[1][~last], clean[3][~last], "lse")
            assert launches == (1 if case is c else 2)
            assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("D", [128, 160])
def test_short_prompts_with_bad_values(rope_gpu, dtype, D):
    """Many short prompts: tall units, none of them split, one launch."""
    n = 40
    own = [14 + (i * 7) % 90 for i in range(n)]
    new = [min(own[i], 8 + i % 13) for i in range(n)]
    c = attend_case(22, dtype, new, own, P=0, hq=16, hk=2, D=D)
    clean = attend_reference(c)
    last = torch.zeros(c["T"], dtype=torch.bool)
    for b in range(0, n, 3):
        j = own[b] - 1
        c["k"][c["table"][b, j // 16], :, j % 16] = float("nan")
        c["v"][c["table"][b, j // 16], :, j % 16] = float("inf")
        last[int(c["starts"][b + 1]) - 1] = True
    before = R.launch_count()
    out, lse = run_attend(R, c)
    assert R.launch_count() - before == 1
    assert_close(out[~last], clean[0][~last], clean[2][~last], "out")
    assert_close(lse[~last], clean[1][~last], clean[3][~last], "lse")
    assert torch.isnan(out[last]).all()
    assert R.get_device_error() == 0
