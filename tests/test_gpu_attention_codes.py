"""Attention over a paged cache of 8-bit codes, against a float64 reference (bounds: tests/serving_ref.py).

Cache rows that hold no token are NaN codes, and scales without tokens are NaN, so a row that leaks shows."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import bytes_of, coded_case, e8m0, run_coded, values_of
from serving_ref import assert_close, attend_reference, widened

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def check(c, what="", **kw):
    """The case as it is and with a wide table: which kernel runs goes by how many keys there may be."""
    ro, rl, to, tl = attend_reference(c)
    T = int(c["starts"][-1])
    first = None
    for case in (c, widened(c)):
        out, lse = run_coded(R, case, **kw)
        assert_close(out[:T], ro[:T], to[:T], what + " out")
        if lse is not None:
            assert_close(lse[:T], rl[:T], tl[:T], what + " lse")
        assert torch.equal(out[T:].view(torch.int16), torch.full_like(out[T:].view(torch.int16), 0x7FA5)), what
        assert R.get_device_error() == 0
        first = first or (out, lse)
    return first


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (8, 2), (5, 1), (14, 2), (32, 1)])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 256])
def test_single_tokens(rope_gpu, dtype, hq, hk, D):
    own = [1, 2, 15, 16, 17, 63, 64, 65, 130]
    check(coded_case(1, dtype, [1] * len(own), own, hq=hq, hk=hk, D=D), "decode")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [16, 48, 224, 288, 512])
def test_other_head_sizes(rope_gpu, dtype, D):
    if dtype != torch.float32 and D in (16, 48):
        pytest.skip("16-bit heads are multiples of 32")
    check(coded_case(2, dtype, [1, 3, 2], [40, 3, 70], P=37, hq=4, hk=2, D=D), "head size")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("P", [0, 1, 16, 37, 128, 129, 300])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [5, 1, 3, 0], [70, 2, 0, 33]])
def test_prefix_and_new_tokens(rope_gpu, dtype, P, new):
    own = [new[0] + 9, new[1], new[2] + 130, new[3] + 64]
    check(coded_case(3, dtype, new, own, P=P, hq=8, hk=2, D=64, S=2), "prefix")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("bs,S", [(1, 1), (3, 3), (7, 1), (12, 4), (17, 17), (64, 4), (128, 1), (200, 100)])
def test_pages_and_scale_blocks(rope_gpu, dtype, bs, S):
    check(coded_case(4, dtype, [1, 4, 20], [260, 4, 77], P=53, hq=4, hk=2, D=128, bs=bs, S=S), "pages")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,own,P", [([300], [300], 0), ([129, 257], [400, 257], 0), ([260, 1, 140], [260, 600, 300], 150)])
def test_prompts(rope_gpu, dtype, D, new, own, P):
    check(coded_case(5, dtype, new, own, P=P, hq=4, hk=1, D=D, bs=32, S=2), "prompt")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_many_short_sequences_behind_a_prefix(rope_gpu, dtype):
    n = 41
    new = [1 + (i % 3 == 0) for i in range(n)]
    own = [new[i] + (i * 37) % 90 for i in range(n)]
    check(coded_case(6, dtype, new, own, P=700, hq=8, hk=2, D=64), "many")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_long_keys_for_few_rows(rope_gpu, dtype):
    """The key axis is split over the device and joined."""
    check(coded_case(7, dtype, [1, 2], [3000, 1], P=0, hq=2, hk=1, D=64), "long")
    check(coded_case(8, dtype, [1, 1], [5, 9], P=2500, hq=2, hk=1, D=128, S=16), "long prefix")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("P", [0, 40])
def test_rows_without_keys(rope_gpu, dtype, P):
    c = coded_case(9, dtype, [4, 0, 3, 2], [4, 0, 3, 2], P=P, hq=4, hk=2, D=64)
    c["lens"] = torch.tensor([2, 0, 30 if P else 1, 0])
    out, lse = check(c, "empty rows")
    assert torch.equal(lse[:2], torch.full((2, 4), float("-inf"))) and not out[:2].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_spare_rows_and_strided_queries(rope_gpu, dtype):
    c = coded_case(10, dtype, [1, 5, 1], [20, 5, 33], P=18, hq=4, hk=2, D=64, spare_rows=9, stride_pad=64)
    check(c, "spare")
    check(c, "without lse", lse=False)
    check(c, "prepared", prepared=True)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("where", ["k_codes", "v_codes", "k_scale", "v_scale"])
@pytest.mark.parametrize("D", [64, 128])
def test_unseen_tokens_of_the_call_have_no_influence(rope_gpu, dtype, where, D):
    """A NaN code or scale of the last token leaves earlier rows alone."""
    for new, own, P in (([6, 40], [50, 40], 0), ([150, 3], [150, 20], 70)):
        c = coded_case(11, dtype, new, own, P=P, hq=4, hk=2, D=D, S=16)
        clean = attend_reference(c)
        for b in range(2):
            j = own[b] - 1
            page = c["table"][b, j // 16]
            if "codes" in where:
                bytes_of(c[where])[page, :, j % 16] = 0x7f
            else:
                bytes_of(c[where])[page, :, j % 16] = 255
        last = {int(c["starts"][1]) - 1, int(c["starts"][2]) - 1}
        rows = [t for t in range(c["T"]) if t not in last]
        for case in (c, widened(c)):
            out, lse = run_coded(R, case)
            assert_close(out[rows], clean[0][rows], clean[2][rows], "out")
            assert_close(lse[rows], clean[1][rows], clean[3][rows], "lse")
            assert torch.isnan(out[list(last)]).all()
            assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_large_scores(rope_gpu, dtype):
    """Scores far apart (the maximum moves by thousands within a row) and a row led by one key."""
    check(coded_case(12, dtype, [1, 20, 1], [200, 150, 300], P=140, hq=4, hk=2, D=64, q_scale=60.0), "large")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("k,v", [(0, 12), (0, -12), (6, 0), (-9, 5)])
def test_units_far_from_one(rope_gpu, dtype, k, v):
    """Keys and values of magnitudes from 2^-12 to 2^12, scales of blocks up to 2^6 apart."""
    c = coded_case(13, dtype, [1, 20], [200, 150], P=40, hq=4, hk=2, D=64, S=4, extreme={"k": k, "v": v},
                   q_scale=2.0 ** -k)
    check(c, "units")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_scales_at_the_ends(rope_gpu, dtype):
    """Blocks of zeros with the byte 0 among others; scales whose values leave binary16 and come near binary32's ends:
    the codes they scale are zeros, or the keys are not seen by most rows."""
    c = coded_case(14, dtype, [1, 20], [200, 150], hq=4, hk=2, D=64, S=16)
    for n in ("k", "v"):
        for b, j in ((0, 3), (0, 100), (1, 7), (1, 64)):
            page = c["table"][b, j // 16]
            bytes_of(c[n + "_codes"])[page, :, j % 16] = 0
            bytes_of(c[n + "_scale"])[page, :, j % 16] = 0 if j % 2 else 254
        c[n] = values_of(c[n + "_codes"], c[n + "_scale"])
    check(c, "ends")


def test_pages_outside_the_cache(rope_gpu):
    """Keys of such a page are keys that no row sees, and the device error says so."""
    for dtype in DTYPES:
        c = coded_case(15, dtype, [1, 30, 3], [100, 64, 40], hq=4, hk=2, D=64)
        c["table"][0, 2] = c["k"].shape[0]
        c["table"][1, 1] = -1
        c["table"][2, 0] = 1 << 50
        ro, rl, to, tl = attend_reference(c)
        out, lse = run_coded(R, c)
        assert R.get_device_error() == R.ROPE_DEVICE_SLOT_OUT_OF_RANGE
        assert_close(out, ro, to, "out")
        assert_close(lse, rl, tl, "lse")


def test_as_the_attention_over_the_same_values(rope_gpu):
    """A cache of the data's type that holds the same values gives the same to two roundings of the output."""
    for dtype in (torch.float16, torch.bfloat16):
        c = coded_case(16, dtype, [1, 40, 1], [500, 300, 64], P=64, hq=8, hk=2, D=128, fill=0.0)
        for n in ("k", "v"):
            c[n + "_scale"] = e8m0(torch.where(bytes_of(c[n + "_scale"]) == 255, torch.tensor(127, dtype=torch.uint8), bytes_of(c[n + "_scale"])))
            c[n] = values_of(c[n + "_codes"], c[n + "_scale"])
        out, lse = run_coded(R, c)
        from serving_ref import run_attend
        other, lse2 = run_attend(R, dict(c, k=c["k"].to(dtype), v=c["v"].to(dtype)))
        ro, rl, to, tl = attend_reference(c)
        assert_close(out, other.double(), 2 * to, "out")
        assert_close(lse, lse2.double(), 2 * tl, "lse")
