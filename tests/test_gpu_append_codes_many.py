"""Append of many tokens to a paged cache of 8-bit codes: batches that are padded to a size of their own, against the
64-bit reference (bounds: tests/codes_ref.py), and large ones, equal to the same tokens in several calls."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import bytes_of, codes_append_case
from test_gpu_append_codes import check

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def padded(c, rows):
    """The batch with tokens that have no slot behind it, `rows` in all."""
    more = rows - c["q"].shape[0]
    g = torch.Generator().manual_seed(99)
    for n in "qkv":
        c[n] = torch.cat([c[n], torch.randn(more, c[n].shape[1], generator=g).to(c["dtype"])])
    c["pos"] = torch.cat([c["pos"], torch.zeros(*c["pos"].shape[:-1], more, dtype=torch.int64)], -1)
    c["slots"] = torch.cat([c["slots"], torch.full((more,), -1, dtype=torch.int64)])
    return c


NEW, HELD = [1, 1, 5, 40, 0, 16, 131, 1], [0, 15, 3, 9, 4, 16, 0, 63]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("bs,S", [(1, 1), (16, 1), (16, 16), (12, 3), (17, 17), (64, 2), (128, 1)])
def test_pages_and_scale_blocks(rope_gpu, dtype, bs, S):
    check(padded(codes_append_case(1, dtype, NEW, HELD, bs, S, neox=bs != 16, scale=4.0), 1030), "pages")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D,Rr", [(32, 32), (96, 96), (128, 64), (256, 64), (512, 512)])
@pytest.mark.parametrize("neox", [True, False])
def test_heads(rope_gpu, dtype, D, Rr, neox):
    """Of so many heads that a warp looks for runs in a window of several tokens."""
    c = codes_append_case(2, dtype, [3, 1, 20, 37, 2], [0, 7, 30, 11, 0], 16, 2, hq=1, hk=16, hv=17, D=D, R=Rr, neox=neox)
    check(padded(c, 1025), "heads")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("sections,mode", [((8, 12, 12), 0), ((8, 8, 8, 8), 0), ((8, 12, 12), 1)])
def test_mrope(rope_gpu, dtype, sections, mode):
    c = codes_append_case(5, dtype, [9, 30, 1], [2, 0, 5], 16, 2, D=64, sections=list(sections), cache_mode=mode, neox=mode == 0)
    check(padded(c, 1025), "mrope")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_ends_and_bad_positions(rope_gpu, dtype):
    """Zeros, the type's largest and smallest values, NaN, infinities; positions outside the table at the beginning, in
    the middle and at the end of runs, and in a whole one."""
    c = codes_append_case(7, dtype, [16, 16, 16, 16, 3, 16, 20], [0, 0, 0, 0, 5, 0, 0], 16, 1, D=64, R=32, max_seq=50)
    info = torch.finfo(dtype)
    v = c["v"]
    v[:16] = 0
    v[16:32] = info.max
    v[32:48] = info.tiny
    v[48:64, ::3] = float("nan")
    v[48:64, 1::3] = float("inf")
    v[64:67] = 0
    c["k"][3, 3] = float("-inf")
    c = padded(c, 1100)
    check(c, "ends")
    check(c, "no query", with_query=False)
    c["pos"][[0, 20, 47, 64, 65, 66, 83, 1099]] = torch.tensor([50, -1, 1 << 40, 50, 51, 52, -3, 60])
    check(c, "positions")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D,hk,bs,S,neox", [(128, 8, 16, 1, True), (128, 8, 64, 1, True), (64, 4, 16, 4, False), (256, 2, 128, 2, True),
                                            (96, 3, 48, 1, False), (512, 16, 16, 1, True), (16, 1, 17, 17, True)])
def test_as_in_several_calls(rope_gpu, dtype, D, hk, bs, S, neox):
    """Thousands of tokens of prompts and single ones, once in one call and once in calls of up to 1024 tokens."""
    if dtype != torch.float32:  # (16-bit heads are of multiples of 32)
        D = max(D, 32)
    g = torch.Generator().manual_seed(D + bs)
    new = torch.randint(1, 700, (16,), generator=g).tolist() + [1] * 900 + torch.randint(1, 6, (300,), generator=g).tolist()
    new += [1000, 1024] + ([] if D > 128 else torch.randint(1, 1000, (20 if D > 16 else 60,), generator=g).tolist())
    held = torch.randint(0, 100, (len(new),), generator=g).tolist()
    c = codes_append_case(3, dtype, new, held, bs, S, hq=hk, hk=hk, D=D, R=D if D != 256 else 64, neox=neox, scale=3.0)
    d = {n: c[n].cuda() for n in ("q", "k", "v", "pos", "table", "slots")}
    pieces, at, first = [], 0, 0
    for n in new:
        if at + n - first > 1024:
            pieces.append((first, at))
            first = at
        at += n
    pieces.append((first, at))
    results = []
    for cuts in ([(0, at)], pieces):
        caches = [bytes_of(c[n]).cuda().view(c[n].dtype) for n in ("kc", "vc", "ks", "vs")]
        qo = torch.full_like(d["q"], float("nan"))
        for a, b in cuts:
            R.append_paged_kv_8bit(d["pos"][a:b], d["q"][a:b], d["k"][a:b], d["v"][a:b], d["table"], d["slots"][a:b],
                                   *caches, D, is_neox=neox, query_out=qo[a:b])
        results.append([qo.view(torch.uint8)] + [bytes_of(x) for x in caches])
    for one, several, n in zip(*results, ("q", "k_cache", "v_cache", "k_scale", "v_scale")):
        assert torch.equal(one, several), n
    assert R.get_device_error() == 0
