"""Append to a paged cache with the rotation on the way, against a float64 reference
(bounds: tests/serving_ref.py)."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from guard import Guards
from parity import same_bits
from serving_ref import append_bound, append_case, append_reference, assert_close

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def _run(c, in_place=False, no_query=False, stream=None, prepared=False):
    g = Guards()
    kc, vc = g.put(c["kc"], "k_cache"), g.put(c["vc"], "v_cache")
    fused = not c["q"].is_contiguous() or not c["k"].is_contiguous()
    if fused:  # the column ranges of one buffer
        buf = g.put(torch.cat([c["q"], c["k"], c["v"]], 1), "qkv")
        a, b = c["q"].shape[1], c["q"].shape[1] + c["k"].shape[1]
        q, k, v = buf[:, :a], buf[:, a:b], buf[:, b:]
    else:
        q, k, v = g.put(c["q"], "q"), g.put(c["k"], "k"), g.put(c["v"], "v")
    qo = None if in_place or no_query else g.empty(tuple(c["q"].shape), c["dtype"], "q_out")
    k0, v0, q0 = k.clone(), v.clone(), q.clone()
    call = R.prepare_append_paged_kv if prepared else R.append_paged_kv
    r = call(g.put(c["pos"], "positions"), None if no_query else q, k, v, g.put(c["table"], "table"),
             g.put(c["slots"], "slots"), kc, vc, c["D"], is_neox=c["neox"], mrope_section=c["sections"],
             cache_mode=c["cache_mode"], query_out=qo, stream=stream)
    if prepared:
        r()
    g.check()
    assert same_bits(k, k0) and same_bits(v, v0)
    if not in_place:
        assert same_bits(q, q0)
    return (q if in_place else qo), kc, vc


def _check(c, **kw):
    q, kc, vc = _run(c, **kw)
    rq, rk, rv, skipped = append_reference(c)
    assert not skipped
    if q is not None:
        assert_close(q, rq, append_bound(rq, c["dtype"]), "query")
    assert_close(kc, rk, append_bound(rk, c["dtype"]), "k_cache")
    assert same_bits(vc, rv.to(c["dtype"]))
    # entries that no token owns, and columns that do not rotate, are copied exactly
    owned = torch.zeros(kc.shape[0] * c["bs"], dtype=torch.bool)
    owned[c["slots"][c["slots"] >= 0]] = True
    free = (~owned).view(kc.shape[0], c["bs"])
    assert same_bits(kc.cpu().transpose(1, 2)[free], c["kc"].transpose(1, 2)[free])
    if q is not None:
        tail = q.cpu().reshape(q.shape[0], -1, c["D"])[..., c["R"]:]
        assert same_bits(tail, c["q"].reshape(q.shape[0], -1, c["D"])[..., c["R"]:])
    assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("T,hq,hk,D,R_,bs", [(1, 1, 1, 32, 32, 1), (3, 4, 2, 64, 32, 16), (7, 5, 1, 96, 64, 12),
                                             (33, 8, 2, 128, 128, 17), (19, 4, 4, 256, 64, 32), (5, 3, 3, 160, 96, 7)])
def test_shapes(rope_gpu, dtype, neox, T, hq, hk, D, R_, bs):
    _check(append_case(1, dtype, T, hq, hk, D, R_, bs, neox=neox))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("fused", [True, False])
def test_table_in_32_bits(rope_gpu, dtype, neox, fused):
    _check(append_case(2, dtype, 21, 6, 3, 64, 64, 8, neox=neox, table_dtype=torch.float32, fused=fused))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("sections,mode", [([8, 12, 12], 0), ([8, 12, 12], 1), ([16, 24, 24], 1), ([16, 16, 16, 16], 0),
                                           ([11, 11, 10], 1), ([5, 0, 27], 0)])
def test_mrope(rope_gpu, dtype, neox, sections, mode):
    _check(append_case(3, dtype, 14, 4, 2, 160, 2 * sum(sections), 16, neox=neox, sections=sections, cache_mode=mode))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("fused", [True, False])
def test_in_place_and_without_query(rope_gpu, dtype, neox, fused):
    c = append_case(4, dtype, 18, 4, 2, 96, 32, 16, neox=neox, fused=fused)
    _check(c, in_place=True)
    _check(c, no_query=True)


def test_other_number_of_value_heads_and_large_heads(rope_gpu):
    _check(append_case(5, torch.bfloat16, 9, 4, 2, 64, 64, 16, hv=5))
    _check(append_case(6, torch.bfloat16, 3, 2, 1, 2048, 2048, 2))
    _check(append_case(6, torch.float32, 3, 2, 1, 1024, 512, 2, neox=False))


def test_more_tokens_than_the_grid(rope_gpu):
    _check(append_case(7, torch.bfloat16, 3001, 4, 1, 64, 64, 16, fused=True))


def test_all_padding_and_prepared_and_stream(rope_gpu):
    c = append_case(8, torch.float16, 6, 2, 2, 64, 64, 4, pad_every=1)
    _check(c)
    _check(append_case(9, torch.float16, 6, 2, 2, 64, 64, 4), prepared=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _check(append_case(9, torch.float16, 6, 2, 2, 64, 64, 4))


def test_positions_and_slots_out_of_range(rope_gpu):
    c = append_case(10, torch.float32, 8, 2, 1, 32, 32, 4, pad_every=0)
    c["pos"][2], c["pos"][5] = -1, 97
    c["slots"][6] = c["kc"].shape[0] * 4
    R.get_device_error()
    q, kc, vc = _run(c)
    assert R.get_device_error() == R.ROPE_DEVICE_POSITION_OUT_OF_RANGE | R.ROPE_DEVICE_SLOT_OUT_OF_RANGE
    rq, rk, rv, skipped = append_reference(c)
    assert skipped == [2, 5]
    keep = [t for t in range(8) if t not in skipped]
    assert_close(q[keep], rq[keep], append_bound(rq[keep], torch.float32), "query")
    assert_close(kc, rk, append_bound(rk, torch.float32), "k_cache")
    assert same_bits(vc, rv.float())
    canary = torch.full((64 * 2,), 0x7FA5, dtype=torch.int16)
    for t in skipped:
        assert torch.equal(q[t].cpu().view(torch.int16), canary)


def test_infinities_and_nan_stay_in_their_pairs(rope_gpu):
    c = append_case(11, torch.bfloat16, 4, 2, 1, 64, 32, 4, pad_every=0)
    c["q"][1, 3], c["k"][2, 40], c["v"][0, 7] = float("inf"), float("nan"), float("-inf")
    q, kc, vc = _run(c)
    rq, rk, rv, _ = append_reference(c)
    fine = torch.isfinite(rq)
    assert torch.equal(torch.isfinite(q.cpu()), fine) and int((~fine).sum()) == 2
    assert_close(q.cpu()[fine], rq[fine], append_bound(rq[fine], torch.bfloat16), "query")
    assert torch.equal(torch.isnan(kc.cpu()), torch.isnan(rk))
    assert torch.equal(vc.cpu().double(), rv)
