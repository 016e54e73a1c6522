"""Refusals of every kind of bad argument by the operators on a cache of 8-bit codes and on its pages.  No call here
launches a kernel; the device pointers are fakes that nothing reads."""
import ctypes

import pytest
import torch

import transformer_rope_positional_gb300 as R
from transformer_rope_positional_gb300 import _capi as C
from transformer_rope_positional_gb300 import build as B

FAKE = 0x100000
BAD, NULL, OK = C.ROPE_ERR_PARAM_INVALID, C.ROPE_ERR_PARAM_NULLPTR, C.ROPE_OK
T, D, HQ, HK, NB, BS, S = 6, 64, 4, 2, 3, 4, 2


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def d(dtype, shape, ptr):
    return ctypes.byref(C.describe(ptr, dtype, shape))


def M(i):
    return i << 20


def call(fn, good, over):
    assert not set(over) - set(good)
    return fn(*dict(good, **over).values(), None)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _append(lib, **over):
    good = {"positions": d(C.I64, (T,), M(1)), "query": d(C.F16, (T, HQ * D), M(2)), "key": d(C.F16, (T, HK * D), M(3)),
            "value": d(C.F16, (T, HK * D), M(4)), "table": d(C.F16, (10, 32), M(5)), "slots": d(C.I64, (T,), M(6)),
            "query_out": d(C.F16, (T, HQ * D), M(7)), "k_cache": d(C.F8E4M3, (NB, HK, BS, D), M(8)),
            "v_cache": d(C.F8E4M3, (NB, HK, BS, D), M(9)), "k_scale": d(C.E8M0, (NB, HK, S), M(10)),
            "v_scale": d(C.E8M0, (NB, HK, S), M(11)), "D": D, "R": 32, "neox": 1, "section": None, "n": 0, "mode": 0,
            "qs": 0, "ks": 0, "vs": 0}
    return call(lib.rope_append_paged_kv_8bit, good, over)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, NULL) for k in ("positions", "key", "value", "table", "slots", "k_cache", "v_cache", "k_scale", "v_scale", "query")],
    ({"k_cache": d(C.F8E4M3, (NB, HK, BS, D), 0)}, NULL), ({"v_scale": d(C.E8M0, (NB, HK, S), 0)}, NULL),
    ({"k_cache": d(C.F16, (NB, HK, BS, D), M(8))}, BAD), ({"v_cache": d(C.U8, (NB, HK, BS, D), M(9))}, BAD),
    ({"k_scale": d(C.U8, (NB, HK, S), M(10))}, BAD), ({"k_scale": d(C.F32, (NB, HK, S), M(10))}, BAD),
    ({"k_scale": d(C.E8M0, (NB, HK), M(10))}, BAD), ({"k_scale": d(C.E8M0, (NB, HK, 3), M(10))}, BAD),
    ({"k_scale": d(C.E8M0, (NB, HK, 0), M(10))}, BAD), ({"k_scale": d(C.E8M0, (NB, HK, 2 * BS), M(10))}, BAD),
    ({"k_scale": d(C.E8M0, (NB, HK, BS), M(10))}, BAD),  # another number of blocks than the values'
    ({"k_scale": d(C.E8M0, (NB + 1, HK, S), M(10))}, BAD), ({"v_scale": d(C.E8M0, (NB, HK + 1, S), M(11))}, BAD),
    ({"key": d(C.F8E4M3, (T, HK * D), M(3))}, BAD), ({"query": d(C.F8E4M3, (T, HQ * D), M(2))}, BAD),
    ({"D": 544}, BAD), ({"D": 48}, BAD), ({"R": 96}, BAD), ({"qs": 8}, BAD),
    ({"k_cache": d(C.F8E4M3, (NB, HK, BS, D), M(8) + 8)}, BAD),
    # what is written shares no memory with anything else
    ({"k_scale": d(C.E8M0, (NB, HK, S), M(8))}, BAD), ({"v_scale": d(C.E8M0, (NB, HK, S), M(10) + 4)}, BAD),
    ({"k_scale": d(C.E8M0, (NB, HK, S), M(3))}, BAD), ({"v_scale": d(C.E8M0, (NB, HK, S), M(6) + 8)}, BAD),
    ({"v_cache": d(C.F8E4M3, (NB, HK, BS, D), M(8) + 512)}, BAD), ({"k_cache": d(C.F8E4M3, (NB, HK, BS, D), M(7))}, BAD)])
def test_append_refusals(lib, over, status):
    n = lib.rope_launch_count()
    assert _append(lib, **over) == status
    assert lib.rope_launch_count() == n


def test_append_of_no_tokens(lib):
    empty = {k: d(C.F16, (0, w * D), 0) for k, w in (("query", HQ), ("key", HK), ("value", HK), ("query_out", HQ))}
    assert _append(lib, positions=d(C.I64, (0,), 0), slots=d(C.I64, (0,), 0), **empty) == OK
    # a scale that cannot be is refused all the same
    assert _append(lib, positions=d(C.I64, (0,), 0), slots=d(C.I64, (0,), 0), k_scale=d(C.E8M0, (NB, HK, 3), M(10)), **empty) == BAD


def test_codes_are_no_data_of_the_other_operators(lib):
    assert lib.rope_append_paged_kv(d(C.I64, (T,), M(1)), None, d(C.F16, (T, HK * D), M(3)), d(C.F16, (T, HK * D), M(4)),
                                    d(C.F16, (10, 32), M(5)), d(C.I64, (T,), M(6)), None, d(C.F8E4M3, (NB, HK, BS, D), M(8)),
                                    d(C.F8E4M3, (NB, HK, BS, D), M(9)), D, 32, 1, None, 0, 0, 0, 0, 0, None) == BAD


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
BATCH, W = 3, 5


def _attend(lib, **over):
    good = {"query": d(C.BF16, (T, HQ * D), M(1)), "qs": 0, "k_cache": d(C.F8E4M3, (NB, HK, BS, D), M(2)),
            "v_cache": d(C.F8E4M3, (NB, HK, BS, D), M(3)), "k_scale": d(C.E8M0, (NB, HK, S), M(4)),
            "v_scale": d(C.E8M0, (NB, HK, S), M(5)), "table": d(C.I64, (BATCH, W), M(6)), "lens": d(C.I64, (BATCH,), M(7)),
            "starts": d(C.I64, (BATCH + 1,), M(8)), "prefix": d(C.I64, (2,), M(9)), "P": 7, "scale": 0.125,
            "out": d(C.BF16, (T, HQ * D), M(10)), "lse": d(C.F32, (T, HQ), M(11)), "ws": M(512), "bytes": 1 << 30}
    return call(lib.rope_paged_attention_8bit, good, over)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, NULL) for k in ("query", "k_cache", "v_cache", "k_scale", "v_scale", "table", "lens", "starts", "out", "prefix", "ws")],
    ({"k_scale": d(C.E8M0, (NB, HK, S), 0)}, NULL), ({"v_cache": d(C.F8E4M3, (NB, HK, BS, D), 0)}, NULL),
    ({"k_cache": d(C.BF16, (NB, HK, BS, D), M(2))}, BAD), ({"query": d(C.F8E4M3, (T, HQ * D), M(1))}, BAD),
    ({"out": d(C.F16, (T, HQ * D), M(10))}, BAD), ({"v_scale": d(C.U8, (NB, HK, S), M(5))}, BAD),
    ({"k_scale": d(C.E8M0, (NB, HK, 3), M(4))}, BAD), ({"v_scale": d(C.E8M0, (NB, HK, 4), M(5))}, BAD),
    ({"k_scale": d(C.E8M0, (NB, 1, S), M(4))}, BAD), ({"k_scale": d(C.E8M0, (NB, HK, S, 1), M(4))}, BAD),
    ({"P": -1}, BAD), ({"P": 9}, BAD), ({"scale": 0.0}, BAD), ({"scale": float("nan")}, BAD), ({"bytes": 255}, BAD),
    ({"ws": M(512) + 8}, BAD), ({"ws": M(4) - 256}, BAD), ({"out": d(C.BF16, (T, HQ * D), M(5))}, BAD),
    ({"lse": d(C.F32, (T, HQ), M(4))}, BAD), ({"qs": HQ * D + 4}, BAD)])
def test_attention_refusals(lib, over, status):
    n = lib.rope_launch_count()
    assert _attend(lib, **over) == status
    assert lib.rope_launch_count() == n


def test_attention_workspace(lib):
    n = ctypes.c_int64()
    f = lib.rope_paged_attention_8bit_workspace
    assert f(4, 32, 8, 128, C.BF16, 0, None) == NULL
    for args in ((4, 32, 5, 128, C.BF16, 0), (4, 32, 8, 100, C.BF16, 0), (4, 32, 8, 544, C.BF16, 0), (4, 32, 8, 128, C.F8E4M3, 0),
                 (-1, 32, 8, 128, C.BF16, 0), (4, 32, 8, 128, C.BF16, -1)):
        assert f(*args, ctypes.byref(n)) == BAD
    for dt in (C.F32, C.F16, C.BF16):
        for D_ in (32, 128, 256, 512):
            for P in (0, 100):
                assert f(17, 8, 2, D_, dt, P, ctypes.byref(n)) == OK and n.value >= 256


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
ROWS = 4


def _rearrange(lib, **over):
    good = {"table": d(C.I64, (BATCH, W), M(1)), "lens": d(C.I64, (BATCH,), M(2)), "refs": d(C.I32, (NB,), M(3)),
            "parents": d(C.I64, (ROWS,), M(4)), "room": d(C.I64, (ROWS,), M(5)), "new_table": d(C.I64, (ROWS, W + 1), M(6)),
            "new_lens": d(C.I64, (ROWS,), M(7)), "new_refs": d(C.I32, (NB,), M(8)), "src": d(C.I64, (ROWS,), M(9)),
            "dst": d(C.I64, (ROWS,), M(10)), "counts": d(C.I64, (2,), M(11)), "bs": 16, "P": 0}
    return call(lib.rope_rearrange_sequences, good, over)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, NULL) for k in ("table", "lens", "refs", "parents", "new_table", "new_lens", "new_refs", "src", "dst", "counts")],
    ({"table": d(C.I64, (BATCH, W), 0)}, NULL), ({"room": d(C.I64, (ROWS,), 0)}, NULL),
    ({"refs": d(C.I64, (NB,), M(3))}, BAD), ({"table": d(C.I32, (BATCH, W), M(1))}, BAD), ({"lens": d(C.I64, (BATCH, 1), M(2))}, BAD),
    ({"table": d(C.I64, (BATCH + 1, W), M(1))}, BAD), ({"parents": d(C.I64, (ROWS + 1,), M(4))}, BAD),
    ({"room": d(C.I64, (ROWS - 1,), M(5))}, BAD), ({"new_refs": d(C.I32, (NB + 1,), M(8))}, BAD),
    ({"counts": d(C.I64, (1,), M(11))}, BAD), ({"bs": 0}, BAD), ({"P": -1}, BAD), ({"bs": 1 << 31}, BAD),
    ({"refs": d(C.I32, (0,), M(3)), "new_refs": d(C.I32, (0,), M(8))}, BAD), ({"lens": d(C.I64, (BATCH,), M(2) + 4)}, BAD),
    ({"new_table": d(C.I64, (ROWS, W), M(1))}, BAD), ({"new_lens": d(C.I64, (ROWS,), M(2))}, BAD),
    ({"src": d(C.I64, (ROWS,), M(10) + 8)}, BAD), ({"new_refs": d(C.I32, (NB,), M(3) + 4)}, BAD),
    ({"dst": d(C.I64, (ROWS,), M(4))}, BAD)])
def test_rearrange_refusals(lib, over, status):
    n = lib.rope_launch_count()
    assert _rearrange(lib, **over) == status
    assert lib.rope_launch_count() == n


def test_rearrange_most_rows(lib):
    r = 8193
    over = {k: d(C.I64, (r,), M(20 + i)) for i, k in enumerate(("parents", "room", "new_lens", "src", "dst"))}
    assert _rearrange(lib, new_table=d(C.I64, (r, W), M(40)), **over) == BAD


def _compact(lib, **over):
    good = {"table": d(C.I64, (BATCH, W), M(1)), "lens": d(C.I64, (BATCH,), M(2)), "refs": d(C.I32, (NB,), M(3)),
            "prefix": d(C.I64, (2,), M(4)), "new_table": d(C.I64, (BATCH, W), M(5)), "new_refs": d(C.I32, (NB,), M(6)),
            "new_prefix": d(C.I64, (2,), M(7)), "src": d(C.I64, (1,), M(8)), "dst": d(C.I64, (1,), M(9)),
            "counts": d(C.I64, (2,), M(10)), "bs": 16, "P": 20}
    return call(lib.rope_compact_pages, good, over)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, NULL) for k in ("table", "lens", "refs", "prefix", "new_table", "new_refs", "new_prefix", "src", "dst", "counts")],
    ({"new_refs": d(C.I32, (NB,), 0)}, NULL), ({"new_table": d(C.I64, (BATCH, W + 1), M(5))}, BAD),
    ({"new_prefix": d(C.I64, (1,), M(7))}, BAD), ({"prefix": d(C.I32, (2,), M(4))}, BAD), ({"src": d(C.I64, (0,), M(8))}, BAD),
    ({"dst": d(C.I64, (2,), M(9))}, BAD), ({"P": 33}, BAD), ({"bs": -1}, BAD), ({"counts": d(C.I64, (2,), M(8))}, BAD),
    ({"new_table": d(C.I64, (BATCH, W), M(1) + 8)}, BAD), ({"new_prefix": d(C.I64, (2,), M(4) + 8)}, BAD),
    ({"new_refs": d(C.I32, (NB,), M(2))}, BAD), ({"dst": d(C.I64, (1,), M(8))}, BAD)])
def test_compact_refusals(lib, over, status):
    n = lib.rope_launch_count()
    assert _compact(lib, **over) == status
    assert lib.rope_launch_count() == n


def _copy(lib, src, dst, count, tensors):
    a = (C.RopeTensor * max(1, len(tensors)))(*[C.describe(p, t, s) for t, s, p in tensors])
    return lib.rope_copy_pages(src, dst, count, a, len(tensors), None)


def test_copy_refusals(lib):
    n = lib.rope_launch_count()
    src, dst, one = d(C.I64, (3,), M(1)), d(C.I64, (3,), M(2)), (C.U8, (8, 32), M(4))
    for s, t in ((None, dst), (src, None), (d(C.I64, (3,), 0), dst)):
        assert _copy(lib, s, t, None, [one]) == NULL
    assert lib.rope_copy_pages(src, dst, None, None, 1, None) == NULL
    assert _copy(lib, src, dst, None, [(C.U8, (8, 32), 0)]) == NULL
    for bad in ([(C.U8, (8, 32), M(4)), (C.U8, (9, 32), M(5))], [one, (C.U8, (8, 4), M(4) + 255)], [(C.U8, (8, 32), M(1) - 250)],
                [(C.F32, (8, 32), M(4) + 2)], [(8, (8, 32), M(4))], [(-1, (8, 32), M(4))], [(C.U8, (0, 32), M(4))], [(C.U8, (-8, 32), M(4))]):
        assert _copy(lib, src, dst, None, bad) == BAD, bad
    assert _copy(lib, src, d(C.I64, (2,), M(2)), None, [one]) == BAD
    assert _copy(lib, src, dst, d(C.I64, (0,), M(3)), [one]) == BAD
    assert _copy(lib, src, dst, d(C.I32, (1,), M(3)), [one]) == BAD
    assert _copy(lib, d(C.I32, (3,), M(1)), dst, None, [one]) == BAD
    # nothing to do
    assert _copy(lib, src, dst, None, []) == OK
    assert _copy(lib, d(C.I64, (0,), 0), d(C.I64, (0,), 0), None, [one]) == OK
    assert _copy(lib, src, dst, None, [(C.U8, (8, 0), 0)]) == OK
    assert lib.rope_launch_count() == n


def test_python_refuses_tensors_that_are_not_on_a_gpu(lib):
    i = torch.zeros(4, dtype=torch.int64)
    t = torch.zeros(4, 4, dtype=torch.int64)
    r = torch.zeros(9, dtype=torch.int32)
    with pytest.raises(ValueError):
        R.copy_pages(i, i, [r])
    with pytest.raises(ValueError):
        R.rearrange_sequences(t, i, r, i, t, i, r, i, i, i, 16)
    with pytest.raises(ValueError):
        R.compact_pages(t, i, r, t, r, i, i, i, 16)
    k = torch.zeros(2, 1, 4, 32, dtype=torch.uint8).view(torch.float8_e4m3fn)
    z = torch.zeros(2, 1, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        R.paged_attention_8bit(x, k, k, z, z, t, i, i, x)
    with pytest.raises(ValueError):
        R.append_paged_kv_8bit(i, x, x, x, x, i, k, k, z, z, 32)
