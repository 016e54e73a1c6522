"""Host side of the serving operators: the frequency formulas, and refusals of every kind of bad argument.
No call here launches a kernel; the device pointers are fakes that nothing reads."""
import ctypes
import math

import pytest
import torch

import transformer_rope_positional_gb300 as R
from transformer_rope_positional_gb300 import _capi as C
from transformer_rope_positional_gb300 import build as B

FAKE = 0x100000
BAD, NULL, OK = C.ROPE_ERR_PARAM_INVALID, C.ROPE_ERR_PARAM_NULLPTR, C.ROPE_OK


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def d(dtype, shape, ptr):
    return ctypes.byref(C.describe(ptr, dtype, shape))


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def _near(got, ref):
    # one power, a few products and a quotient in binary64
    assert got.dtype == torch.float64 and len(got) == len(ref)
    for g, r in zip(got.tolist(), ref):
        assert abs(g - r) <= 1e-14 * abs(r), (g, r)


@pytest.mark.parametrize("dim,base", [(2, 10000.0), (64, 10000.0), (128, 1e6), (96, 500000.0)])
def test_unscaled_linear_base_and_factors(lib, dim, base):
    plain = [base ** (-2 * i / dim) for i in range(dim // 2)]
    inv, scale = R.rope_frequencies(dim, base)
    _near(inv, plain)
    assert scale == 1.0
    inv, scale = R.rope_frequencies(dim, base, {"kind": "none"})
    _near(inv, plain)
    inv, scale = R.rope_frequencies(dim, base, {"kind": "linear", "factor": 4, "attention": 1.5})
    _near(inv, [f / 4 for f in plain])
    assert scale == 1.5
    factors = [1 + 0.25 * i for i in range(dim // 2)]
    _near(R.rope_frequencies(dim, base, {"kind": "factors", "factors": factors})[0],
          [f / w for f, w in zip(plain, factors)])
    if dim > 2:
        b = base * 3.0 ** (dim / (dim - 2))
        _near(R.rope_frequencies(dim, base, {"kind": "base", "factor": 3})[0],
              [b ** (-2 * i / dim) for i in range(dim // 2)])
        # the lowest frequency is stretched by the factor, the highest kept
        inv = R.rope_frequencies(dim, base, {"kind": "base", "factor": 3})[0]
        assert abs(float(inv[-1]) * 3 / plain[-1] - 1) < 1e-12 and float(inv[0]) == 1.0


def test_yarn(lib):
    dim, base, n, f = 128, 10000.0, 4096, 16.0
    inv, scale = R.rope_frequencies(dim, base, {"kind": "yarn", "factor": f, "original_length": n})
    assert abs(scale - (0.1 * math.log(16) + 1)) < 1e-15
    plain = [base ** (-2 * i / dim) for i in range(dim // 2)]
    # i(32) = 20.94..., i(1) = 45.03...: kept up to 20, divided from 46
    lo, hi = 20, 46
    ref = []
    for i, p in enumerate(plain):
        r = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        ref.append(p * (1 - r) + p / f * r)
    _near(inv, ref)
    assert R.rope_frequencies(dim, base, {"kind": "yarn", "factor": 0.5, "original_length": n})[1] == 1.0
    # an original length of a few turns: the ramp has no width at all
    inv, _ = R.rope_frequencies(8, 10000.0, {"kind": "yarn", "factor": 2, "original_length": 1.0})
    _near(inv, [0.5 * 10 ** -i if i else 1.0 for i in range(4)])


def test_wavelength(lib):
    dim, base, n, f = 128, 500000.0, 8192, 8.0
    inv, scale = R.rope_frequencies(dim, base, {"kind": "wavelength", "factor": f, "original_length": n, "low": 1, "high": 4})
    assert scale == 1.0
    ref = []
    for i in range(dim // 2):
        p = base ** (-2 * i / dim)
        t = n * p / (2 * math.pi)
        ref.append(p if t >= 4 else p / f if t <= 1 else p * (t - 1) / 3 + p / f * (4 - t) / 3)
    _near(inv, ref)
    assert ref[0] == 1.0 and ref[-1] == base ** (-126 / 128) / 8


@pytest.mark.parametrize("dim,base,scaling", [
    (0, 1e4, None), (3, 1e4, None), (-2, 1e4, None), (2050, 1e4, None), (64, 0.0, None), (64, -1.0, None),
    (64, math.nan, None), (64, math.inf, None), (64, 1e4, {"kind": "linear"}), (64, 1e4, {"kind": "linear", "factor": -1}),
    (64, 1e4, {"kind": "other"}), (64, 1e4, {"kind": "linear", "factor": 2, "extra": 1}), (64, 1e4, {}),
    (2, 1e4, {"kind": "base", "factor": 2}), (64, 1e4, {"kind": "yarn", "factor": 2}),
    (64, 1.0, {"kind": "yarn", "factor": 2, "original_length": 4096}),
    (64, 1e4, {"kind": "yarn", "factor": 2, "original_length": 4096, "low": 8, "high": 4}),
    (64, 1e4, {"kind": "wavelength", "factor": 2, "original_length": 4096}),
    (64, 1e4, {"kind": "wavelength", "factor": 2, "original_length": 4096, "low": 4, "high": 4}),
    (64, 1e4, {"kind": "factors", "factors": [1.0] * 31}), (64, 1e4, {"kind": "factors", "factors": [0.0] * 32}),
    (64, 1e300, {"kind": "base", "factor": 1e10}), (1 << 60, 1e4, None),
    (64, 1e4, {"kind": "linear", "factor": math.nan}), (64, 1e4, {"kind": "linear", "factor": 2, "attention": -1})])
def test_frequencies_refused(lib, dim, base, scaling):
    with pytest.raises(R.RopeError) as e:
        R.rope_frequencies(dim, base, scaling)
    assert e.value.status == BAD


def test_frequencies_null(lib):
    s = ctypes.c_double()
    assert lib.rope_scaled_frequencies(4, 1e4, None, None, ctypes.byref(s)) == NULL
    buf = (ctypes.c_double * 2)()
    assert lib.rope_scaled_frequencies(4, 1e4, None, buf, None) == NULL
    bad = C.RopeScaling(5, 0, 0, 0, 0, 0)
    assert lib.rope_scaled_frequencies(4, 1e4, ctypes.byref(bad), buf, ctypes.byref(s)) == NULL


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------
def _table(lib, F=32, cos=None, sin=None, positions=None, scale=1.0, freq=None, mode=0, cache=False):
    f = torch.zeros(max(F, 1), dtype=torch.float64) if freq is None else freq
    if cache:
        return lib.rope_scaled_cos_sin_cache(f.data_ptr() if f is not False else None, F, scale, positions, 0, cos, None)
    return lib.rope_scaled_cos_sin(f.data_ptr() if f is not False else None, F, scale, positions, 0, mode, cos, sin, None)


def test_table_refusals(lib):
    n = lib.rope_launch_count()
    good = d(C.F32, (4, 64), FAKE)
    other = d(C.F32, (4, 64), 2 * FAKE)
    assert _table(lib, cos=d(C.F32, (0, 64), 0), cache=True) == OK  # empty: nothing to do
    assert lib.rope_scaled_cos_sin_cache(None, 32, 1.0, None, 0, good, None) == NULL
    assert _table(lib, cos=None, cache=True) == NULL
    assert _table(lib, cos=good, sin=None) == NULL
    assert _table(lib, cos=d(C.F32, (4, 64), 0), cache=True) == NULL
    assert _table(lib, cos=good, sin=d(C.F32, (4, 64), 0)) == NULL
    for F in (0, -1, 1025):
        assert _table(lib, F=F, cos=d(C.F32, (4, max(0, 2 * F)), FAKE), cache=True) == BAD
    assert _table(lib, cos=d(C.F32, (4, 62), FAKE), cache=True) == BAD
    assert _table(lib, cos=d(C.I64, (4, 64), FAKE), cache=True) == BAD
    assert _table(lib, cos=good, scale=math.inf, cache=True) == BAD
    assert _table(lib, cos=good, scale=math.nan, cache=True) == BAD
    assert _table(lib, cos=good, scale=1e300, cache=True) == BAD
    for v in (math.nan, math.inf, 1.1e6):
        assert _table(lib, cos=good, freq=torch.full((32,), v, dtype=torch.float64), cache=True) == BAD
    assert _table(lib, cos=good, sin=d(C.F16, (4, 64), 2 * FAKE)) == BAD
    assert _table(lib, cos=good, sin=d(C.F32, (5, 64), 2 * FAKE)) == BAD
    assert _table(lib, cos=good, sin=d(C.F32, (1, 4, 64), 2 * FAKE)) == BAD
    assert _table(lib, cos=good, sin=other, mode=2) == BAD
    assert _table(lib, cos=good, sin=d(C.F32, (4, 64), FAKE + 16)) == BAD  # they share memory
    assert _table(lib, cos=d(C.F32, (4, 64), FAKE + 2), cache=True) == BAD
    assert _table(lib, cos=good, positions=d(C.I64, (5,), 2 * FAKE), cache=True) == BAD
    assert _table(lib, cos=good, positions=d(C.F32, (4,), 2 * FAKE), cache=True) == BAD
    assert _table(lib, cos=good, positions=d(C.I64, (4,), 0), cache=True) == NULL
    assert _table(lib, cos=good, positions=d(C.I64, (4,), 2 * FAKE + 4), cache=True) == BAD
    assert _table(lib, cos=good, positions=d(C.I64, (4,), FAKE + 1016), cache=True) == BAD  # the table's last bytes
    assert _table(lib, cos=d(C.F32, (1 << 40, 1 << 40, 64), FAKE), cache=True) == BAD
    assert lib.rope_launch_count() == n


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
T, D, HQ, HK, NB, BS = 6, 64, 4, 2, 3, 4


def _append(lib, **over):
    at = {"positions": d(C.I64, (T,), 1 << 20), "query": d(C.F16, (T, HQ * D), 2 << 20),
          "key": d(C.F16, (T, HK * D), 3 << 20), "value": d(C.F16, (T, HK * D), 4 << 20),
          "table": d(C.F16, (10, 32), 5 << 20), "slots": d(C.I64, (T,), 6 << 20),
          "query_out": d(C.F16, (T, HQ * D), 7 << 20), "k_cache": d(C.F16, (NB, HK, BS, D), 8 << 20),
          "v_cache": d(C.F16, (NB, HK, BS, D), 9 << 20), "D": D, "R": 32, "neox": 1, "section": None, "n": 0, "mode": 0,
          "qs": 0, "ks": 0, "vs": 0}
    assert not set(over) - set(at)
    at.update(over)
    if at["section"] is not None:
        at["n"] = len(at["section"])
        at["section"] = (ctypes.c_int64 * len(at["section"]))(*at["section"])
    return lib.rope_append_paged_kv(*at.values(), None)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, NULL) for k in ("positions", "key", "value", "table", "slots", "k_cache", "v_cache")],
    ({"query": None}, NULL),  # an output without an input
    *[({k: d(C.F16, s, 0)}, NULL) for k, s in (("query", (T, HQ * D)), ("key", (T, HK * D)), ("value", (T, HK * D)),
                                                ("table", (10, 32)), ("query_out", (T, HQ * D)),
                                                ("k_cache", (NB, HK, BS, D)), ("v_cache", (NB, HK, BS, D)))],
    ({"positions": d(C.I64, (T,), 0)}, NULL), ({"slots": d(C.I64, (T,), 0)}, NULL),
    ({"positions": d(C.F32, (T,), FAKE)}, BAD), ({"slots": d(C.F32, (T,), FAKE)}, BAD),
    ({"positions": d(C.I64, (T + 1,), FAKE)}, BAD), ({"slots": d(C.I64, (T, 1), FAKE)}, BAD),
    ({"slots": d(C.I64, (T - 1,), FAKE)}, BAD), ({"positions": d(C.I64, (3, T), FAKE)}, BAD),
    ({"query": d(C.BF16, (T, HQ * D), 2 << 20)}, BAD), ({"value": d(C.F32, (T, HK * D), 4 << 20)}, BAD),
    ({"table": d(C.BF16, (10, 32), 5 << 20)}, BAD), ({"k_cache": d(C.F32, (NB, HK, BS, D), 8 << 20)}, BAD),
    ({"key": d(C.I64, (T, HK * D), 3 << 20)}, BAD),
    ({"table": d(C.F16, (10, 64), 5 << 20)}, BAD), ({"table": d(C.F16, (0, 32), 5 << 20)}, BAD),
    ({"D": 48}, BAD), ({"D": 0}, BAD), ({"D": -64}, BAD), ({"D": 4096}, BAD), ({"R": 16}, BAD), ({"R": 96}, BAD),
    ({"R": 0}, BAD), ({"key": d(C.F16, (T, HK * D + 8), 3 << 20)}, BAD), ({"key": d(C.F16, (T + 1, HK * D), 3 << 20)}, BAD),
    ({"query_out": d(C.F16, (T, D), 7 << 20)}, BAD), ({"value": d(C.F16, (T, 3 * D), 4 << 20)}, BAD),
    ({"k_cache": d(C.F16, (NB, HK, BS, D + 32), 8 << 20)}, BAD), ({"v_cache": d(C.F16, (NB, HK, BS + 1, D), 9 << 20)}, BAD),
    ({"k_cache": d(C.F16, (0, HK, BS, D), 8 << 20)}, BAD), ({"k_cache": d(C.F16, (NB, HK, BS * D), 8 << 20)}, BAD),
    ({"qs": HQ * D - 8}, BAD), ({"ks": HK * D + 4}, BAD), ({"vs": 1 << 60}, BAD), ({"qs": -8}, BAD),
    ({"mode": 1}, BAD), ({"mode": 2}, BAD), ({"section": [4, 6]}, BAD), ({"section": [4, 6, 7]}, BAD),
    ({"section": [4, -6, 18]}, BAD), ({"section": [4, 6, 6]}, BAD),  # mrope takes [3, T] positions
    ({"section": [1, 1 << 62, 1 << 62], "positions": d(C.I64, (3, T), FAKE)}, BAD),
    *[({k: d(C.F16, s, (9 << 24) + 8)}, BAD) for k, s in (("query", (T, HQ * D)), ("key", (T, HK * D)),
                                                           ("table", (10, 32)), ("k_cache", (NB, HK, BS, D)))],
    ({"slots": d(C.I64, (T,), FAKE + 4)}, BAD),
    # shared memory
    ({"query_out": d(C.F16, (T, HQ * D), (2 << 20) + 16)}, BAD), ({"query_out": d(C.F16, (T, HQ * D), 3 << 20)}, BAD),
    ({"query_out": d(C.F16, (T, HQ * D), 5 << 20)}, BAD), ({"query_out": d(C.F16, (T, HQ * D), 8 << 20)}, BAD),
    ({"v_cache": d(C.F16, (NB, HK, BS, D), 8 << 20)}, BAD), ({"k_cache": d(C.F16, (NB, HK, BS, D), 3 << 20)}, BAD),
    ({"v_cache": d(C.F16, (NB, HK, BS, D), 6 << 20)}, BAD),
    ({"query_out": None, "query": d(C.F16, (T, HQ * D), (3 << 20) - 64)}, BAD),  # in place, over the keys
    ({"query": d(C.F16, (T, HQ * D), 7 << 20), "qs": 512}, BAD),  # the output is the strided query's buffer
])
def test_append_refusals(lib, over, status):
    n = lib.rope_launch_count()
    assert _append(lib, **over) == status
    assert lib.rope_launch_count() == n


def test_append_of_no_tokens(lib):
    z = lambda w: d(C.F16, (0, w), 0)  # noqa: E731
    assert _append(lib, positions=d(C.I64, (0,), 0), slots=d(C.I64, (0,), 0), query=z(HQ * D), key=z(HK * D),
                   value=z(HK * D), query_out=z(HQ * D)) == OK


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
NBATCH, W = 2, 5


def _attend(lib, **over):
    at = {"query": d(C.BF16, (T, HQ * D), 2 << 20), "qs": 0, "k_cache": d(C.BF16, (NB, HK, BS, D), 8 << 20),
          "v_cache": d(C.BF16, (NB, HK, BS, D), 9 << 20), "block_table": d(C.I64, (NBATCH, W), 3 << 20),
          "seq_lens": d(C.I64, (NBATCH,), 4 << 20), "starts": d(C.I64, (NBATCH + 1,), 5 << 20),
          "prefix": d(C.I64, (2,), 6 << 20), "P": 7, "scale": 0.125, "out": d(C.BF16, (T, HQ * D), 7 << 20),
          "lse": d(C.F32, (T, HQ), 10 << 20), "workspace": 16 << 20, "bytes": 1 << 30}
    assert not set(over) - set(at)
    at.update(over)
    return lib.rope_paged_attention(*at.values(), None)


@pytest.mark.parametrize("over,status", [
    *[({k: None}, NULL) for k in ("query", "k_cache", "v_cache", "block_table", "seq_lens", "starts", "out", "prefix",
                                  "workspace")],
    *[({k: d(C.BF16, s, 0)}, NULL) for k, s in (("query", (T, HQ * D)), ("k_cache", (NB, HK, BS, D)),
                                                 ("v_cache", (NB, HK, BS, D)), ("out", (T, HQ * D)))],
    *[({k: d(C.I64, s, 0)}, NULL) for k, s in (("block_table", (NBATCH, W)), ("seq_lens", (NBATCH,)),
                                                ("starts", (NBATCH + 1,)), ("prefix", (2,)))],
    ({"lse": d(C.F32, (T, HQ), 0)}, NULL),
    ({"query": d(C.F16, (T, HQ * D), 2 << 20)}, BAD), ({"out": d(C.F32, (T, HQ * D), 7 << 20)}, BAD),
    ({"v_cache": d(C.F16, (NB, HK, BS, D), 9 << 20)}, BAD), ({"lse": d(C.BF16, (T, HQ), 10 << 20)}, BAD),
    ({"block_table": d(C.F32, (NBATCH, W), 3 << 20)}, BAD), ({"seq_lens": d(C.F32, (NBATCH,), 4 << 20)}, BAD),
    ({"prefix": d(C.F32, (2,), 6 << 20)}, BAD), ({"query": d(C.I64, (T, HQ * D), 2 << 20)}, BAD),
    ({"query": d(C.BF16, (T, 3 * D), 2 << 20), "out": d(C.BF16, (T, 3 * D), 7 << 20)}, BAD),  # 3 heads on 2
    ({"query": d(C.BF16, (T, HQ * D + 8), 2 << 20)}, BAD), ({"query": d(C.BF16, (T, 0), 2 << 20)}, BAD),
    ({"query": d(C.BF16, (T, HQ, D), 2 << 20)}, BAD),
    ({"k_cache": d(C.BF16, (NB, HK, BS, 48), 8 << 20), "v_cache": d(C.BF16, (NB, HK, BS, 48), 9 << 20),
      "query": d(C.BF16, (T, HQ * 48), 2 << 20), "out": d(C.BF16, (T, HQ * 48), 7 << 20)}, BAD),
    ({"k_cache": d(C.BF16, (NB, HK, BS, 544), 8 << 20), "v_cache": d(C.BF16, (NB, HK, BS, 544), 9 << 20),
      "query": d(C.BF16, (T, HQ * 544), 2 << 20), "out": d(C.BF16, (T, HQ * 544), 7 << 20)}, BAD),
    ({"v_cache": d(C.BF16, (NB, HK, BS + 1, D), 9 << 20)}, BAD), ({"k_cache": d(C.BF16, (0, HK, BS, D), 8 << 20)}, BAD),
    ({"qs": HQ * D - 8}, BAD), ({"qs": HQ * D + 4}, BAD), ({"qs": 1 << 61}, BAD),
    ({"block_table": d(C.I64, (NBATCH + 1, W), 3 << 20)}, BAD), ({"block_table": d(C.I64, (NBATCH, 0), 3 << 20)}, BAD),
    ({"block_table": d(C.I64, (NBATCH, 1 << 29), 3 << 20)}, BAD), ({"starts": d(C.I64, (NBATCH,), 5 << 20)}, BAD),
    ({"seq_lens": d(C.I64, (0,), 4 << 20), "starts": d(C.I64, (1,), 5 << 20), "block_table": d(C.I64, (0, W), 3 << 20)}, BAD),
    ({"P": -1}, BAD), ({"P": 9}, BAD), ({"P": (1 << 30) + 1}, BAD),
    ({"P": 1 << 30, "prefix": d(C.I64, (1 << 28,), 1 << 44),  # each in its range, but 2^31 keys together
      "block_table": d(C.I64, (NBATCH, 1 << 28), 1 << 45)}, BAD),
    ({"scale": 0.0}, BAD), ({"scale": -1.0}, BAD), ({"scale": math.nan}, BAD), ({"scale": math.inf}, BAD),
    ({"out": d(C.BF16, (T + 1, HQ * D), 7 << 20)}, BAD), ({"lse": d(C.F32, (T, HK), 10 << 20)}, BAD),
    ({"bytes": 0}, BAD), ({"bytes": 255}, BAD), ({"workspace": (16 << 20) + 128}, BAD),
    ({"query": d(C.BF16, (T, HQ * D), (2 << 20) + 8)}, BAD), ({"out": d(C.BF16, (T, HQ * D), (7 << 20) + 2)}, BAD),
    ({"seq_lens": d(C.I64, (NBATCH,), (4 << 20) + 4)}, BAD), ({"prefix": d(C.I64, (2,), (6 << 20) + 4)}, BAD),
    # shared memory
    ({"out": d(C.BF16, (T, HQ * D), 2 << 20)}, BAD), ({"out": d(C.BF16, (T, HQ * D), 8 << 20)}, BAD),
    ({"lse": d(C.F32, (T, HQ), 7 << 20)}, BAD), ({"lse": d(C.F32, (T, HQ), 3 << 20)}, BAD),
    ({"workspace": 1 << 20}, BAD),  # its 1 GB reach over the tensors
    ({"prefix": d(C.I64, (2,), 7 << 20)}, BAD),
])
def test_attend_refusals(lib, over, status):
    n = lib.rope_launch_count()
    assert _attend(lib, **over) == status
    assert lib.rope_launch_count() == n


def test_attend_of_no_tokens(lib):
    assert _attend(lib, query=d(C.BF16, (0, HQ * D), 0), out=d(C.BF16, (0, HQ * D), 0), lse=None, workspace=None) == OK


def test_workspace_sizes(lib):
    def size(*a):
        n = ctypes.c_int64(-1)
        st = lib.rope_paged_attention_workspace(*a, ctypes.byref(n))
        return st, n.value

    for a in ((1, 1, 1, 64, C.F16, 0), (4096, 32, 8, 128, C.BF16, 4096), (7, 4, 2, 64, C.F32, 5), (0, 4, 2, 64, C.F32, 0),
              (1 << 20, 1 << 10, 1, 512, C.BF16, 1), (1 << 20, 1 << 10, 1, 128, C.BF16, 1)):
        st, n = size(*a)
        assert st == OK and n >= 256, a
    for a in ((-1, 1, 1, 64, C.F16, 0), (1, 3, 2, 64, C.F16, 0), (1, 2, 2, 48, C.F16, 0), (1, 2, 2, 64, C.I64, 0),
              (1, 2, 2, 64, C.F16, -1), ((1 << 31) + 1, 2, 2, 64, C.F16, 0), (1 << 30, 2, 2, 64, C.F16, 0),
              (1, 1 << 17, 1, 64, C.F16, 0), (1, 0, 1, 64, C.F16, 0), (1, 2, 2, 544, C.F16, 0)):
        assert size(*a)[0] == BAD, a
    assert lib.rope_paged_attention_workspace(1, 1, 1, 64, C.F16, 0, None) == NULL


# ---------------------------------------------------------------------------
# the Python binding
# ---------------------------------------------------------------------------
def test_binding_takes_cuda_tensors_only(lib):
    x = torch.zeros(4, 64)
    i = torch.zeros(4, dtype=torch.int64)
    kv = torch.zeros(3, 1, 4, 64)
    with pytest.raises(ValueError):
        R.scaled_cos_sin_cache(x, [0.0] * 32)
    with pytest.raises(ValueError):
        R.scaled_cos_sin(x, x, [0.0] * 32)
    with pytest.raises(ValueError):
        R.append_paged_kv(i, x, x, x, x, i, kv, kv, 64)
    with pytest.raises(ValueError):
        R.paged_attention(x, kv, kv, i.view(4, 1), i, torch.zeros(5, dtype=torch.int64), x)


def test_heads_of_no_columns(lib):
    """Without a scale: no power of zero."""
    kv = torch.zeros(3, 1, 4, 0)
    i = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        R.paged_attention(torch.zeros(4, 64), kv, kv, i.view(4, 1), i, torch.zeros(5, dtype=torch.int64),
                          torch.zeros(4, 64))


@pytest.mark.parametrize("scaling", [None, {"kind": "factors", "factors": [2.0, 4.0]}])
def test_frequencies_stay_on_the_host_under_another_default_device(lib, scaling):
    want = R.rope_frequencies(4, 10000.0, scaling)[0]
    with torch.device("meta"):
        got = R.rope_frequencies(4, 10000.0, scaling)[0]
        given = C._host_frequencies([1.0, 0.5])
    assert got.device.type == "cpu" and torch.equal(got, want)
    assert given.device.type == "cpu" and given.tolist() == [1.0, 0.5]
