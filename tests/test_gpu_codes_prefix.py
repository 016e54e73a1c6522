"""The attention over a cache of 8-bit codes with a prefix that has a launch of its own: one where that saves more than 8 MB of
re-reads, (B - 1) * P * Nk * D * 2 bytes of codes.  Three launches then: the prefix, the sequences' own keys, the join."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import bytes_of, coded_case, run_coded
from guard import Guards
from scales_ref import put, reference
from serving_ref import assert_close

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def shared(c):
    return (len(c["lens"]) - 1) * c["P"] * c["hk"] * c["D"] * 2 > 8e6


def run_shared(c, error=0):
    assert shared(c)
    n = R.launch_count()
    out, lse = run_coded(R, c)
    assert R.launch_count() == n + 3
    assert R.get_device_error() == error
    return out, lse


def check_shared(c, what=""):
    out, lse = run_shared(c)
    T = int(c["starts"][-1])
    ro, rl, to, tl = reference(c)
    assert_close(out[:T], ro[:T], to[:T], what + " out")
    assert_close(lse[:T], rl[:T], tl[:T], what + " lse")
    assert torch.equal(out[T:].view(torch.int16), torch.full_like(out[T:].view(torch.int16), 0x7FA5)), what
    return out, lse


def batch(n, most, own):
    new = [1 + i % most for i in range(n)]
    return new, [new[i] + (i * 37) % own for i in range(n)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D,hk,P", [(32, 4, 1500), (64, 2, 1500), (96, 2, 1100), (128, 1, 1500), (192, 1, 800), (256, 1, 700)])
@pytest.mark.parametrize("n,most,G", [(41, 2, 4), (41, 1, 1), (41, 3, 16)])
def test_shared_prefix(rope_gpu, dtype, D, hk, P, n, most, G):
    """Few and many rows: over the prefix units of 16 rows or (984 rows, 16-bit) tall ones, over the own keys of 8 to 16 and of
    more rows."""
    new, own = batch(n, most, 90)
    c = coded_case(31, dtype, new, own, P=P, hq=G * hk, hk=hk, D=D, S=4)
    check_shared(c, "prefix")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [64, 256])
def test_tall_units_over_the_prefix(rope_gpu, dtype, D):
    new, own = batch(30, 8, 200)
    check_shared(coded_case(32, dtype, new, own, P=3001, hq=24, hk=2, D=D, S=2, bs=32), "tall")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [128, 256])
def test_few_rows_behind_a_long_prefix(rope_gpu, dtype, D):
    """8 rows and fewer in all."""
    check_shared(coded_case(33, dtype, [1, 2, 1], [1, 40, 7], P=20011, hq=2, hk=2, D=D, S=16), "few")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_rows_without_own_keys_and_within_the_prefix(rope_gpu, dtype, D):
    """Sequences that end at the prefix's end, inside it, before its first key, and that get no token."""
    n = 41
    new = [1 + i % 4 if i % 7 else 0 for i in range(n)]
    own = [new[i] + 30 for i in range(n)]
    c = coded_case(34, dtype, new, own, P=1500, hq=8, hk=2, D=D, S=1, spare_rows=5)
    c["lens"] = torch.tensor([1500 if i % 5 == 0 else 1500 - 37 * i if i % 5 == 1 else 2 if i % 5 == 2 else 0 if i % 10 == 3
                              else 1500 + own[i] for i in range(n)])
    _, lse = check_shared(c, "within")
    assert bool((lse[:int(c["starts"][-1])] == float("-inf")).any())  # (positions before the first key)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("most,G", [(1, 2), (3, 16)])
def test_scales_far_apart_behind_a_shared_prefix(rope_gpu, dtype, D, most, G):
    """Key 4 is 400 ahead of all others; V's units grow by 2^95 in the prefix, in the own keys or in both; zeros in front."""
    new, own = batch(41, most, 60)
    for where in ((200,), (1520,), (200, 1520)):
        c = coded_case(35, dtype, new, own, P=1500, hq=2 * G, hk=2, D=D, S=16)
        if not shared(c):
            c = coded_case(35, dtype, new, own, P=3500, hq=2 * G, hk=2, D=D, S=16)
        c["q"][:] = 50 / D ** 0.5
        bytes_of(c["k_codes"])[:] = 0
        for name in ("k_scale", "v_scale"):
            bytes_of(c[name])[:] = 127
        put(c, "k", 4, code=0x50)
        for j in where:
            j += c["P"] - 1500 if j >= 1500 else 0
            put(c, "v", j, byte=222)
        check_shared(c, "jump at %s" % (where,))
    c = coded_case(36, dtype, new, own, P=c["P"], hq=2 * G, hk=2, D=D, S=16)
    for j in range(c["P"] // 2):
        put(c, "v", j, byte=0, code=0, b=0)  # (the prefix is every sequence's)
    check_shared(c, "zeros")


def test_nan_and_pages_outside_in_a_shared_prefix(rope_gpu):
    """A key of NaN codes that some sequences end before; a page outside the cache."""
    for dtype in DTYPES:
        new, own = batch(41, 2, 60)
        c = coded_case(37, dtype, new, own, P=1500, hq=8, hk=2, D=64, S=16)
        put(c, "v", 1499, code=0x7f, b=0)
        for i in range(0, 41, 3):
            c["lens"][i] = 1499
        out, _ = check_shared(c, "nan")
        assert torch.isnan(out).any() and not torch.isnan(out).all()
        c = coded_case(37, dtype, new, own, P=1500, hq=8, hk=2, D=64, S=16)
        good = c["prefix"][3].clone()
        c["prefix"][3] = c["k_codes"].shape[0]
        out, lse = run_shared(c, R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
        c["prefix"][3] = good
        # as the sequences without the 16 keys of that page, which no row sees
        keep = [p for i, p in enumerate(c["prefix"].tolist()) if i != 3]
        c2 = dict(c, prefix=torch.tensor(keep), P=1500 - 16, lens=c["lens"] - 16)
        ro, rl, to, tl = reference(c2)
        assert_close(out, ro, to, "out")
        assert_close(lse, rl, tl, "lse")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_shared_prefix_in_a_graph_with_any_workspace(rope_gpu, dtype):
    """Captured once and replayed over other lengths and tables of the same shape, with a workspace full of NaN."""
    new, own = batch(41, 2, 90)
    c = coded_case(38, dtype, new, own, P=1500, hq=8, hk=2, D=64, S=4)
    assert shared(c)
    g = Guards()
    q, table, lens, starts, prefix = (g.put(c[n], n) for n in ("q", "table", "lens", "starts", "prefix"))
    caches = [g.put(bytes_of(c[n]), n).view(c[n].dtype) for n in ("k_codes", "v_codes", "k_scale", "v_scale")]
    out, lse = g.empty(c["q"].shape, dtype, "out"), g.empty((c["T"], c["hq"]), torch.float32, "lse")
    n = R.paged_attention_workspace(q, caches[0], 1500)
    ws = g.put(torch.full((n,), 0xff, dtype=torch.uint8), "workspace", offset=0)
    stream = torch.cuda.Stream()
    call = lambda: R.paged_attention_8bit(q, *caches, table, lens, starts, out, scale=c["scale"], prefix_blocks=prefix,  # noqa: E731
                                          prefix_len=1500, lse=lse, workspace=ws)
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for k in range(3):
        less = dict(c, lens=c["lens"] - torch.tensor([(7 * i * k) % max(own[i] - new[i], 1) for i in range(41)]))
        lens.copy_(less["lens"])
        ws.fill_(0xff)
        out.fill_(0)
        graph.replay()
        g.check()
        ro, rl, to, tl = reference(less)
        assert_close(out, ro, to, "out")
        assert_close(lse, rl, tl, "lse")
    assert R.get_device_error() == 0
