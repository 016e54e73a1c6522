"""Append to a paged cache of 8-bit codes, against a 64-bit reference (bounds: tests/codes_ref.py)."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import bytes_of, check_codes, codes_append_case, codes_append_reference
from guard import Guards
from serving_ref import append_bound, assert_close

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def run(c, in_place=False, with_query=True, stream=None, prepared=False):
    g = Guards()
    put = lambda t, n: g.put(bytes_of(t), n).view(t.dtype)  # noqa: E731
    kc, vc, ks, vs = (put(c[n], n) for n in ("kc", "vc", "ks", "vs"))
    if c.get("fused"):
        buf = g.put(torch.cat([c["q"], c["k"], c["v"]], 1), "qkv")
        w = [c["q"].shape[1], c["k"].shape[1]]
        q, k, v = buf[:, :w[0]], buf[:, w[0]:w[0] + w[1]], buf[:, w[0] + w[1]:]
    else:
        q, k, v = (g.put(c[n], n) for n in "qkv")
    qo = None if in_place or not with_query else g.empty(tuple(c["q"].shape), c["dtype"], "q_out")
    call = R.prepare_append_paged_kv_8bit if prepared else R.append_paged_kv_8bit
    r = call(g.put(c["pos"], "pos"), q if with_query else None, k, v, g.put(c["table"], "table"),
             g.put(c["slots"], "slots"), kc, vc, ks, vs, c["D"], is_neox=c["neox"], mrope_section=c["sections"],
             cache_mode=c["cache_mode"], query_out=qo, stream=stream)
    if prepared:
        r()
    g.check()
    return (q if in_place else qo), kc, vc, ks, vs


def check(c, what="", **kw):
    q_ref, skipped, (kr, vr) = codes_append_reference(c)
    q, kc, vc, ks, vs = run(c, **kw)
    check_codes(kc, ks, kr, what + " k")
    check_codes(vc, vs, vr, what + " v")
    if q is not None:
        rows = [t for t in range(len(q_ref)) if t not in skipped]
        assert_close(q[rows], q_ref[rows], append_bound(q_ref[rows], c["dtype"]), what + " q")
    assert R.get_device_error() == (R.ROPE_DEVICE_POSITION_OUT_OF_RANGE if skipped else 0)
    return q, kc, vc, ks, vs


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("bs,S", [(1, 1), (16, 1), (16, 16), (16, 4), (17, 17), (12, 3), (64, 2), (128, 1)])
@pytest.mark.parametrize("neox", [True, False])
def test_pages_and_scale_blocks(rope_gpu, dtype, bs, S, neox):
    """Runs that begin and end inside a block, fill it, and go through several."""
    new, held = [1, 1, 5, 40, 0, 16, 131, 1], [0, 15, 3, 9, 4, 16, 0, 63]
    c = codes_append_case(1, dtype, new, held, bs, S, neox=neox, scale=4.0)
    check(c, "pages")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("D,Rr", [(32, 32), (64, 32), (96, 96), (128, 64), (160, 160), (256, 64), (512, 512)])
@pytest.mark.parametrize("hq,hk,hv", [(1, 1, 1), (5, 1, 1), (8, 2, 3), (16, 16, 16)])
def test_heads(rope_gpu, dtype, D, Rr, hq, hk, hv):
    for neox in (True, False):
        check(codes_append_case(2, dtype, [3, 1, 20], [0, 7, 30], 16, 2, hq=hq, hk=hk, hv=hv, D=D, R=Rr, neox=neox), "heads")


@pytest.mark.parametrize("D", [16, 48])
def test_narrow_heads(rope_gpu, D):
    check(codes_append_case(3, torch.float32, [3, 20], [5, 0], 8, 1, D=D, R=16), "narrow")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("neox", [True, False])
def test_tables_in_32_bits_and_views_of_one_buffer(rope_gpu, dtype, neox):
    c = codes_append_case(4, dtype, [9, 1, 17], [2, 31, 0], 16, 1, D=128, table_dtype=torch.float32, neox=neox)
    c["fused"] = True
    check(c, "fused")
    check(c, "in place", in_place=True)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("sections,mode", [((8, 12, 12), 0), ((8, 8, 8, 8), 0), ((8, 12, 12), 1)])
@pytest.mark.parametrize("neox", [True, False])
def test_mrope(rope_gpu, dtype, sections, mode, neox):
    check(codes_append_case(5, dtype, [9, 30], [2, 0], 16, 2, D=64, sections=list(sections), cache_mode=mode, neox=neox), "mrope")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_without_queries_and_padding(rope_gpu, dtype):
    c = codes_append_case(6, dtype, [5, 1, 33], [11, 0, 2], 16, 1, pad=3)
    check(c, "no query", with_query=False)
    check(c, "padded")
    check(c, "prepared", prepared=True)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_values_at_the_ends(rope_gpu, dtype):
    """Zeros, the type's largest and smallest values, NaN and infinities, and steps of the scale."""
    c = codes_append_case(7, dtype, [16, 16, 16, 16, 3, 16], [0, 0, 0, 0, 5, 0], 16, 1, D=64, R=32)
    info = torch.finfo(dtype)
    v = c["v"]
    v[:16] = 0
    v[16:32] = info.max
    v[32:48] = info.tiny
    v[40] = -info.tiny * (3 if dtype == torch.float32 else info.eps)
    v[48:64, ::3] = float("nan")
    v[48:64, 1::3] = float("inf")
    v[64:67] = 0  # zeros behind tokens that are there
    v[67:83] = 448.0
    v[70, 5] = 449.0 if dtype != torch.bfloat16 else 450.0
    c["k"][3, 3] = float("-inf")
    c["k"][20] = 0
    q, kc, vc, ks, vs = check(c, "ends")
    first = int(c["slots"][0]) // 16
    assert (bytes_of(vs)[first] == 0).all() and (bytes_of(vc)[first] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_scales_grow_and_stay(rope_gpu, dtype):
    """A token after another, each larger or smaller than those before: the block's values stay what they were, to
    one rounding."""
    bs, D = 16, 64
    c = codes_append_case(8, dtype, [1], [0], bs, 1, hq=1, hk=1, D=D)
    g = torch.Generator().manual_seed(9)
    dev = lambda t: t.cuda()  # noqa: E731
    kc, vc, ks, vs = (bytes_of(c[n]).cuda().view(c[n].dtype) for n in ("kc", "vc", "ks", "vs"))
    page = int(c["slots"][0]) // bs
    sizes = [0.0, 1.0, 1e-3, 30.0, 2.0, 1000.0, 1e-4, 1000.0, 0.5]
    put = []
    for i, f in enumerate(sizes):
        x = (torch.randn(1, D, generator=g) * f).to(dtype)
        put.append(x.double())
        R.append_paged_kv_8bit(dev(torch.tensor([0])), None, dev(x), dev(x), dev(torch.cat([torch.ones(1, D // 2), torch.zeros(1, D // 2)], 1).to(dtype)),
                               dev(torch.tensor([page * bs + i])), kc, vc, ks, vs, D)
        for codes, scale in ((kc, ks), (vc, vs)):
            b = int(bytes_of(scale)[page, 0, 0])
            got = bytes_of(codes)[page, 0, :i + 1].cpu().view(torch.float8_e4m3fn).double() * 2.0 ** (b - 127)
            ref = torch.cat(put)
            most = float(ref.abs().max())
            assert (b == 0) == (most == 0)
            if most:
                assert 224 * 2.0 ** (b - 127) < most * (1 + 1e-6) and most <= 448 * 2.0 ** (b - 127)
            # one rounding to 3 fraction bits, and one to the subnormals' step of every scale since: they add up to less
            # than twice the last
            assert bool(((got - ref).abs() <= 2.0 ** -4 * ref.abs() + 2 * 2.0 ** (b - 137)).all())
    assert R.get_device_error() == 0


def test_positions_and_slots_out_of_range(rope_gpu):
    c = codes_append_case(10, torch.bfloat16, [4, 20, 1], [3, 0, 8], 16, 2, max_seq=50)
    c["pos"][2] = 50
    c["pos"][9] = -1
    c["pos"][24] = 1 << 40
    check(c, "positions")
    c = codes_append_case(11, torch.bfloat16, [4, 20], [3, 0], 16, 2)
    # (the last tokens: those of a scale block have to stand one after the other)
    c["slots"][21] = c["kc"].shape[0] * 16
    c["slots"][22:] = 1 << 60
    q_ref, skipped, (kr, vr) = codes_append_reference(c)
    q, kc, vc, ks, vs = run(c)
    assert R.get_device_error() == R.ROPE_DEVICE_SLOT_OUT_OF_RANGE
    check_codes(kc, ks, kr, "slots")
    assert_close(q, q_ref, append_bound(q_ref, c["dtype"]), "q")


def test_empty_batch(rope_gpu):
    c = codes_append_case(12, torch.bfloat16, [1], [0], 16, 1)
    n = R.launch_count()
    for x in "qkv":
        c[x] = c[x][:0]
    c["pos"], c["slots"] = c["pos"][:0], c["slots"][:0]
    run(c)
    assert R.launch_count() == n
