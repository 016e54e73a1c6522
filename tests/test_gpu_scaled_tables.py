"""cos/sin tables for scaled frequencies against float64 sin and cos (bounds: tests/serving_ref.py)."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from guard import Guards
from serving_ref import assert_close, table_bound, table_reference

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
SCALINGS = [None, {"kind": "linear", "factor": 4}, {"kind": "base", "factor": 2.5},
            {"kind": "yarn", "factor": 8, "original_length": 16384},
            {"kind": "wavelength", "factor": 8, "low": 1, "high": 4, "original_length": 8192}]


def _check(dtype, rows, dim, layout, first=0, positions=None, scaling=None, offset=0, inv=None, scale=None):
    g = Guards()
    if inv is None:
        inv, scale = R.rope_frequencies(dim, 10000.0, scaling)
    pos = g.put(positions, "positions") if positions is not None else None
    at = (positions if positions is not None else torch.arange(rows)) + first
    if layout == "cache":
        out = g.empty((rows, dim), dtype, "cache", offset)
        R.scaled_cos_sin_cache(out, inv, scale, positions=pos, first_position=first)
        g.check()
        ref, slack = table_reference(inv, scale, at, layout)
        assert_close(out.cpu(), ref, table_bound(ref, slack, dtype), "cache")
        return
    c, s = g.empty((1, rows, 1, dim), dtype, "cos", offset), g.empty((1, rows, 1, dim), dtype, "sin", offset)
    R.scaled_cos_sin(c, s, inv, scale, layout, positions=pos, first_position=first)
    g.check()
    rc, rs, slack = table_reference(inv, scale, at, layout)
    assert_close(c.cpu().reshape(rows, dim), rc, table_bound(rc, slack, dtype), "cos")
    assert_close(s.cpu().reshape(rows, dim), rs, table_bound(rs, slack, dtype), "sin")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("layout", ["cache", "half", "interleave"])
@pytest.mark.parametrize("rows,dim", [(1, 2), (3, 6), (1, 64), (37, 96), (130, 128), (5, 256), (7, 258), (2, 2048)])
def test_layouts_and_sizes(rope_gpu, dtype, layout, rows, dim):
    _check(dtype, rows, dim, layout, first=11)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s["kind"] if s else "none")
def test_scalings(rope_gpu, dtype, scaling):
    _check(dtype, 300, 128, "cache", first=4000, scaling=scaling)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("layout", ["cache", "half", "interleave"])
def test_given_positions(rope_gpu, dtype, layout):
    """Positions of packed sequences: repeated, out of order, negative, and far."""
    pos = torch.cat([torch.arange(40), torch.arange(17), torch.tensor([0, -1, -5000, 1 << 20, 2097151, 7, 7])])
    _check(dtype, len(pos), 64, layout, positions=pos)
    _check(dtype, len(pos), 64, layout, positions=pos, first=1000)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_unaligned_output(rope_gpu, dtype):
    """Element alignment is enough; the pieces are then single elements."""
    _check(dtype, 9, 64, "cache", offset=torch.empty(0, dtype=dtype).element_size())
    _check(dtype, 9, 64, "half", offset=torch.empty(0, dtype=dtype).element_size())


def test_far_positions_keep_their_angle(rope_gpu):
    """Row p of the frequency 2 pi / 3 is row p mod 3 for any p: angles are exact modulo whole turns.
    The frequency is a binary64 number, off by 2^-53 of itself: at p = 2^40 that is 2 pi / 3 * 2^-13."""
    import math
    f = [2 * math.pi / 3]
    for first in (3 << 20, 3 << 38):
        out = torch.empty(6, 2, device="cuda")
        R.scaled_cos_sin_cache(out, f, 1.0, first_position=first)
        near = torch.empty(6, 2, device="cuda")
        R.scaled_cos_sin_cache(near, f, 1.0)
        bound = first * f[0] * 2.0 ** -52 + 2.0 ** -21
        assert float((out - near).abs().max()) <= bound


def test_negative_frequencies_keep_their_angle(rope_gpu):
    """cos is even and sin is odd in the frequency, at far positions as well.  An angle is off by 2^-64 turns a
    position (half a unit in each of two tables, and what a table's piece of 9 bits leaves out): 2^-24 of a turn,
    2 pi * 2^-24 < 2^-21, at 2^40; the values are then within 4 half steps each."""
    f = torch.tensor([1e-4, 2.0 ** -30, 0.3, 7.0, 1e5], dtype=torch.float64)
    a, b = torch.empty(3, 10, device="cuda"), torch.empty(3, 10, device="cuda")
    for first in (5, 1 << 40):
        R.scaled_cos_sin_cache(a, f, first_position=first)
        R.scaled_cos_sin_cache(b, -f, first_position=first)
        sign = torch.cat([torch.ones(5), -torch.ones(5)]).cuda()
        assert float((a - b * sign).abs().max()) <= 2.0 ** -21 + 8 * 2.0 ** -24


def test_large_table_every_row(rope_gpu):
    """More rows than one pass of the grid."""
    inv, scale = R.rope_frequencies(64, 500000.0, SCALINGS[3])
    out = torch.empty(50001, 64, device="cuda", dtype=torch.bfloat16)
    R.scaled_cos_sin_cache(out, inv, scale, first_position=70000)
    ref, slack = table_reference(inv, scale, torch.arange(50001) + 70000, "cache")
    assert_close(out.cpu(), ref, table_bound(ref, slack, torch.bfloat16), "large")


def test_feeds_the_existing_operators(rope_gpu):
    """A table made here, read by the cache-indexed and the in-place operator: both rotate by the same angle."""
    D, T = 64, 50
    inv, scale = R.rope_frequencies(D, 10000.0, SCALINGS[3])
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(3)).cuda()
    cache = torch.empty(T, D, device="cuda")
    R.scaled_cos_sin_cache(cache, inv, scale)
    q, k = x.clone(), x.clone()
    R.rope_with_sin_cos_cache(torch.arange(T, device="cuda"), q, k, cache, D)
    cos, sin = (torch.empty(1, T, 1, D, device="cuda") for _ in range(2))
    R.scaled_cos_sin(cos, sin, inv, scale, "half")
    y = x.clone().view(1, T, 1, D)
    R.rope_inplace_partial(y, cos, sin, "half")
    assert torch.equal(q, k) and torch.equal(q, y.view(T, D))
    ang = torch.arange(T).double()[:, None] * inv
    a, b = x.cpu().double()[:, :32], x.cpu().double()[:, 32:]
    ref = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], 1) * scale
    # cos and sin each off by 4 half steps, the rotation by 2: (4 + 2) e of the terms, times two terms
    terms = torch.cat([a.abs() + b.abs()] * 2, 1) * scale
    assert_close(q, ref, 8 * 2.0 ** -24 * terms, "rotated")


def test_empty_output_launches_nothing(rope_gpu):
    n = R.launch_count()
    R.scaled_cos_sin_cache(torch.empty(0, 64, device="cuda"), [0.0] * 32)
    assert R.launch_count() == n
