"""Attention over a paged cache of 8-bit codes whose scales lie far apart, against a float64 reference (tests/scales_ref.py),
in every kernel that the lengths choose between: units of 8, of 16 and of 128 or 256 rows, and a warp a row."""
import functools

import pytest
import torch

from codes_ref import bytes_of, coded_case
from scales_ref import check, put, put_bytes

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
HALVES = [torch.float16, torch.bfloat16]

# (new, own, query heads a key head, key heads, wide table): what the kernels are chosen by.  Small units of two tiles of keys
# are not split; of many heads' most come to several tiles a CTA.
UNITS = {"8": ([1, 1], [240, 133], 2, 1, False), "16": ([7], [240], 2, 1, False),
         "8 many": ([1] * 4, [400, 398, 390, 260], 2, 64, False), "16 many": ([3] * 4, [400, 395, 390, 260], 4, 64, False),
         "tall one tile": ([100], [400], 1, 1, True), "tall two tiles": ([150, 70], [400, 70], 3, 1, True)}
ALL = list(UNITS)
FEW = [u for u in ALL if "many" not in u]


@functools.lru_cache(maxsize=1)
def made(units, seed, dtype, D, P, q_scale):
    new, own, G, hk, wide = UNITS[units]
    c = coded_case(seed, dtype, new, own, hq=G * hk, hk=hk, D=D, P=P, S=16, q_scale=q_scale)
    del c["k"], c["v"]  # (what the codes stand for changes)
    c["wide"] = wide
    return c


def case(units, seed, dtype, D, P=0, q_scale=1.0):
    return {n: x.clone() if torch.is_tensor(x) else x for n, x in made(units, seed, dtype, D, P, q_scale).items()}


def led_by_key_4(units, dtype, D):
    """Key 4 is 400 ahead of all others, whose weights are e^-400 of its own; V of about 64 in units of 1."""
    c = case(units, 21, dtype, D)
    c["q"][:] = 50 / D ** 0.5
    bytes_of(c["k_codes"])[:] = 0
    for name in ("k_scale", "v_scale"):
        bytes_of(c[name])[:] = 127
    put(c, "k", 4, code=0x50)  # 8
    return c


@pytest.mark.parametrize("step", [90, 91, 95])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("units", ALL)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 128, 160, 256])
def test_v_in_units_beyond_2_to_the_90_of_the_one_that_counts(rope_gpu, dtype, units, D, step):
    """A later V in units that many times as large, with no weight to speak of."""
    if dtype != torch.float32 and D in (16, 48):
        pytest.skip("16-bit heads are multiples of 32")
    c = led_by_key_4(units, dtype, D)
    put(c, "v", 130, byte=127 + step)
    check(c, "jump")
    c = led_by_key_4(units, dtype, D)  # and one that the last token alone sees
    for b, n in enumerate(c["lens"].tolist()):
        put(c, "v", n - 1, byte=127 + step, b=b)
    check(c, "last")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("units", ALL)
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_v_in_units_that_grow_again_and_again(rope_gpu, dtype, units, D):
    """V's units grow by 2^88 twice, each time by less than what a row is computed again for, or by 2^14 each 32 keys."""
    c = led_by_key_4(units, dtype, D)
    j = torch.arange(400)
    put_bytes(c, "v", 70 + 88 * (j // 128).clamp(max=2))
    check(c, "stairs")
    put_bytes(c, "v", 70 + j // 32 * 14)
    check(c, "slope")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("units", ALL)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [0, 96])
def test_zeros_in_front(rope_gpu, dtype, units, D, P):
    """V's first blocks are zeros with the byte 0: as with any other byte for them, bit for bit, so that no row is
    computed again key by key for it."""
    c = case(units, 22, dtype, D, P=P)
    for j in range(192):
        put(c, "v", j, byte=100, code=0)
    a = check(c, "zeros in units of 2^-27")
    put_bytes(c, "v", torch.zeros(192))
    b = check(c, "zeros")
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("far", [9, 11, 15, 16, 40])
@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("units", FEW)
@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256])
def test_scales_apart(rope_gpu, dtype, units, D, name, far):
    """Scales up to 2^far apart: from key to key, growing and shrinking along the keys and from one 32 keys to the next,
    with blocks of zeros among them."""
    if far == 40 and D not in (64, 256):
        pytest.skip("as for the others")
    c = case(units, 23, dtype, D, q_scale=2.0)
    g = torch.Generator().manual_seed(far)
    n = 400
    for kind, bytes_ in (("any", torch.randint(122 - far, 123, (n,), generator=g)),
                         ("up", 122 - far + torch.arange(n) * far // (n - 1)),
                         ("down", 122 - torch.arange(n) * far // (n - 1)),
                         ("by 32", 122 - far * (torch.arange(n) // 32 % 2)),
                         ("last of 32", 122 - far * (torch.arange(n) % 32 == 31).long())):
        put_bytes(c, name, torch.where(torch.arange(n) % 50 == 7, 0, bytes_))
        check(c, kind)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("units", FEW)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("down", [9, 14])
def test_large_values_without_weight(rope_gpu, dtype, units, D, down):
    """The keys in the largest units have almost no weight, and the others are 2^-9 or 2^-14 of those units."""
    c = case(units, 24, dtype, D)
    large = torch.arange(400) % 40 == 3
    put_bytes(c, "v", torch.where(large, 122, 122 - down))
    put_bytes(c, "k", torch.where(large, 118, 113))
    for j in range(3, 400, 40):
        put(c, "k", j, code=0xd8)  # -16 / 512: 14 behind the others, whose scores are about 0
    c["q"][:] = c["q"].abs() + 56 * 8 / D ** 0.5
    check(c, "no weight")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("units", FEW)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores_and_ends(rope_gpu, dtype, units, D):
    """Scores thousands apart; zeros with the bytes 0 and 254."""
    c = case(units, 25, dtype, D, q_scale=60.0)
    for j in (3, 40, 100, 300):
        for name in ("k", "v"):
            put(c, name, j, byte=0 if j % 2 else 254, code=0)
    check(c, "large")


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", ["k", "v"])
def test_a_far_scale_that_few_rows_see(rope_gpu, dtype, D, name):
    """A key in units of 2^-30 of the others': rows that see none of the 32 keys around it are as without it."""
    new = [250] if D <= 128 else [125]
    c = coded_case(26, dtype, new, new, hq=1, hk=1, D=D, S=16)
    c["wide"] = True
    n = new[0]
    put_bytes(c, name, 119 + (torch.arange(n) % 3 > 0).long())
    clean, clean_lse = check(c, "clean")
    put(c, name, n - 1, byte=90)
    out, lse = check(c, "far")
    first = (n - 1) // 32 * 32
    assert torch.equal(out[:first], clean[:first]) and torch.equal(lse[:first], clean_lse[:first])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("units", ALL)
@pytest.mark.parametrize("D", [64, 256])
def test_a_scale_that_is_nan_without_weight(rope_gpu, dtype, units, D):
    """V's scale is NaN and its codes are not, of a key of hardly any weight: NaN for the rows that see it, no others."""
    c = led_by_key_4(units, dtype, D)
    b = 0
    n, new = int(c["lens"][b]), int(c["starts"][b + 1])
    put(c, "v", n - 1, byte=255, b=b)
    out, _ = check(c, "nan")
    assert torch.isnan(out[new - 1]).all() and not torch.isnan(out[:new - 1]).any() and not torch.isnan(out[new:]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("units", FEW)
@pytest.mark.parametrize("D", [64, 256, 288])
def test_values_beyond_binary32(rope_gpu, dtype, units, D):
    """Code times scale beyond binary32's range: of V without weight, of K where the query is 0."""
    c = led_by_key_4(units, dtype, D)
    put(c, "v", 130, byte=254, code=0x7e)
    check(c, "v")
    c = case(units, 27, dtype, D)
    bytes_of(c["k_codes"])[:] = 0
    bytes_of(c["k_codes"])[..., 0] = 0x7e
    bytes_of(c["k_scale"])[:] = 254
    c["q"].view(c["q"].shape[0], -1, D)[..., 0] = 0
    check(c, "k")
