"""Paged attention where its units follow one another in ways that small batches do not reach: many units a CTA of every
shape, against a float64 reference (bounds: tests/serving_ref.py)."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from serving_ref import E32, TINY, assert_close, half_step, run_attend, widened

pytestmark = pytest.mark.gpu


def batch(seed, dtype, new, own, P, hq, hk, D, bs):
    """As serving_ref.attend_case, for large batches: on the GPU, all tokens at once."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, T = len(new), sum(new)
    held = [-(-n // bs) for n in own]
    shared = -(-P // bs)
    NB = shared + sum(held) + 2
    pages = torch.randperm(NB, generator=g, device="cuda")
    table = torch.full((B, max(held) + 1), 1 << 40, dtype=torch.int64, device="cuda")
    k = torch.full((NB, hk, bs, D), float("nan"), dtype=dtype, device="cuda")
    v = k.clone()
    at, prefix = shared, pages[:shared].clone()
    page, row = [prefix[torch.arange(P, device="cuda") // bs]], [torch.arange(P, device="cuda") % bs]
    for b in range(B):
        table[b, :held[b]] = pages[at:at + held[b]]
        j = torch.arange(own[b], device="cuda")
        page.append(table[b, j // bs])
        row.append(j % bs)
        at += held[b]
    page, row = torch.cat(page), torch.cat(row)
    for cache in (k, v):
        cache[page, :, row] = torch.randn(len(page), hk, D, generator=g, device="cuda").to(dtype)
    return {"q": torch.randn(T, hq * D, generator=g, device="cuda").to(dtype), "width": hq * D, "k": k, "v": v,
            "table": table, "lens": torch.tensor([P + n for n in own], device="cuda"),
            "starts": torch.tensor([0] + list(new), device="cuda").cumsum(0), "prefix": prefix, "P": P, "hq": hq,
            "hk": hk, "D": D, "bs": bs, "T": T, "scale": D ** -0.5}


def reference(c, new, own):
    """(out, lse, out bound, lse bound), a sequence at a time."""
    hq, hk, D, bs, P = (c[x] for x in ("hq", "hk", "D", "bs", "P"))
    dtype = c["q"].dtype
    uw = 0.0 if dtype == torch.float32 else half_step(dtype)
    res = [[], [], [], []]
    t = 0
    for b, (n, m) in enumerate(zip(new, own)):
        j = torch.arange(P + m, device="cuda")
        page = torch.cat([c["prefix"][j[:P] // bs], c["table"][b, (j[P:] - P) // bs]])
        row = torch.cat([j[:P] % bs, (j[P:] - P) % bs])
        k, v = (c[x][page, :, row].double().transpose(0, 1)[:, None] for x in ("k", "v"))  # [hk, 1, keys, D]
        q = c["q"][t:t + n].double().view(n, hk, hq // hk, D).permute(1, 2, 0, 3)
        late = j[None] > (P + m - n + torch.arange(n, device="cuda"))[:, None]
        s = (q @ k.transpose(-1, -2) * c["scale"]).masked_fill(late, float("-inf"))
        big = (q.abs() @ k.abs().transpose(-1, -2) * c["scale"]).masked_fill(late, 0).amax(-1)
        w = torch.softmax(s, -1)
        o, A, lse = w @ v, w @ v.abs(), torch.logsumexp(s, -1)
        seen = (~late).sum(-1).double()
        d = 2 * (D + 4) * E32 * big
        tol = half_step(dtype) * o.abs() + (uw + 2 * d + (4 * seen + 64) * E32)[..., None] * A + TINY[dtype]
        ltol = d + (seen + 64) * E32 + 4 * E32 * lse.abs()
        for x, y in zip(res, (o, lse, tol, ltol)):
            x.append((y.permute(2, 0, 1, 3).reshape(n, -1) if y.dim() == 4 else y.permute(2, 0, 1).reshape(n, -1)).cpu())
        t += n
    return [torch.cat(x) for x in res]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("P", [0, 70])
def test_short_prompts_between_longer_ones(rope_gpu, dtype, D, P):
    """About 30 units a CTA: runs of more than 16 of one row tile and one key tile, then units of two row tiles, or of
    one with several key tiles, which the second softmax group has a part of again."""
    new, own = [], []
    for i in range(140):
        n = 40 + (i * 37) % 61 if i % 4 else 130 + (i * 53) % 121
        if i % 8 == 4:  # few rows behind many keys
            new.append(1 + i % 9)
            own.append(129 + (i * 31) % 272)
        else:
            new.append(n)
            own.append(n)
    c = batch(31, dtype, new, own, P, 32, 32, D, 16)
    ro, rl, to, tl = reference(c, new, own)
    wide = widened({k: v.cpu() if k == "table" else v for k, v in c.items()})
    for case in (c, wide):
        out, lse = run_attend(R, case)
        assert_close(out, ro, to, "out")
        assert_close(lse, rl, tl, "lse")
        assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("lead", [15.0, 17.6])
@pytest.mark.parametrize("D,new,G", [(64, 1, 8), (128, 1, 16), (256, 1, 4), (256, 2, 8), (64, 40, 8), (128, 17, 8), (256, 20, 8)])
def test_one_key_far_above_many(rope_gpu, dtype, lead, D, new, G):
    """One key leads 20000 others by so much that the weights of these, relative to its own, are below the smallest
    normal binary16 (15 nats) or below half its smallest value (17.6); together they are the whole of the output, as
    the leading key's value is 0.  So many sequences, all on the same pages, that a CTA takes them whole."""
    n, bs = 20000, 64
    B = 304
    g = torch.Generator(device="cuda").manual_seed(32)
    pages = -(-n // bs)
    k = torch.zeros(pages, 1, bs, D, dtype=dtype, device="cuda")
    v = (1 + 0.1 * torch.randn(pages, 1, bs, D, generator=g, device="cuda")).to(dtype)
    k[0, 0, 3], v[0, 0, 3] = lead * D ** -0.5, 0
    q = (1 + torch.arange(new * G, device="cuda")[:, None] % 8 / 256).expand(-1, D).reshape(new, G * D).to(dtype)
    one = {"q": q, "k": k, "v": v, "table": torch.arange(pages, device="cuda")[None], "width": G * D,
           "lens": torch.tensor([n], device="cuda"), "starts": torch.tensor([0, new], device="cuda"),
           "prefix": torch.zeros(0, dtype=torch.int64, device="cuda"), "P": 0, "hq": G, "hk": 1, "D": D, "bs": bs,
           "T": new, "scale": D ** -0.5}
    ro, rl, to, tl = reference(one, [new], [n])
    many = dict(one, q=q.repeat(B, 1), table=one["table"].repeat(B, 1), lens=one["lens"].repeat(B), T=new * B,
                starts=torch.arange(B + 1, device="cuda") * new)
    for c, times in ((one, 1), (many, B)):
        out, lse = run_attend(R, c)
        assert_close(out, ro.repeat(times, 1), to.repeat(times, 1), "out of %d" % times)
        assert_close(lse, rl.repeat(times, 1), tl.repeat(times, 1), "lse of %d" % times)
        assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D,new,own,P", [(64, [1, 1, 1], [70, 5, 300], 0), (128, [1, 2, 1], [40, 3, 2000], 40),
                                         (64, [90, 40, 3], [90, 500, 20], 0), (128, [90, 140], [400, 140], 30),
                                         (256, [90, 40], [90, 500], 0), (288, [1, 20], [30, 20], 3)])
def test_products_beyond_binary32(rope_gpu, dtype, sign, D, new, own, P):
    """Scores of -9 to -5 (or 5 to 9) with a scale of 2^-126: every product of a query and a key is beyond
    binary32.  A sequence of no tokens yet (length 0) beside them sees nothing."""
    c = batch(33, dtype, new + [1], own + [1], P, 4, 2, D, 16)
    q, k = c["q"], c["k"]
    q[:] = 2.0 ** 64
    k.copy_(torch.where(torch.isnan(k), k, sign * (5 + 4 * torch.rand_like(k, dtype=torch.float32).to(dtype)) * 2.0 ** 62 / D))
    c["scale"] = 2.0 ** -126
    c["lens"][-1] = 0
    ro, rl, to, tl = reference(c, new, own)
    for case in (c, widened({x: y.cpu() if x == "table" else y for x, y in c.items()})):
        out, lse = run_attend(R, case)
        assert_close(out[:-1], ro, to, "out")
        assert_close(lse[:-1], rl, tl, "lse")
        assert not out[-1].any() and torch.equal(lse[-1], torch.full((4,), float("-inf")))
        assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_products_beyond_binary32_behind_a_shared_prefix(rope_gpu, dtype):
    """The same with a launch for the prefix."""
    n = 60
    new, own = [1] * n, [1 + (i * 7) % 50 for i in range(n)]
    c = batch(34, dtype, new + [1], own + [1], 1000, 4, 2, 128, 16)
    c["q"][:] = 2.0 ** 64
    k = c["k"]
    k.copy_(torch.where(torch.isnan(k), k, -(5 + 4 * torch.rand_like(k, dtype=torch.float32).to(dtype)) * 2.0 ** 62 / 128))
    c["scale"] = 2.0 ** -126
    c["lens"][-1] = 0
    ro, rl, to, tl = reference(c, new, own)
    before = R.launch_count()
    out, lse = run_attend(R, c)
    assert R.launch_count() - before == 3
    assert_close(out[:-1], ro, to, "out")
    assert_close(lse[:-1], rl, tl, "lse")
    assert not out[-1].any() and torch.equal(lse[-1], torch.full((4,), float("-inf")))
    assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 32), (torch.float32, 16)], ids=str)
def test_cache_of_more_than_2_31_rows(rope_gpu, dtype, D):
    """The smallest heads with so many pages that a cache row no longer fits 32 bits (137 GB, keys and values in one
    tensor, of which only the pages in use are ever written)."""
    bs, NB = 128, (1 << 24) + 8
    if torch.cuda.mem_get_info()[0] < NB * bs * 64 + (8 << 30):
        pytest.skip("needs 146 GB")
    cache = torch.empty(NB, 1, bs, D, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(35)
    table = torch.tensor([[NB - 1, 0, NB - 7], [1, NB - 2, 3], [(1 << 24) - 1, 1 << 24, 5]], device="cuda")
    prefix = torch.tensor([NB - 3, 7], device="cuda")
    for page in torch.cat([table.flatten(), prefix]).tolist():
        cache[page] = torch.randn(1, bs, D, generator=g, device="cuda").to(dtype)
    new, own, P = [1, 130, 40], [300, 200, 384], 150
    c = {"q": torch.randn(sum(new), 4 * D, generator=g, device="cuda").to(dtype), "width": 4 * D, "k": cache, "v": cache,
         "table": table, "lens": torch.tensor([P + n for n in own], device="cuda"),
         "starts": torch.tensor([0] + new, device="cuda").cumsum(0), "prefix": prefix, "P": P, "hq": 4, "hk": 1,
         "D": D, "bs": bs, "scale": D ** -0.5}
    ro, rl, to, tl = reference(c, new, own)
    out = torch.empty(sum(new), 4 * D, dtype=dtype, device="cuda")
    lse = torch.empty(sum(new), 4, device="cuda")
    R.paged_attention(c["q"], cache, cache, table, c["lens"], c["starts"], out, prefix_blocks=prefix, prefix_len=P, lse=lse)
    assert_close(out, ro, to, "out")
    assert_close(lse, rl, tl, "lse")
    assert R.get_device_error() == 0
    del cache, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,own", [([1, 1], [300, 40]), ([3, 1], [300, 1000]), ([40, 60], [300, 900])])
def test_scores_of_which_one_unit_is_less_than_a_step(rope_gpu, dtype, D, new, own):
    """Scores of 2^23 to 2^31, where binary32 steps by 1 to 256, thousands apart: the key that leads has all the
    weight, so its value is the result (rounded once: half a step, and 2^-20 for sums and weights).  The score itself is a sum of up to 13 rounded
    parts with 5 more roundings of scales and units, each 2^-24: 2^-19."""
    for power in range(0, 9):
        c = batch(36, dtype, new, own, 0, 8, 2, D, 16)
        k = c["k"]
        step = 2 ** -7 if dtype == torch.bfloat16 else 2 ** -10  # of the keys, relative
        fall = 1 - step * (1 + torch.randint(0, 50, k.shape[:3], device="cuda")[..., None])
        k.copy_(torch.where(torch.isnan(k), k, (512 * fall).to(dtype).expand_as(k)))
        lead = [(int(c["table"][b, 0]), min(n - 1, 3) if n > a + 3 else 0) for b, (a, n) in enumerate(zip(new, own))]
        for page, row in lead:
            k[page, :, row] = 512
        c["q"][:] = 4096 / (D // 64)
        c["scale"] = 0.0625 * 2.0 ** power
        want = torch.cat([c["v"][page, :, row].double()[None, :, None].expand(a, 2, 4, D).reshape(a, -1)
                          for (page, row), a in zip(lead, new)]).cpu()
        for case in (c, widened({x: y.cpu() if x == "table" else y for x, y in c.items()})):
            out, lse = run_attend(R, case)
            assert_close(out, want, (half_step(dtype) + 2.0 ** -20) * want.abs() + TINY[dtype], "out at 2^%d" % power)
            top = 64 * 4096 * 512 * c["scale"]
            assert_close(lse, torch.full((sum(new), 8), top, dtype=torch.float64),
                         torch.full((sum(new), 8), top * 2.0 ** -19), "lse at 2^%d" % power)
            assert R.get_device_error() == 0
