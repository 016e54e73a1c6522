"""Pages of a cache: sequences forked, reordered, dropped and given room, live pages moved to the front, pages
copied.  Whole numbers and copied bytes: equal to plain references (tests/codes_ref.py)."""
import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import compact_reference, pages_case, rearrange_reference
from guard import Guards

pytestmark = pytest.mark.gpu
CANARY = -77


def run_rearrange(c, parents, room=None, new_W=None, in_place=False, error=None):
    g = Guards()
    rows, W = len(parents), new_W or c["table"].shape[1]
    full = lambda shape, dtype, n: g.put(torch.full(shape, CANARY, dtype=dtype), n)  # noqa: E731
    refs = g.put(c["refs"], "refs")
    o = {"new_table": full((rows, W), torch.int64, "new_table"), "new_lens": full((rows,), torch.int64, "new_lens"),
         "new_refs": refs if in_place else full((c["NB"],), torch.int32, "new_refs"),
         "src": full((rows,), torch.int64, "src"), "dst": full((rows,), torch.int64, "dst"),
         "counts": full((2,), torch.int64, "counts")}
    R.rearrange_sequences(g.put(c["table"], "table"), g.put(c["lens"], "lens"), refs,
                          g.put(torch.tensor(parents, dtype=torch.int64), "parents"), o["new_table"], o["new_lens"],
                          o["new_refs"], o["src"], o["dst"], o["counts"], c["bs"], prefix_len=c["P"],
                          room=None if room is None else g.put(torch.tensor(room, dtype=torch.int64), "room"))
    g.check()
    o = {k: v.cpu() for k, v in o.items()}
    if error is None:  # free pages enough, or recorded that they are not
        error = R.ROPE_DEVICE_PAGES_EXHAUSTED if bool((o["new_table"] == -1).any()) else 0
    assert R.get_device_error() == error
    return o


def same(got, want):
    for k, v in want.items():
        assert torch.equal(got[k], v), (k, got[k], v)


LENS = [0, 1, 15, 16, 17, 33, 48, 160, 7, 31, 32, 100]


@pytest.mark.parametrize("bs", [1, 7, 16, 64])
@pytest.mark.parametrize("P", [0, 40])
@pytest.mark.parametrize("in_place", [False, True])
def test_rearrange(rope_gpu, bs, P, in_place):
    c = pages_case(1, LENS, bs, P=P, spare=200)
    n = len(LENS)
    g = torch.Generator().manual_seed(2)
    for parents in (list(range(n)), [5], [], [-1] * 4, list(range(n)) * 3, [n - 1 - i for i in range(n)],
                    torch.randint(-1, n, (23,), generator=g).tolist()):
        for room in (None, [(7 * i) % 40 for i in range(len(parents))]):
            width = c["table"].shape[1] + 50
            same(run_rearrange(c, parents, room, width, in_place),
                 rearrange_reference(c, parents, room, width))


@pytest.mark.parametrize("parents", [[0, 1], [1, 0], [1, 1, 0], [1, -1], [0, 0]])
def test_rearrange_a_sequence_cut_short(rope_gpu, parents):
    """Sequence 1 shares whole pages with sequence 0 and was then cut to end inside one: its child may not write on what
    another's child reads."""
    for spare_columns in (2, 6000):  # one CTA, a cluster
        c = pages_case(12, [40, 40], 8, spare=9, share=False, spare_columns=spare_columns)
        c["refs"][c["table"][1, :4]] = 0
        c["table"][1, :4] = c["table"][0, :4]
        c["refs"][c["table"][0, :4]] = 2
        c["refs"][c["table"][1, 4]] = 0
        c["lens"][1] = 27  # pages 0 to 3, the last with three tokens
        same(run_rearrange(c, parents), rearrange_reference(c, parents))


def test_rearrange_many_rows(rope_gpu):
    """More rows than a CTA has threads, more pages than a warp's range has lanes, the most rows that are taken."""
    g = torch.Generator().manual_seed(3)
    for n, rows in ((1500, 3000), (700, 8192)):
        lens = torch.randint(0, 90, (n,), generator=g).tolist()
        c = pages_case(4, lens, 8, spare=40000, share=True)
        parents = torch.randint(-1, n, (rows,), generator=g).tolist()
        room = torch.randint(0, 20, (rows,), generator=g).tolist()
        same(run_rearrange(c, parents, room, 20), rearrange_reference(c, parents, room, 20))


def test_rearrange_holders_outside_the_batch(rope_gpu):
    """A page that is written on and that somebody else holds is copied by all; a page in two old rows, which fork
    without a copy left so, is kept by the first."""
    c = pages_case(5, [20, 20, 20], 16, spare=20, share=False)
    c["refs"][c["table"][0, 1]] += 1
    c["table"][2, 1] = c["table"][1, 1]
    c["refs"][c["table"][1, 1]] += 1
    for parents in ([0, 1, 2], [2, 1, 0, 0, 1]):
        same(run_rearrange(c, parents), rearrange_reference(c, parents))


def test_rearrange_pages_run_out(rope_gpu):
    c = pages_case(6, [20, 33, 5], 16, spare=3, share=False)
    over = []
    for parents, room in (([0, 1, 2, 0, 1, 2], [0] * 6), ([0, 1, 2], [16, 40, 30]), ([1, 1, 1, 1, 0], [1, 1, 1, 1, 100])):
        want = rearrange_reference(c, parents, room, 12)
        over.append(bool((want["new_table"] == -1).any()))
        same(run_rearrange(c, parents, room, 12), want)
    assert over.count(True) >= 2


def test_rearrange_bad_numbers(rope_gpu):
    """Pages outside the cache, parents outside the batch, lengths past the table: passed over, and recorded."""
    c = pages_case(7, [20, 33, 5], 16, spare=9, share=False)
    good = rearrange_reference(c, [0, -1, 2])
    got = run_rearrange(c, [0, 3, 2], error=R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
    same(got, good)
    page = int(c["table"][1, 1])
    c["table"][1, 1] = 1 << 40
    got = run_rearrange(c, [0, 2], error=R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
    assert got["new_refs"][page] == 1  # still held: the table did not name it
    c = pages_case(7, [20, 33, 5], 16, spare=9, share=False, spare_columns=0)
    c["lens"][1] = 1000
    got = run_rearrange(c, [1], error=R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
    assert int(got["new_lens"][0]) == 48


def run_compact(c, pairs=None, in_place=False, error=0):
    g = Guards()
    pairs = c["NB"] // 2 if pairs is None else pairs
    table, refs, prefix = g.put(c["table"], "table"), g.put(c["refs"], "refs"), g.put(c["prefix"], "prefix")
    full = lambda like, n: g.put(torch.full_like(like, CANARY), n)  # noqa: E731
    o = {"new_table": table if in_place else full(c["table"], "new_table"),
         "new_refs": refs if in_place else full(c["refs"], "new_refs"),
         "new_prefix": prefix if in_place else full(c["prefix"], "new_prefix"),
         "src": full(torch.zeros(pairs, dtype=torch.int64), "src"), "dst": full(torch.zeros(pairs, dtype=torch.int64), "dst"),
         "counts": full(torch.zeros(2, dtype=torch.int64), "counts")}
    R.compact_pages(table, g.put(c["lens"], "lens"), refs, o["new_table"], o["new_refs"], o["src"], o["dst"], o["counts"],
                    c["bs"], prefix_blocks=prefix if c["P"] else None, new_prefix_blocks=o["new_prefix"] if c["P"] else None,
                    prefix_len=c["P"])
    g.check()
    assert R.get_device_error() == error
    return {k: v.cpu() for k, v in o.items()}


@pytest.mark.parametrize("bs", [1, 16])
@pytest.mark.parametrize("P", [0, 40])
@pytest.mark.parametrize("spare", [0, 1, 5, 60, 3000, 40000])
def test_compact(rope_gpu, bs, P, spare):
    c = pages_case(8, LENS, bs, P=P, spare=spare)
    want = compact_reference(c, c["NB"] // 2)
    if not P:
        want["new_prefix"] = torch.full_like(c["prefix"], CANARY)
    same(run_compact(c), want)
    got = run_compact(c, pairs=c["NB"] // 2 + 3, in_place=True)
    more = compact_reference(c, c["NB"] // 2 + 3)
    held = more["new_table"] != CANARY
    assert torch.equal(got["new_table"][held], more["new_table"][held])
    assert torch.equal(got["new_table"][~held], c["table"][~held])
    for k in ("new_refs", "src", "dst", "counts"):
        assert torch.equal(got[k], more[k]), k
    if P:
        assert torch.equal(got["new_prefix"], more["new_prefix"])


def test_compact_of_nothing_and_of_bad_entries(rope_gpu):
    c = pages_case(9, [0, 0], 16, spare=50)
    got = run_compact(c)
    assert got["counts"].tolist() == [0, 0] and not got["new_refs"].any() and (got["src"] == -1).all()
    c = pages_case(9, [40, 20], 16, spare=50)
    c["table"][0, 1] = 1 << 40
    got = run_compact(c, error=R.ROPE_DEVICE_SLOT_OUT_OF_RANGE)
    assert int(got["new_table"][0, 1]) == 1 << 40


# ---------------------------------------------------------------------------
# copies
# ---------------------------------------------------------------------------
SHAPES = [((16, 16, 8), torch.bfloat16), ((2, 7), torch.float8_e4m3fn), ((3,), torch.float8_e8m0fnu), ((1,), torch.uint8),
          ((5, 2), torch.int32), ((3, 5000), torch.uint8), ((4097,), torch.float32), ((2, 3, 5), torch.float16)]


def tensors(g, NB, seed, shapes=SHAPES):
    gen = torch.Generator().manual_seed(seed)
    ref = []
    for shape, dtype in shapes:
        n = NB * int(torch.Size(shape).numel()) * torch.empty(0, dtype=dtype).element_size()
        ref.append(torch.randint(0, 256, (n,), generator=gen, dtype=torch.uint8).reshape(NB, -1))
    dev = [g.put(r, str(i)).view(-1).view(d).view(NB, *s) for i, (r, (s, d)) in enumerate(zip(ref, SHAPES if shapes is SHAPES else shapes))]
    return ref, dev


@pytest.mark.parametrize("pairs", [0, 1, 3, 40, 500])
def test_copies(rope_gpu, pairs):
    NB = 1003
    g = Guards()
    ref, dev = tensors(g, NB, pairs)
    order = torch.randperm(NB, generator=torch.Generator().manual_seed(1))
    src, dst = order[:pairs].clone(), order[pairs:2 * pairs].clone()
    src[2::7] = -1
    dst[3::7] = -5
    for count in (None, torch.tensor([pairs // 2, 9]), torch.tensor([pairs + 100]), torch.tensor([-3])):
        want = [r.clone() for r in ref]
        n = pairs if count is None else min(max(int(count[0]), 0), pairs)
        for a, b in zip(src[:n].tolist(), dst[:n].tolist()):
            if a >= 0 and b >= 0:
                for w in want:
                    w[b] = w[a]
        R.copy_pages(g.put(src, "src"), g.put(dst, "dst"), dev, count=None if count is None else g.put(count, "count"))
        g.check()
        for w, d in zip(want, dev):
            assert torch.equal(d.view(torch.uint8).reshape(NB, -1).cpu() if d.dtype != torch.uint8 else d.reshape(NB, -1).cpu(), w)
            d.view(torch.uint8).reshape(-1).copy_(ref[[x is d for x in dev].index(True)].reshape(-1).cuda())
    assert R.get_device_error() == 0


def test_copies_at_odd_addresses_and_of_many_tensors(rope_gpu):
    NB = 9
    g = Guards()
    dev = [g.put(torch.full((NB, 33 + i), i, dtype=torch.uint8).add_(torch.arange(NB, dtype=torch.uint8)[:, None]), str(i), offset=i % 17)
           for i in range(150)]
    want = [d.cpu().clone() for d in dev]
    for w in want:
        w[7] = w[2]
        w[0] = w[8]
    R.copy_pages(torch.tensor([2, 8]).cuda(), torch.tensor([7, 0]).cuda(), dev)
    g.check()
    assert all(torch.equal(d.cpu(), w) for d, w in zip(dev, want))


def test_copies_of_pages_outside(rope_gpu):
    g = Guards()
    ref, dev = tensors(g, 10, 3)
    R.copy_pages(torch.tensor([1, 10, 3]).cuda(), torch.tensor([2, 4, 1 << 40]).cuda(), tuple(dev))
    g.check()
    assert R.get_device_error() == R.ROPE_DEVICE_SLOT_OUT_OF_RANGE
    for r, d in zip(ref, dev):
        r = r.clone()
        r[2] = r[1]
        assert torch.equal(d.contiguous().view(torch.uint8).reshape(10, -1).cpu(), r)
