"""The operators on a paged cache of 8-bit codes and on its pages together and in the ways programs call them: prompts,
beams that fork and die, compaction, captured graphs, other streams, threads, prepared calls, large caches."""
import math
import threading

import pytest
import torch

import transformer_rope_positional_gb300 as R
from codes_ref import bytes_of, check_codes, codes_append_case, codes_append_reference, coded_case, e8m0, run_coded, values_of
from serving_ref import append_bound, assert_close, attend_reference

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


class Program:
    """Sequences behind a shared prefix: what a serving program keeps."""

    def __init__(self, dtype, B, P, D=64, hq=4, hk=2, bs=16, S=2, NB=60, W=6, most=128, spare_rows=0):
        self.dtype, self.P, self.D, self.hq, self.hk, self.bs, self.S, self.NB = dtype, P, D, hq, hk, bs, S, NB
        self.g = torch.Generator().manual_seed(7)
        self.table = torch.randn(256, D, generator=self.g).to(dtype).cuda()
        self.caches = [torch.full((NB, hk, bs, D), 0x7f, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
        self.caches += [e8m0(torch.full((NB, hk, S), 255)).cuda() for _ in range(2)]
        shared = -(-P // bs)
        self.prefix = torch.arange(3, 3 + shared, device="cuda")
        self.refs = torch.zeros(NB, dtype=torch.int32, device="cuda")
        self.refs[self.prefix] = 1
        self.blocks = torch.full((most, W), -1, dtype=torch.int64, device="cuda")
        self.lens = torch.full((B,), P, dtype=torch.int64, device="cuda")
        self.most, self.W = most, W

    def rearrange(self, parents, room):
        n = len(parents)
        new_blocks = torch.full((n, self.W), -1, dtype=torch.int64, device="cuda")
        new_lens, src, dst = (torch.empty(n, dtype=torch.int64, device="cuda") for _ in range(3))
        counts = torch.empty(2, dtype=torch.int64, device="cuda")
        R.rearrange_sequences(self.blocks[:len(self.lens)], self.lens, self.refs, torch.tensor(parents, device="cuda"),
                              new_blocks, new_lens, self.refs, src, dst, counts, self.bs,
                              room=torch.tensor(room, device="cuda"), prefix_len=self.P)
        R.copy_pages(src, dst, self.caches, count=counts[:1])
        self.blocks, self.lens = new_blocks, new_lens

    def slots(self, new):
        """Of the last new[b] tokens of every sequence."""
        lens, blocks = self.lens.tolist(), self.blocks.tolist()
        at = [(b, j) for b, n in enumerate(new) for j in range(lens[b] - n, lens[b])]
        return (torch.tensor([blocks[b][(j - self.P) // self.bs] * self.bs + (j - self.P) % self.bs for b, j in at]),
                torch.tensor([j for _, j in at]))

    def append(self, slots, pos):
        T = len(slots)
        x = [torch.randn(T, h * self.D, generator=self.g).to(self.dtype) for h in (self.hq, self.hk, self.hk)]
        q_out = torch.empty(T, self.hq * self.D, device="cuda", dtype=self.dtype)
        R.append_paged_kv_8bit(pos.cuda(), *(t.cuda() for t in x), self.table, slots.cuda(), *self.caches, self.D,
                               query_out=q_out)
        return x, q_out

    def attend(self, q, new, out=None, **kw):
        starts = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), device="cuda")
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[0], self.hq, device="cuda")
        R.paged_attention_8bit(q, *self.caches, self.blocks[:len(new)], self.lens, starts, out,
                               prefix_blocks=self.prefix if self.P else None, prefix_len=self.P, lse=lse, **kw)
        c = {"q": q.cpu(), "width": q.shape[1], "hq": self.hq, "hk": self.hk, "D": self.D, "bs": self.bs, "P": self.P,
             "k": values_of(self.caches[0].cpu(), self.caches[2].cpu()), "v": values_of(self.caches[1].cpu(), self.caches[3].cpu()),
             "table": self.blocks.cpu(), "lens": self.lens.cpu(), "starts": starts.cpu(), "prefix": self.prefix.cpu(),
             "scale": 1 / math.sqrt(self.D)}
        ro, rl, to, tl = attend_reference(c)
        assert_close(out, ro, to, "out")
        assert_close(lse, rl, tl, "lse")
        return out, lse

    def held(self, b):
        """[2, tokens, hk, D]: the values that sequence b holds of its own."""
        n = int(self.lens[b]) - self.P
        pages = self.blocks[b, :-(-n // self.bs)].cpu()
        x = [values_of(self.caches[i].cpu(), self.caches[2 + i].cpu())[pages].transpose(1, 2).reshape(-1, self.hk, self.D)[:n]
             for i in range(2)]
        return torch.stack(x)

    def rotated(self, k, pos):
        """In float64."""
        h = self.D // 2
        x = k.double().view(len(pos), self.hk, self.D)
        c, s = (t[:, None] for t in self.table.cpu().double()[pos].split(h, 1))
        return torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)

    def check_refs(self):
        """As many holders of each page as the tables say."""
        want = torch.zeros(self.NB, dtype=torch.int32)
        for p in self.prefix.tolist():
            want[p] += 1
        for b, n in enumerate(self.lens.tolist()):
            for p in self.blocks[b, :-(-(n - self.P) // self.bs)].tolist():
                want[p] += 1
        assert torch.equal(self.refs.cpu(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("bs,S", [(16, 1), (16, 4), (8, 8)])
def test_beams_of_a_serving_program(rope_gpu, dtype, bs, S):
    """A shared prompt; a chunk for each of two sequences; beams that fork, reorder and die, a token a step, every step:
    what a beam holds is what its parent held, plus the token, and the attention over it is right; then the cache is
    compacted and made smaller, and answers the same bits."""
    P = 37
    p = Program(dtype, 2, P, bs=bs, S=S, W=96 // bs)
    slots = (p.prefix.cpu()[:, None] * bs + torch.arange(bs)).reshape(-1)[:P]
    p.append(slots, torch.arange(P))
    p.rearrange([0, 1], [21, bs])
    new = [21, bs]
    held = None
    for parents in (None, [0, 0, 1], [2, 0, 0, 1, 1], [4, 3, -1, 1], [3, 3, 3, 0, 1, 2], [5, 4, 0], [0, 1, 2], [2]):
        if parents is not None:
            p.rearrange(parents, [1] * len(parents))
            new = [1] * len(parents)
        p.check_refs()
        slots, pos = p.slots(new)
        if parents is not None:  # (before the token is written; the child's own page holds what the parent's did)
            for b, parent in enumerate(parents):
                n = held[parent].shape[1] if parent >= 0 else 0
                assert torch.equal(p.held(b)[:, :n], held[parent][:, :n] if parent >= 0 else p.held(b)[:, :0])
        (q, k, v), q_out = p.append(slots, pos)
        # the last token of each: half a step of E4M3 and what a subnormal's step is in units of its block, which no other token
        # makes larger than 2^-9 of 2^e, 448 * 2^(e - 1) < most; K's two roundings are nothing beside it
        at = torch.tensor(new).cumsum(0) - 1
        held = [p.held(b) for b in range(len(new))]
        for i, x in ((0, p.rotated(k, pos)), (1, v.double().view(-1, p.hk, p.D))):
            b = bytes_of(p.caches[2 + i]).cpu()[slots[at] // bs, :, slots[at] % bs // (bs // S)].double()[..., None]
            last = torch.stack([h[i, -1] for h in held])
            assert bool(((last - x[at]).abs() <= (2.0 ** -4 + 2.0 ** -20) * x[at].abs() + 2.0 ** (b - 127 - 10) * (1 + 2.0 ** -8)).all())
        out, lse = p.attend(q_out, new)
    # ---- compaction
    NB = p.NB
    new_blocks, new_refs = torch.full_like(p.blocks, -1), torch.empty_like(p.refs)
    new_prefix = torch.empty_like(p.prefix)
    src, dst = (torch.empty(NB // 2, dtype=torch.int64, device="cuda") for _ in range(2))
    counts = torch.empty(2, dtype=torch.int64, device="cuda")
    R.compact_pages(p.blocks, p.lens, p.refs, new_blocks, new_refs, src, dst, counts, bs, prefix_blocks=p.prefix,
                    new_prefix_blocks=new_prefix, prefix_len=P)
    R.copy_pages(src, dst, p.caches, count=counts[:1])
    live = int(counts[1])
    assert live == int((p.refs > 0).sum())
    p.blocks, p.refs, p.prefix, p.NB = new_blocks, new_refs[:live].clone(), new_prefix, live
    p.caches = [bytes_of(x)[:live].clone().view(x.dtype) for x in p.caches]
    p.check_refs()
    out2, lse2 = p.attend(q_out, new)
    assert torch.equal(out.view(torch.uint8), out2.view(torch.uint8)) and torch.equal(lse, lse2)
    assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_step_in_a_graph(rope_gpu, dtype):
    """A whole step captured, with the slots worked out on the device, and replayed as the sequences grow and fork: the
    same bits as the calls one by one."""
    D, hq, hk, bs, B, NB, W = 64, 4, 2, 8, 5, 40, 4
    g = torch.Generator().manual_seed(3)
    table = torch.randn(64, D, generator=g).to(dtype).cuda()
    steps = [([0, 0, 1, 2, 3], 1), ([4, 4, 4, 0, 1], 1), ([0, 1, 2, 3, 4], 1), ([3, -1, 0, 0, 1], 1)] * 4
    xs = [[torch.randn(B, h * D, generator=g).to(dtype).cuda() for h in (hq, hk, hk)] for _ in steps]

    def start():
        s = {"blocks": torch.full((B, W), -1, dtype=torch.int64), "new_blocks": torch.full((B, W), -1, dtype=torch.int64),
             "lens": torch.zeros(B, dtype=torch.int64), "new_lens": torch.zeros(B, dtype=torch.int64),
             "refs": torch.zeros(NB, dtype=torch.int32), "parents": torch.arange(B), "room": torch.ones(B, dtype=torch.int64),
             "src": torch.zeros(B, dtype=torch.int64), "dst": torch.zeros(B, dtype=torch.int64),
             "counts": torch.zeros(2, dtype=torch.int64), "starts": torch.arange(B + 1),
             "q": torch.zeros(B, hq * D, dtype=dtype), "k": torch.zeros(B, hk * D, dtype=dtype), "v": torch.zeros(B, hk * D, dtype=dtype),
             "q_out": torch.zeros(B, hq * D, dtype=dtype), "out": torch.zeros(B, hq * D, dtype=dtype)}
        s = {n: t.cuda() for n, t in s.items()}
        s["caches"] = [torch.zeros(NB, hk, bs, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
        s["caches"] += [e8m0(torch.zeros(NB, hk, 1)).cuda() for _ in range(2)]
        return s

    def step(s):
        R.rearrange_sequences(s["blocks"], s["lens"], s["refs"], s["parents"], s["new_blocks"], s["new_lens"], s["refs"],
                              s["src"], s["dst"], s["counts"], bs, room=s["room"])
        R.copy_pages(s["src"], s["dst"], s["caches"], count=s["counts"][:1])
        s["blocks"].copy_(s["new_blocks"])
        s["lens"].copy_(s["new_lens"])
        pos = s["lens"] - 1
        slots = s["blocks"].gather(1, (pos // bs)[:, None])[:, 0] * bs + pos % bs
        R.append_paged_kv_8bit(pos, s["q"], s["k"], s["v"], table, slots, *s["caches"], D, query_out=s["q_out"])
        R.paged_attention_8bit(s["q_out"], *s["caches"], s["blocks"], s["lens"], s["starts"], s["out"])

    def feed(s, i):
        s["parents"].copy_(torch.tensor(steps[i][0]))
        for n, x in zip("qkv", xs[i]):
            s[n].copy_(x)

    eager, got = start(), start()
    step(start())  # what the first call sets up is not captured
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(got)
    torch.cuda.synchronize()
    for i in range(len(steps)):
        feed(eager, i)
        step(eager)
        feed(got, i)
        graph.replay()
        torch.cuda.synchronize()
        for n in ("blocks", "lens", "refs", "out", "q_out"):
            assert torch.equal(eager[n].view(torch.uint8), got[n].view(torch.uint8)), (i, n)
        assert bool(torch.isfinite(got["out"].float()).all())
    assert R.get_device_error() == 0


def test_two_graphs_with_one_workspace(rope_gpu):
    """Captured calls that are given the same workspace, replayed one after the other on one stream."""
    cs = [coded_case(33 + i, torch.bfloat16, [1, 2], own, P=P, hq=8, hk=2, D=128)
          for i, (own, P) in enumerate((([2600, 90], 0), ([30, 40], 900)))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    runs = []
    need = max(R.paged_attention_workspace(c["q"].cuda(), c["k_codes"].cuda(), c["P"]) for c in cs)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xff)
    for c in cs:
        d = {k: (bytes_of(v).cuda().view(v.dtype) if v.element_size() == 1 else v.cuda()) for k, v in c.items()
             if isinstance(v, torch.Tensor)}
        out = torch.empty(3, c["width"], device="cuda", dtype=torch.bfloat16)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                R.paged_attention_8bit(d["q"], d["k_codes"], d["v_codes"], d["k_scale"], d["v_scale"], d["table"], d["lens"],
                                       d["starts"], out, scale=c["scale"], prefix_blocks=d["prefix"] if c["P"] else None,
                                       prefix_len=c["P"], workspace=ws)
        runs.append((graph, out, attend_reference(c), d))
    with torch.cuda.stream(s):
        for _ in range(3):
            for graph, *_ in runs:
                graph.replay()
    torch.cuda.synchronize()
    for _, out, ref, _ in runs:
        assert_close(out, ref[0], ref[2], "shared workspace")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_workspace_contents_do_not_matter(rope_gpu, dtype):
    c = coded_case(35, dtype, [1, 3, 1], [700, 20, 3], P=300, hq=4, hk=2, D=64)
    n = R.paged_attention_workspace(c["q"].cuda(), c["k_codes"].cuda(), 300)
    ref = attend_reference(c)
    for fill in (0x00, 0xff, 0x7f):
        ws = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")[:n]
        out, lse = run_coded(R, c, workspace=ws)
        assert_close(out, ref[0], ref[2], "workspace")
        assert_close(lse, ref[1], ref[3], "workspace lse")
    with pytest.raises(R.RopeError):
        run_coded(R, c, workspace=torch.empty(n - 256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        run_coded(R, c, workspace=torch.empty(n, dtype=torch.uint8))


def test_streams_prepared_calls_and_threads(rope_gpu):
    """Calls on streams other than the current one (object and handle), prepared calls, and calls from several threads at
    once, each with sequences, codes and pages of its own."""
    c = coded_case(36, torch.bfloat16, [1, 2, 9], [300, 5, 60], P=130, hq=8, hk=2, D=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ref = attend_reference(c)
    for kw in ({"stream": s}, {"stream": s.cuda_stream}, {"prepared": True}):
        out, _ = run_coded(R, c, **kw)
        assert_close(out, ref[0], ref[2], str(kw))
    a = codes_append_case(20, torch.bfloat16, [3, 1, 40], [5, 0, 20], 16, 1)
    q_ref, _, (kr, vr) = codes_append_reference(a)
    errors = []

    def work(i):
        try:
            mine = torch.cuda.Stream()
            up = lambda v: bytes_of(v).cuda().view(v.dtype) if v.element_size() == 1 else v.cuda()  # noqa: E731
            with torch.cuda.stream(mine):
                d = {k: up(v) for k, v in c.items() if isinstance(v, torch.Tensor)}
                for _ in range(10):
                    o = torch.full((c["T"], c["width"]), float("nan"), device="cuda", dtype=torch.bfloat16)
                    R.paged_attention_8bit(d["q"], d["k_codes"], d["v_codes"], d["k_scale"], d["v_scale"], d["table"], d["lens"],
                                           d["starts"], o, scale=c["scale"], prefix_blocks=d["prefix"], prefix_len=130)
                    e = {k: up(v) for k, v in a.items() if isinstance(v, torch.Tensor)}
                    qo = torch.empty_like(e["q"])
                    R.append_paged_kv_8bit(e["pos"], e["q"], e["k"], e["v"], e["table"], e["slots"], e["kc"], e["vc"], e["ks"],
                                           e["vs"], a["D"], is_neox=a["neox"], query_out=qo)
                    refs = torch.zeros(9, dtype=torch.int32, device="cuda")
                    n = torch.arange(2, device="cuda")
                    blocks, lens = torch.full((2, 3), -1, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
                    nb, nl, src, dst = blocks.clone(), lens.clone(), lens.clone(), lens.clone()
                    R.rearrange_sequences(blocks, lens, refs, n, nb, nl, refs, src, dst, torch.zeros_like(lens), 4,
                                          room=torch.full_like(lens, 7 + i % 2))
                    mine.synchronize()
                    assert_close(o, ref[0], ref[2], "thread %d" % i)
                    check_codes(e["kc"], e["ks"], kr, "thread k")
                    check_codes(e["vc"], e["vs"], vr, "thread v")
                    assert_close(qo, q_ref, append_bound(q_ref, torch.bfloat16), "thread q")
                    assert nb.tolist() == [[0, 1, -1], [2, 3, -1]] and refs.tolist() == [1] * 4 + [0] * 5
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    assert R.get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("n", [33, 130, 500, 1100])
def test_many_sequences(rope_gpu, dtype, n):
    """More sequences than a warp, a CTA, and several CTAs' threads look at in one pass; some are empty."""
    new = [0 if i % 7 == 3 else 1 for i in range(n)]
    own = [1 + (i * 5) % 23 for i in range(n)]
    c = coded_case(37, dtype, new, own, P=0, hq=2, hk=1, D=32, bs=8)
    ref = attend_reference(c)
    out, lse = run_coded(R, c)
    assert_close(out, ref[0], ref[2], "many")
    assert_close(lse, ref[1], ref[3], "many lse")


def test_many_sequences_of_several_tokens(rope_gpu):
    new = [1 + (i * 3) % 20 for i in range(70)]
    own = [new[i] + (i * 11) % 50 for i in range(70)]
    c = coded_case(38, torch.float16, new, own, P=20, hq=8, hk=2, D=64)
    ref = attend_reference(c)
    out, _ = run_coded(R, c)
    assert_close(out, ref[0], ref[2], "many chunks")


def test_cache_past_32_bit_offsets(rope_gpu):
    """Pages whose codes lie past 2^31 and 2^32: attention, append (of few tokens and of many), copies."""
    D, hk, bs = 128, 8, 64
    NB = (1 << 32) // (hk * bs * D) + 40
    if torch.cuda.mem_get_info()[0] < 3 * NB * hk * bs * D:
        pytest.skip("needs 13 GB")
    small = coded_case(39, torch.bfloat16, [1, 30], [150, 64], P=64, hq=16, hk=hk, D=D, bs=bs)
    n = small["k"].shape[0]
    pages = torch.tensor([NB - 1 - 3 * i for i in range(n)])
    big = {}
    for name, shape in (("k_codes", (NB, hk, bs, D)), ("v_codes", (NB, hk, bs, D)), ("k_scale", (NB, hk, 1)), ("v_scale", (NB, hk, 1))):
        x = torch.empty(shape, dtype=torch.uint8, device="cuda")
        x[pages.cuda()] = bytes_of(small[name]).cuda()
        big[name] = x.view(small[name].dtype)
    table = torch.where(small["table"] < n, pages[small["table"].clamp(max=n - 1)], small["table"])
    out = torch.empty(31, 16 * D, device="cuda", dtype=torch.bfloat16)
    ref = attend_reference(small)
    R.paged_attention_8bit(small["q"].cuda(), *big.values(), table.cuda(), small["lens"].cuda(), small["starts"].cuda(), out,
                           scale=small["scale"], prefix_blocks=pages[small["prefix"]].cuda(), prefix_len=64)
    assert_close(out, ref[0], ref[2], "large cache")
    # copies between its ends, and the attention over these
    other = torch.arange(n)
    R.copy_pages(pages.cuda(), other.cuda(), list(big.values()))
    out.fill_(float("nan"))
    R.paged_attention_8bit(small["q"].cuda(), *big.values(), small["table"].cuda(), small["lens"].cuda(),
                           small["starts"].cuda(), out, scale=small["scale"], prefix_blocks=small["prefix"].cuda(), prefix_len=64)
    assert_close(out, ref[0], ref[2], "copied pages")
    for rows in (0, 1030):
        c = codes_append_case(40, torch.bfloat16, [5, 70], [3, 100], bs, 1, hq=8, hk=hk, D=D)
        if rows:
            from test_gpu_append_codes_many import padded
            c = padded(c, rows)
        m = c["kc"].shape[0]
        for name, x in (("k_codes", "kc"), ("v_codes", "vc"), ("k_scale", "ks"), ("v_scale", "vs")):
            bytes_of(big[name])[-m:] = bytes_of(c[x]).cuda()
        qo = torch.empty(c["q"].shape, device="cuda", dtype=torch.bfloat16)
        slots = torch.where(c["slots"] >= 0, c["slots"] + (NB - m) * bs, c["slots"])
        R.append_paged_kv_8bit(c["pos"].cuda(), c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), c["table"].cuda(), slots.cuda(),
                               *big.values(), D, is_neox=c["neox"], query_out=qo)
        q_ref, _, (kr, vr) = codes_append_reference(c)
        check_codes(big["k_codes"][-m:], big["k_scale"][-m:], kr, "k")
        check_codes(big["v_codes"][-m:], big["v_scale"][-m:], vr, "v")
        assert_close(qo, q_ref, append_bound(q_ref, torch.bfloat16), "q")
    assert R.get_device_error() == 0


def test_unordered_starts_stay_inside_the_tensors(rope_gpu):
    """Values of query_start_loc and seq_lens that mean nothing: unspecified rows, but no access outside a tensor
    (the guard bands hold, and the bounds-checking build reports nothing), and later calls are not disturbed."""
    for dtype in (torch.float32, torch.bfloat16):
        c = coded_case(41, dtype, [3, 2, 4], [40, 30, 20], P=18, hq=4, hk=2, D=64)
        good = c["starts"].clone(), c["lens"].clone()
        ref = attend_reference(c)
        for starts, lens in (([0, 9, 2, 9], [58, 48, 38]), ([5, 5, 5, 5], [58, 48, 38]), ([0, 100, 3, 9], [58, 48, 38]),
                             ([-7, 3, 5, 9], [58, 48, 38]), ([0, 3, 5, 1 << 40], [58, 48, 38]),
                             ([0, 3, 5, 9], [-(1 << 50), 48, 0]), ([0, 3, 5, 9], [1 << 50, 1 << 62, 38])):
            c["starts"], c["lens"] = torch.tensor(starts), torch.tensor(lens)
            run_coded(R, c)
            R.get_device_error()
        c["starts"], c["lens"] = good
        out, _ = run_coded(R, c)
        assert_close(out, ref[0], ref[2], "after")


def test_no_tokens(rope_gpu):
    n = R.launch_count()
    k = torch.zeros(2, 1, 4, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    s = e8m0(torch.zeros(2, 1, 1)).cuda()
    R.paged_attention_8bit(torch.empty(0, 64, device="cuda"), k, k.clone(), s, s.clone(), torch.zeros(1, 1, dtype=torch.int64, device="cuda"),
                           torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"),
                           torch.empty(0, 64, device="cuda"))
    i = torch.empty(0, dtype=torch.int64, device="cuda")
    R.copy_pages(i, i.clone(), [k])
    assert R.launch_count() == n


@pytest.mark.skipif(not hasattr(torch, "_lazy_clone"), reason="this torch makes no such tensors")
def test_the_source_of_a_lazy_clone_keeps_its_values(rope_gpu):
    """Tensors that share their memory until one of them is written: what these operators write is separated first."""
    D, bs, NB = 64, 4, 6
    table = torch.cat([torch.ones(8, D // 2), torch.zeros(8, D // 2)], 1).cuda()
    x = torch.randn(3, D, device="cuda")
    caches = [torch.zeros(NB, 1, bs, D, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    caches += [e8m0(torch.zeros(NB, 1, 1)).cuda() for _ in range(2)]
    refs = torch.zeros(NB, dtype=torch.int32, device="cuda")
    blocks, lens = torch.full((1, 2), -1, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    q_out, out = torch.zeros_like(x), torch.zeros_like(x)
    sources = caches + [refs, blocks, lens, q_out, out]
    before = [t.view(torch.uint8).clone() for t in sources]
    c, r, b, n, q, o = [torch._lazy_clone(t) for t in caches], *(torch._lazy_clone(t) for t in (refs, blocks, lens, q_out, out))
    i = lambda *v: torch.tensor(v, device="cuda")  # noqa: E731
    pair = [torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2)]
    R.rearrange_sequences(blocks, lens, r, i(0), b, n, r, *pair, i(0, 0), bs, room=i(3))
    R.append_paged_kv_8bit(i(0, 1, 2), x, x, x, table, i(0, 1, 2), *c, D, query_out=q)
    R.paged_attention_8bit(q, *c, b, n, i(0, 3), o)
    R.copy_pages(i(0), i(5), c)
    assert n.tolist() == [3] and r.tolist() == [1, 0, 0, 0, 0, 0] and int(b[0, 0]) == 0
    assert torch.equal(q, x) and bool((bytes_of(c[0])[5] == bytes_of(c[0])[0]).all())
    for t, was in zip(sources, before):
        assert torch.equal(t.view(torch.uint8), was)
