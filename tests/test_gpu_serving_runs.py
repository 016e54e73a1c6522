"""The serving operators together and in the ways programs call them: table, append and attention in
sequence over several steps, captured graphs, other streams, threads, prepared calls, large caches."""
import math
import threading

import pytest
import torch

import transformer_rope_positional_gb300 as R
from parity import same_bits
from serving_ref import (E32, append_bound, append_case, append_reference, assert_close, attend_case,
                         attend_reference, check_attend, half_step, run_attend)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("neox", [True, False])
def test_steps_of_a_serving_program(rope_gpu, dtype, neox):
    """A shared prompt, a chunk for each of three sequences, then two decoding steps: tables from scaled
    frequencies, keys and values appended with the rotation, attention over the pages.  Against float64 on the
    values that the program itself holds in its type (the rotated q and k, which are rounded once)."""
    D, hq, hk, bs, P, B = 64, 4, 2, 16, 37, 3
    G = hq // hk
    g = torch.Generator().manual_seed(5)
    inv, scale = R.rope_frequencies(D, 10000.0, {"kind": "yarn", "factor": 4, "original_length": 64})
    table = torch.empty(256, D, device="cuda", dtype=torch.float32)
    R.scaled_cos_sin_cache(table, inv, scale)
    ang = torch.arange(256).double()[:, None] * inv
    cos, sin = ang.cos() * scale, ang.sin() * scale
    NB = 3 + B * 4
    pages = torch.randperm(NB, generator=g)
    prefix_blocks, own = pages[:3].cuda(), pages[3:].view(B, 4).cuda()
    kc = torch.full((NB, hk, bs, D), float("nan"), dtype=dtype, device="cuda")
    vc = kc.clone()
    held_k, held_v = [[] for _ in range(B + 1)], [[] for _ in range(B + 1)]  # rotated keys and values, float64

    def rotate(x, pos):
        x = x.double().view(x.shape[0], -1, D).clone()
        ia = torch.arange(D // 2) if neox else 2 * torch.arange(D // 2)
        ib = ia + (D // 2 if neox else 1)
        c, s = cos[pos][:, None], sin[pos][:, None]
        a, b = x[..., ia].clone(), x[..., ib].clone()
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
        return x

    def step(new, lens, blocks, shared):
        T = sum(new)
        qkv = (torch.randn(T, (hq + 2 * hk) * D, generator=g)).to(dtype)
        pos = torch.cat([torch.arange(n - a, n) for n, a in zip(lens, new)])
        slots = torch.cat([torch.tensor([int(blocks[b][(j - shared) // bs]) * bs + (j - shared) % bs
                                         for j in range(lens[b] - new[b], lens[b])], dtype=torch.int64)
                           for b in range(len(new))])
        dev = qkv.cuda()
        q, k, v = dev[:, :hq * D], dev[:, hq * D:(hq + hk) * D], dev[:, (hq + hk) * D:]
        q_out = torch.empty(T, hq * D, device="cuda", dtype=dtype)
        R.append_paged_kv(pos.cuda(), q, k, v, table, slots.cuda(), kc, vc, D, is_neox=neox, query_out=q_out)
        rq, rk = rotate(qkv[:, :hq * D], pos), rotate(qkv[:, hq * D:(hq + hk) * D], pos)
        # the table is binary32: 4 half steps on cos and sin of each of the two terms, 2 on the rotation
        terms = lambda x: scale * (x.abs() + x.roll(D // 2 if neox else 1, -1).abs() + x.roll(-1, -1).abs())  # noqa: E731
        raw_q = qkv[:, :hq * D].double().view(T, -1, D)
        assert_close(q_out.view(T, -1, D), rq, (half_step(dtype) + 4 * E32) * rq.abs() + 12 * E32 * terms(raw_q) + 1e-7,
                     "rotated query")
        got_k = kc.transpose(1, 2).reshape(-1, hk, D)[slots.cuda()].cpu()
        raw_k = qkv[:, hq * D:(hq + hk) * D].double().view(T, -1, D)
        assert_close(got_k, rk, (half_step(dtype) + 4 * E32) * rk.abs() + 12 * E32 * terms(raw_k) + 1e-7, "rotated key")
        return T, q_out, got_k.double(), qkv[:, (hq + hk) * D:].double().view(T, hk, D), slots

    # the shared prompt fills the prefix pages
    T, q_out, k, v, _ = step([P], [P], [prefix_blocks.tolist()], 0)
    prefix_k, prefix_v = k, v
    out = torch.empty(T, hq * D, device="cuda", dtype=dtype)
    R.paged_attention(q_out, kc, vc, prefix_blocks[None], torch.tensor([P], device="cuda"),
                      torch.tensor([0, P], device="cuda"), out)
    own_k, own_v = [[] for _ in range(B)], [[] for _ in range(B)]

    def check(new, q_out, out, lse):
        t = 0
        for b, n in enumerate(new):
            ks = torch.cat([prefix_k] + own_k[b])
            vs = torch.cat([prefix_v] + own_v[b])
            for i in range(n):
                seen = ks.shape[0] - n + i + 1
                q = q_out[t].cpu().double().view(hk, G, D)
                s = torch.einsum("kgd,nkd->kgn", q, ks[:seen]) * D ** -0.5
                w = torch.softmax(s, -1)
                o = torch.einsum("kgn,nkd->kgd", w, vs[:seen])
                A = torch.einsum("kgn,nkd->kgd", w, vs[:seen].abs())
                big = torch.einsum("kgd,nkd->kgn", q.abs(), ks[:seen].abs()).amax(-1) * D ** -0.5
                uw = 0.0 if dtype == torch.float32 else half_step(dtype)
                tol = half_step(dtype) * o.abs() + (uw + 4 * (D + 4) * E32 * big[..., None] + (4 * seen + 64) * E32) * A + 1e-7
                assert_close(out[t].view(hk, G, D), o, tol, "row %d" % t)
                assert abs(float(lse[t].view(hk, G)[0, 0]) - float(torch.logsumexp(s, -1)[0, 0])) < 1e-4
                t += 1

    lens = [P] * B
    for new in ([21, 1, 9], [1, 1, 1], [3, 1, 2]):
        lens = [n + a for n, a in zip(lens, new)]
        T, q_out, k, v, _ = step(new, lens, own.tolist(), P)
        t = 0
        for b, n in enumerate(new):
            own_k[b].append(k[t:t + n])
            own_v[b].append(v[t:t + n])
            t += n
        out = torch.empty(T, hq * D, device="cuda", dtype=dtype)
        lse = torch.empty(T, hq, device="cuda")
        R.paged_attention(q_out, kc, vc, own, torch.tensor(lens, device="cuda"),
                          torch.tensor([0] + new, device="cuda").cumsum(0), out, prefix_blocks=prefix_blocks,
                          prefix_len=P, lse=lse)
        check(new, q_out, out, lse)
    assert R.get_device_error() == 0


def test_fused_block_feeds_the_attention(rope_gpu):
    """The caches and queries of the fused QKV operator are what the attention reads."""
    import workloads as W
    qc = W.qkv_case("attend_after_fused", 21, [5, 1, 3], [0, 17, 40], 4, 2, 2, 128, 16, torch.bfloat16)
    kc, vc, qo = qc.k_cache.cuda(), qc.v_cache.cuda(), qc.q_out.cuda()
    R.qkv_rmsnorm_rope_cache(qc.qkv.cuda(), qc.nq, qc.nk, qc.nv, qc.q_gamma.cuda(), qc.k_gamma.cuda(), qc.eps,
                             qc.cache.cuda(), qc.seq_lens.cuda(), qc.query_start_loc.cuda(), qc.slot_mapping.cuda(),
                             qo, kc, vc)
    # this call's tokens only: their pages are those of the slots
    slots = qc.slot_mapping.tolist()
    starts = qc.query_start_loc.tolist()
    out = torch.empty_like(qo)
    for b in range(3):
        rows = list(range(starts[b], starts[b + 1]))
        if any(slots[t] < 0 for t in rows):
            continue
        n = len(rows)
        one = torch.tensor([[slots[t] // 16 for t in rows]])
        # every token on a page of its own (page size 1 over the same memory is not what the layout is): gather
        k = torch.stack([kc[slots[t] // 16, :, slots[t] % 16] for t in rows])
        v = torch.stack([vc[slots[t] // 16, :, slots[t] % 16] for t in rows])
        k1, v1 = k[:, :, None].contiguous(), v[:, :, None].contiguous()  # [n, hk, 1, D]: pages of one row
        o = torch.empty(n, 4 * 128, device="cuda", dtype=torch.bfloat16)
        R.paged_attention(qo[starts[b]:starts[b + 1]].contiguous(), k1, v1, torch.arange(n, device="cuda")[None],
                          torch.tensor([n], device="cuda"), torch.tensor([0, n], device="cuda"), o)
        q = qo[starts[b]:starts[b + 1]].double().view(n, 2, 2, 128)
        s = torch.einsum("tkgd,nkd->kgtn", q, k.double()) / math.sqrt(128)
        s = s.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -math.inf)
        ref = torch.einsum("kgtn,nkd->tkgd", torch.softmax(s, -1), v.double()).reshape(n, -1)
        A = torch.einsum("kgtn,nkd->tkgd", torch.softmax(s, -1), v.double().abs()).reshape(n, -1)
        assert_close(o, ref.cpu(), (half_step(torch.bfloat16) * (ref.abs() + A) + 1e-4 * A).cpu(), "after fused")
        assert one.numel() == n


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
def test_captured_and_replayed_with_other_lengths(rope_gpu, dtype):
    """Lengths live on the device: a captured attention replayed after they changed answers for the new ones."""
    c = attend_case(31, dtype, [1, 1, 1], [40, 200, 7], P=50, hq=4, hk=2, D=64)
    d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    out = torch.empty(3, c["width"], device="cuda", dtype=dtype)
    lse = torch.empty(3, 4, device="cuda")
    R.load()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            R.paged_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["starts"], out, scale=c["scale"],
                              prefix_blocks=d["prefix"], prefix_len=50, lse=lse)
    torch.cuda.synchronize()
    for lens in ([90, 250, 57], [51, 60, 57], [90, 130, 52]):
        c["lens"] = torch.tensor(lens)
        d["lens"].copy_(c["lens"])
        out.fill_(float("nan"))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        ro, rl, to, tl = attend_reference(c)
        assert_close(out, ro, to, "replayed out")
        assert_close(lse, rl, tl, "replayed lse")
    assert R.get_device_error() == 0


def test_append_and_table_in_a_graph(rope_gpu):
    c = append_case(32, torch.bfloat16, 20, 4, 2, 64, 64, 16)
    d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    qo = torch.empty(20, 256, device="cuda", dtype=torch.bfloat16)
    tab = torch.empty(97, 64, device="cuda", dtype=torch.bfloat16)
    R.load()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            R.scaled_cos_sin_cache(tab, *R.rope_frequencies(64))
            R.append_paged_kv(d["pos"], d["q"], d["k"], d["v"], tab, d["slots"], d["kc"], d["vc"], 64, query_out=qo)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    c["table"] = tab.cpu()
    rq, rk, rv, _ = append_reference(c)
    assert_close(qo, rq, append_bound(rq, torch.bfloat16), "query")
    assert_close(d["kc"], rk, append_bound(rk, torch.bfloat16), "k_cache")
    assert same_bits(d["vc"], rv.to(torch.bfloat16))


def test_two_graphs_with_one_workspace(rope_gpu):
    """Captured calls that are given the same workspace, replayed one after the other on one stream."""
    cs = [attend_case(33 + i, torch.bfloat16, [1, 2], own, P=P, hq=8, hk=2, D=128)
          for i, (own, P) in enumerate((([600, 90], 0), ([30, 40], 900)))]
    need = 0
    for c in cs:
        q = c["q"].cuda()
        need = max(need, R.paged_attention_workspace(q, c["k"].cuda(), c["P"]))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0xff)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    runs = []
    for c in cs:
        d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
        out = torch.empty(3, c["width"], device="cuda", dtype=torch.bfloat16)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                R.paged_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["starts"], out, scale=c["scale"],
                                  prefix_blocks=d["prefix"] if c["P"] else None, prefix_len=c["P"], workspace=ws)
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
    c = attend_case(35, dtype, [1, 3, 1], [700, 20, 3], P=300, hq=4, hk=2, D=64)
    q, k = c["q"].cuda(), c["k"].cuda()
    n = R.paged_attention_workspace(q, k, 300)
    for fill in (0x00, 0xff, 0x7f):
        ws = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")[:n]
        check_attend(R, c, "workspace", workspace=ws)
    with pytest.raises(R.RopeError):
        run_attend(R, c, workspace=torch.empty(n - 256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        run_attend(R, c, workspace=torch.empty(n, dtype=torch.uint8))


def test_streams_prepared_calls_and_threads(rope_gpu):
    """Calls on streams other than the current one (object and handle), prepared calls issued again, and calls
    from several threads at once."""
    c = attend_case(36, torch.bfloat16, [1, 2, 9], [300, 5, 60], P=130, hq=8, hk=2, D=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = run_attend(R, c, stream=s)
    ref = attend_reference(c)
    assert_close(out, ref[0], ref[2], "stream")
    out, _ = run_attend(R, c, stream=s.cuda_stream)
    assert_close(out, ref[0], ref[2], "stream handle")
    out, _ = run_attend(R, c, prepared=True)
    assert_close(out, ref[0], ref[2], "prepared")
    errors = []

    def work(i):
        try:
            mine = torch.cuda.Stream()
            with torch.cuda.stream(mine):
                d = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
                for _ in range(20):
                    o = torch.full((c["T"], c["width"]), float("nan"), device="cuda", dtype=torch.bfloat16)
                    R.paged_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["starts"], o, scale=c["scale"],
                                      prefix_blocks=d["prefix"], prefix_len=130)
                    mine.synchronize()
                    assert_close(o, ref[0], ref[2], "thread %d" % i)
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
    check_attend(R, attend_case(37, dtype, new, own, P=0, hq=2, hk=1, D=32, bs=8), "many")


def test_many_sequences_of_several_tokens(rope_gpu):
    new = [1 + (i * 3) % 20 for i in range(70)]
    own = [new[i] + (i * 11) % 50 for i in range(70)]
    check_attend(R, attend_case(38, torch.float16, new, own, P=20, hq=8, hk=2, D=64), "many chunks")


def test_cache_past_32_bit_offsets(rope_gpu):
    """Pages whose elements lie past 2^31 and 2^32."""
    D, hk, bs = 128, 8, 64
    NB = (1 << 32) // (hk * bs * D) + 40
    free = torch.cuda.mem_get_info()[0]
    if free < 3 * NB * hk * bs * D * 2:
        pytest.skip("needs 26 GB")
    small = attend_case(39, torch.bfloat16, [1, 30], [150, 64], P=64, hq=16, hk=hk, D=D, bs=bs, fill=0.0)
    pages = torch.tensor([NB - 1 - 3 * i for i in range(small["k"].shape[0])])
    big_k = torch.empty(NB, hk, bs, D, dtype=torch.bfloat16, device="cuda")
    big_v = torch.empty_like(big_k)
    big_k[pages.cuda()] = small["k"].cuda()
    big_v[pages.cuda()] = small["v"].cuda()
    table = torch.where(small["table"] < small["k"].shape[0], pages[small["table"].clamp(max=len(pages) - 1)], small["table"])
    out = torch.empty(31, 16 * D, device="cuda", dtype=torch.bfloat16)
    R.paged_attention(small["q"].cuda(), big_k, big_v, table.cuda(), small["lens"].cuda(), small["starts"].cuda(), out,
                      scale=small["scale"], prefix_blocks=pages[small["prefix"]].cuda(), prefix_len=64)
    ref = attend_reference(small)
    assert_close(out, ref[0], ref[2], "large cache")
    # and the append to the last pages
    c = append_case(40, torch.bfloat16, 5, 8, hk, D, D, bs, NB=2)
    big_k[-2:] = c["kc"].cuda()
    big_v[-2:] = c["vc"].cuda()
    qo = torch.empty(5, 8 * D, device="cuda", dtype=torch.bfloat16)
    slots = torch.where(c["slots"] >= 0, c["slots"] + (NB - 2) * bs, c["slots"])
    R.append_paged_kv(c["pos"].cuda(), c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), c["table"].cuda(), slots.cuda(), big_k,
                      big_v, D, query_out=qo)
    rq, rk, rv, _ = append_reference(c)
    assert_close(big_k[-2:], rk, append_bound(rk, torch.bfloat16), "append past 2^32")
    assert same_bits(big_v[-2:], rv.to(torch.bfloat16))
    assert R.get_device_error() == 0


def test_unordered_starts_stay_inside_the_tensors(rope_gpu):
    """Values of query_start_loc and seq_lens that mean nothing: unspecified rows, but no access outside a tensor
    (the guard bands hold, and the bounds-checking build reports nothing), and later calls are not disturbed."""
    for dtype in (torch.float32, torch.bfloat16):
        c = attend_case(41, dtype, [3, 2, 4], [40, 30, 20], P=18, hq=4, hk=2, D=64)
        good = c["starts"].clone(), c["lens"].clone()
        for starts, lens in (([0, 9, 2, 9], [58, 48, 38]), ([5, 5, 5, 5], [58, 48, 38]), ([0, 100, 3, 9], [58, 48, 38]),
                             ([-7, 3, 5, 9], [58, 48, 38]), ([0, 3, 5, 1 << 40], [58, 48, 38]),
                             ([0, 3, 5, 9], [-(1 << 50), 48, 0]), ([0, 3, 5, 9], [1 << 50, 1 << 62, 38])):
            c["starts"], c["lens"] = torch.tensor(starts), torch.tensor(lens)
            run_attend(R, c)
            R.get_device_error()
        c["starts"], c["lens"] = good
        check_attend(R, c, "after")


def test_no_tokens(rope_gpu):
    n = R.launch_count()
    k = torch.zeros(2, 1, 4, 64, device="cuda")
    R.paged_attention(torch.empty(0, 64, device="cuda"), k, k.clone(), torch.zeros(1, 1, dtype=torch.int64, device="cuda"),
                      torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"),
                      torch.empty(0, 64, device="cuda"))
    e = torch.empty(0, 64, device="cuda")
    i = torch.empty(0, dtype=torch.int64, device="cuda")
    R.append_paged_kv(i, e, e, e, torch.zeros(1, 64, device="cuda"), i, k, k.clone(), 64, query_out=e.clone())
    assert R.launch_count() == n
