"""Cases of the operators of a paged cache that is held in 8 bits: written, read, and its pages managed.

Four kinds of case, in the order in which a serving program meets them:

* ``append``: queries and keys rotated, keys and values quantised on the way to their cache slots;
* ``attend``: attention of a batch's new tokens over the 8-bit cache;
* ``fork``: sequences forked, reordered and dropped, given pages for what comes, and the pages that they
  must not share copied in every layer's cache;
* ``compact``: the live pages moved to the front of the cache.

A cache holds codes (float8_e4m3fn) [blocks, heads, block size, head size] and a power of two
(float8_e8m0fnu) for each block of tokens of a page and head, [blocks, heads, scale blocks]: a cached value is
code * scale.  ``run`` computes all of it with elementary torch operations in 32 bits where ``own`` is false,
and with this package's operators where it is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _append(name, dtype, seqs, new, held, hq, hk, head, rotary, neox, block, scales, table="same", fused=True):
    """``seqs`` sequences that get 1..``new`` tokens each (all ``new`` where it is given negative) after up to
    ``held`` earlier ones; ``scales`` blocks of tokens a page."""
    return {"name": name, "kind": "append", "dtype": dtype, "seqs": seqs, "new": new, "held": held, "hq": hq, "hk": hk,
            "head": head, "rotary": rotary, "neox": neox, "block": block, "scales": scales, "table": table,
            "fused": fused}


def _attend(name, dtype, seqs, new, prefix, own_max, hq, hk, head, block, scales):
    """``seqs`` sequences with 1..``new`` new tokens each (all ``new`` where it is given negative), on top of up to
    ``own_max`` tokens of their own (new ones included) after ``prefix`` shared ones."""
    return {"name": name, "kind": "attend", "dtype": dtype, "seqs": seqs, "new": new, "prefix": prefix,
            "own_max": own_max, "hq": hq, "hk": hk, "head": head, "block": block, "scales": scales}


def _fork(name, seqs, own_max, beams, grow, layers, hk, head, block, scales, spare):
    """``seqs`` sequences of up to ``own_max`` tokens.  ``beams`` > 0: each is forked into so many.  < 0: groups of
    so many are reordered, some dropped and some doubled.  All get room for ``grow`` tokens.  ``spare`` free pages."""
    return {"name": name, "kind": "fork", "seqs": seqs, "own_max": own_max, "beams": beams, "grow": grow,
            "layers": layers, "hk": hk, "head": head, "block": block, "scales": scales, "spare": spare}


def _compact(name, seqs, own_max, prefix, holes, layers, hk, head, block, scales):
    """A cache whose pages are to ``holes`` percent free, between those of ``seqs`` sequences of up to ``own_max``
    tokens and a prefix of ``prefix``."""
    return {"name": name, "kind": "compact", "seqs": seqs, "own_max": own_max, "prefix": prefix, "holes": holes,
            "layers": layers, "hk": hk, "head": head, "block": block, "scales": scales}


def listed():
    return [
        # one decoding step of 64 requests, a scale a page and head that has to grow at times: latency
        _append("append8_bf16_64req_decode_32q8k_h128", "bf16", 64, -1, 4096, 32, 8, 128, 128, True, 16, 1),
        # prompt chunks of 4 requests, q, k and v being column ranges of one projection, table in 32 bits
        _append("append8_bf16_4x4096tok_32q8k_h128", "bf16", 4, -4096, 1000, 32, 8, 128, 128, True, 16, 1, table="f32"),
        # ragged pieces, interleaved layout on the first 64 of 256 columns, four scales a page of 64
        _append("append8_f16_40req_ragged_16q16k_h256_r64", "f16", 40, 300, 500, 16, 16, 256, 64, False, 64, 4),
        # one decoding step of 4 short requests: latency
        _attend("attend8_bf16_4seq_decode_300", "bf16", 4, -1, 0, 300, 32, 8, 128, 16, 1),
        # one decoding step of 64 requests of up to 8192 tokens, nothing shared: bound by the cache's bytes
        _attend("attend8_bf16_64seq_decode_8192", "bf16", 64, -1, 0, 8192, 32, 8, 128, 16, 1),
        # prompt chunks of 1984 tokens behind a shared prompt of 4096: bound by the matrix units
        _attend("attend8_bf16_4seq_chunks_p4096", "bf16", 4, -1984, 4096, 1984, 32, 8, 128, 32, 2),
        # up to 5 drafted tokens a request to be verified, heads of 256, pages that are no power of two
        _attend("attend8_f16_32seq_draft5_p2048_h256", "f16", 32, 5, 2048, 517, 16, 16, 256, 12, 3),
        # 32 bits, ragged in everything, a scale a token
        _attend("attend8_f32_6seq_ragged_p101_h64", "f32", 6, 40, 101, 333, 4, 2, 64, 17, 17),
        # one step of beam search: 16 beams reordered, some dropped and some doubled, in one layer's cache: latency
        _fork("fork_16seq_beams4_300", 16, 300, -4, 1, 1, 8, 128, 16, 1, 64),
        # 64 prompts of up to 1000 tokens, four samples of each to come, 8 layers
        _fork("fork_64seq_samples4_8layers", 64, 1000, 4, 16, 8, 8, 128, 16, 1, 1024),
        # a few short sequences: latency
        _compact("compact_4seq_300", 4, 300, 0, 40, 1, 8, 128, 16, 1),
        # a cache of 8 layers, 35 of 100 pages free, before it is made smaller
        _compact("compact_100seq_8layers", 100, 1600, 2048, 35, 8, 8, 128, 16, 1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One case of the listed ones' ranges."""
    kind = rng.choice(["append", "attend", "attend", "attend", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    block = rng.choice([1, 12, 16, 16, 17, 32, 64, 128])
    scales = rng.choice([s for s in range(1, block + 1) if block % s == 0])
    if kind == "append":
        while True:
            hk = rng.choice([1, 2, 3, 4, 8])
            head = 32 * rng.randint(2, 8)
            rotary = min(head, 32 * rng.randint(1, 8))
            c = _append("", dtype, _log(rng, 1, 128), rng.choice([-1, 8, -_log(rng, 2, 4096), _log(rng, 2, 4096)]),
                        _log(rng, 1, 4096), hk * rng.choice([1, 2, 4, 5, 7]), hk, head, rotary, rng.random() < 0.7, block,
                        scales, rng.choice(["same", "f32"]), rng.random() < 0.5)
            if c["seqs"] * abs(c["new"]) <= 16384 and work(c)["bytes"] < work(listed()[1])["bytes"]:
                break
    elif kind == "attend":
        most = work(listed()[5])["flops"]
        while True:
            hk = rng.choice([1, 2, 4, 8])
            head = rng.choice([64, 64, 96, 128, 128, 128, 160, 256])
            new = rng.choice([-1, -1, 8, -_log(rng, 2, 64), _log(rng, 2, 2048)])
            c = _attend("", dtype, _log(rng, 1, 128), new, rng.choice([0, _log(rng, 1, 16384)]),
                        abs(new) + _log(rng, 1, 4096), hk * rng.choice([1, 2, 4, 5, 8]), hk, head, block, scales)
            # no more than the largest listed one costs either side; the plain form's scores stay a few GB
            scores = c["seqs"] * abs(new) * c["hq"] * (c["prefix"] + c["own_max"])
            pages = c["seqs"] * c["own_max"] * hk * head
            if work(c)["flops"] < most / (8 if dtype == "f32" else 1) and scores < 1.5e9 and pages < 3e8:
                break
    else:
        while True:
            hk, head, layers = rng.choice([1, 2, 4, 8]), rng.choice([64, 96, 128, 256]), rng.randint(1, 8)
            if kind == "fork":
                c = _fork("", _log(rng, 1, 128), _log(rng, 1, 2048), rng.choice([-4, -3, 1, 2, 4]), _log(rng, 1, 64), layers,
                          hk, head, block, scales, 0)
                # pages enough for what all rows of the new batch may need, or few of them to spare
                c["spare"] = c["seqs"] * max(1, c["beams"]) * (2 + -(-c["grow"] // block)) + rng.choice([0, _log(rng, 1, 1000)])
                pages = c["spare"] + c["seqs"] * (1 + c["own_max"] // block)
            else:
                c = _compact("", _log(rng, 1, 128), _log(rng, 1, 2048), rng.choice([0, _log(rng, 1, 4096)]),
                             rng.randint(3, 70), layers, hk, head, block, scales)
                pages = (c["prefix"] // block + 1 + c["seqs"] * (1 + c["own_max"] // block)) * 100 / (100 - c["holes"])
            if pages * block * hk * head * layers < 1.5e9:
                break
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _spread(n):
    return [((i * 7919 + 3) % 9973) / 9973.0 for i in range(n)]


def _lengths(case):
    """(new tokens, own tokens) of every sequence: ragged over the whole range, the same for every seed."""
    n, new = case["seqs"], case["new"]
    q = [-new if new < 0 else 1 + int(s * new) for s in _spread(n)]
    own_len = [max(a, int(round(case["own_max"] * (1.0 - 0.97 * ((i * 0.6180339887) % 1.0))))) for i, a in enumerate(q)]
    return q, own_len


def _appended(case):
    """(new tokens, earlier tokens) of every sequence."""
    q = [-case["new"] if case["new"] < 0 else 1 + int(s * case["new"]) for s in _spread(case["seqs"])]
    return q, [int(case["held"] * ((i * 0.6180339887) % 1.0)) for i in range(case["seqs"])]


def _held(case):
    """Tokens of every sequence."""
    return [max(1, int(round(case["own_max"] * (1.0 - 0.9 * ((i * 0.6180339887) % 1.0))))) for i in range(case["seqs"])]


def _codes(g, dev, *shape):
    """Codes of values that were quantised: the largest of a block reaches a few hundred."""
    return torch.empty(shape, dtype=torch.float16, device=dev).normal_(0.0, 80.0, generator=g).clamp_(-448, 448).to(E4M3)


def _scales(g, dev, *shape):
    """2^-9 to 2^-6: values of about one half to four."""
    return torch.randint(118, 122, shape, generator=g, device=dev, dtype=torch.uint8).view(E8M0)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    if case["kind"] == "append":
        return _prepare_append(case, s, g, dev)
    if case["kind"] == "attend":
        return _prepare_attend(case, s, g, dev, seed)
    return _prepare_pages(case, s, g, dev, seed)


def _prepare_append(case, s, g, dev):
    dt = DTYPES[case["dtype"]]
    hq, hk, D, R, bs, S = (case[k] for k in ("hq", "hk", "head", "rotary", "block", "scales"))
    new, held = _appended(case)
    T, per = sum(new), bs // S

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    if case["fused"]:
        qkv = normal(T, (hq + 2 * hk) * D)
        s["q"], s["k"], s["v"] = qkv[:, :hq * D], qkv[:, hq * D:(hq + hk) * D], qkv[:, (hq + hk) * D:]
    else:
        s["q"], s["k"], s["v"] = normal(T, hq * D), normal(T, hk * D), normal(T, hk * D)
    length = max(a + b for a, b in zip(new, held))
    angle = torch.arange(length, device=dev, dtype=torch.float64)[:, None] * torch.pow(
        torch.tensor(10000.0, device=dev, dtype=torch.float64),
        -torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32 if case["table"] == "f32" else dt)
    # every sequence's pages, somewhere in the cache; a program makes up the slots, and so knows which scale blocks
    # a step touches, from which token on, and in which of them each token falls
    start = torch.tensor(held)
    count = torch.tensor(new)
    seq = torch.repeat_interleave(torch.arange(len(new)), count)
    first = torch.cumsum(count, 0) - count
    position = start[seq] + torch.arange(T) - first[seq]
    need = (start + count + bs - 1) // bs
    blocks = int(need.sum()) + 3
    base = torch.cumsum(need, 0) - need
    order = torch.randperm(blocks, generator=g, device=dev).cpu()
    slots = order[base[seq] + position // bs] * bs + position % bs
    touched, of = torch.unique(slots // per, return_inverse=True)
    s["positions"], s["slots"] = position.to(dev), slots.to(dev)
    s["touched"], s["of"] = touched.to(dev), of.to(dev)
    s["kept"] = torch.full((len(touched),), per).scatter_reduce_(0, of, slots % per, "amin").to(dev)
    s["k_cache"], s["v_cache"] = _codes(g, dev, blocks, hk, bs, D), _codes(g, dev, blocks, hk, bs, D)
    s["k_scale"], s["v_scale"] = _scales(g, dev, blocks, hk, S), _scales(g, dev, blocks, hk, S)
    s["q_out"] = torch.empty(T, hq * D, device=dev, dtype=dt)
    return s


def _prepare_attend(case, s, g, dev, seed):
    dt = DTYPES[case["dtype"]]
    hq, hk, D, bs, S, P = (case[k] for k in ("hq", "hk", "head", "block", "scales", "prefix"))
    q, own_len = _lengths(case)
    order = torch.randperm(len(q), generator=torch.Generator().manual_seed(seed)).tolist()  # the seed shuffles the sequences
    q, own_len = [q[i] for i in order], [own_len[i] for i in order]
    T = sum(q)
    s["new_max"], s["own_max"] = max(q), max(own_len)  # a program knows these when it makes up the batch
    s["q"] = torch.randn(T, hq * D, generator=g, device=dev, dtype=torch.float32).to(dt)
    s["seq_lens"] = torch.tensor([P + n for n in own_len], dtype=torch.int64, device=dev)
    s["starts"] = torch.tensor([0] + q, dtype=torch.int64).cumsum(0).to(dev)
    held = [-(-n // bs) for n in own_len]
    shared = -(-P // bs)
    blocks = sum(held) + shared + 2
    pages = torch.randperm(blocks, generator=g, device=dev)
    s["prefix_blocks"] = pages[:shared].contiguous() if P else None
    width = max(held)
    col = torch.arange(width, device=dev)
    first = torch.tensor([0] + held[:-1], dtype=torch.int64).cumsum(0).to(dev)
    at = shared + first[:, None] + col
    s["block_table"] = torch.where(col < torch.tensor(held, device=dev)[:, None], pages[at.clamp(max=blocks - 1)], 0)
    s["k_cache"], s["v_cache"] = _codes(g, dev, blocks, hk, bs, D), _codes(g, dev, blocks, hk, bs, D)
    s["k_scale"], s["v_scale"] = _scales(g, dev, blocks, hk, S), _scales(g, dev, blocks, hk, S)
    s["out"] = torch.empty(T, hq * D, device=dev, dtype=dt)
    s["lse"] = torch.empty(T, hq, device=dev, dtype=torch.float32)
    return s


def _prepare_pages(case, s, g, dev, seed):
    hk, D, bs, S = (case[k] for k in ("hk", "head", "block", "scales"))
    c = torch.Generator().manual_seed(seed)
    length = torch.tensor(_held(case))[torch.randperm(case["seqs"], generator=c)]
    B, P = case["seqs"], case.get("prefix", 0)
    need = (length + bs - 1) // bs
    shared = -(-P // bs)
    live = shared + int(need.sum())
    if case["kind"] == "fork":
        blocks = live + case["spare"]
    else:
        blocks = max(live, int(round(live * 100 / (100 - case["holes"]))))
    pages = torch.randperm(blocks, generator=c)
    room = case["grow"] if case["kind"] == "fork" else 0
    width = int((length.max() + room + bs - 1) // bs)
    col = torch.arange(width)
    base = shared + torch.cumsum(need, 0) - need
    table = torch.where(col < need[:, None], pages[(base[:, None] + col).clamp(max=blocks - 1)], 0)
    # every fourth sequence came of the one before it: it shares the whole pages that both have
    for b in range(3, B, 4):
        n = int(min(length[b] // bs, length[b - 1] // bs) // 2)
        table[b, :n] = table[b - 1, :n]
    refs = torch.zeros(blocks, dtype=torch.int32)
    refs.index_add_(0, table[col < need[:, None]], torch.ones(int(need.sum()), dtype=torch.int32))
    refs[pages[:shared]] += 1
    s["prefix_blocks"] = pages[:shared].to(dev) if P else None
    s["block_table"], s["seq_lens"], s["refs"] = table.to(dev), (P + length).to(dev), refs.to(dev)
    s["caches"] = []
    for _ in range(case["layers"]):
        s["caches"] += [torch.randint(0, 0x7f, (blocks, hk, bs, D), generator=g, device=dev, dtype=torch.uint8).view(E4M3)
                        for _ in range(2)]
        s["caches"] += [_scales(g, dev, blocks, hk, S) for _ in range(2)]
    s["new_refs"] = torch.zeros(blocks, dtype=torch.int32, device=dev)
    s["counts"] = torch.zeros(2, dtype=torch.int64, device=dev)
    if case["kind"] == "compact":
        s["new_table"] = torch.zeros(B, width, dtype=torch.int64, device=dev)
        s["new_prefix"] = torch.zeros(shared, dtype=torch.int64, device=dev) if P else None
        most = blocks // 2
    else:
        n = case["beams"]
        if n > 0:
            parents = torch.repeat_interleave(torch.arange(B), n)
        else:  # beams of a group of -n follow any of its sequences; at times one is given up
            group = torch.arange(B) // -n * -n
            parents = (group + torch.randint(0, -n, (B,), generator=c)).clamp(max=B - 1)
            parents[torch.rand(B, generator=c) < 0.05] = -1
        s["parents"] = parents.to(dev)
        most = len(parents)
        s["room"] = torch.where(parents >= 0, case["grow"], 0).to(dev)
        s["new_table"] = torch.zeros(most, width, dtype=torch.int64, device=dev)
        s["new_lens"] = torch.zeros(most, dtype=torch.int64, device=dev)
    s["src"], s["dst"] = (torch.full((most,), -1, dtype=torch.int64, device=dev) for _ in range(2))
    return s


# ---------------------------------------------------------------------------
# The calls, and the plain forms
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        import transformer_rope_positional_gb300 as R

        if case["kind"] == "append":
            R.append_paged_kv_8bit(s["positions"], s["q"], s["k"], s["v"], s["table"], s["slots"], s["k_cache"],
                                   s["v_cache"], s["k_scale"], s["v_scale"], case["head"], is_neox=case["neox"],
                                   query_out=s["q_out"])
            return s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        if case["kind"] == "attend":
            R.paged_attention_8bit(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                                   s["seq_lens"], s["starts"], s["out"], scale=case["head"] ** -0.5,
                                   prefix_blocks=s["prefix_blocks"], prefix_len=case["prefix"], lse=s["lse"])
            return s["out"], s["lse"]
        if case["kind"] == "fork":
            R.rearrange_sequences(s["block_table"], s["seq_lens"], s["refs"], s["parents"], s["new_table"], s["new_lens"],
                                  s["new_refs"], s["src"], s["dst"], s["counts"], case["block"], room=s["room"])
            R.copy_pages(s["src"], s["dst"], s["caches"], count=s["counts"])
            return (s["new_table"], s["new_lens"], s["new_refs"], s["src"], s["dst"], s["counts"], s["caches"])
        R.compact_pages(s["block_table"], s["seq_lens"], s["refs"], s["new_table"], s["new_refs"], s["src"], s["dst"],
                        s["counts"], case["block"], prefix_blocks=s["prefix_blocks"], new_prefix_blocks=s["new_prefix"],
                        prefix_len=case["prefix"])
        R.copy_pages(s["src"], s["dst"], s["caches"], count=s["counts"])
        return (s["new_table"], s["new_prefix"], s["new_refs"], s["src"], s["dst"], s["counts"], s["caches"])
    return {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact}[case["kind"]](s)


def _exponent(most):
    """The smallest e with most <= 448 * 2^e, as the byte of 2^e; 0 for a block of zeros."""
    fraction, e = torch.frexp(most)  # most = fraction * 2^e, fraction in [1/2, 1)
    return torch.where(most > 0, (e - 9 + (fraction > 0.875).int() + 127).clamp(1, 254), 0)


def _plain_append(s):
    case = s["case"]
    hk, D, R, bs, S = (case[k] for k in ("hk", "head", "rotary", "block", "scales"))
    per = bs // S
    row = s["table"][s["positions"]].float()
    cos, sin = row[:, None, :R // 2], row[:, None, R // 2:]

    def rotate(x):
        x = x.float().reshape(x.shape[0], -1, D)
        a, b = (x[..., :R // 2], x[..., R // 2:R]) if case["neox"] else (x[..., 0:R:2], x[..., 1:R:2])
        first, second = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat([first, second], -1) if case["neox"] else torch.stack([first, second], -1).flatten(-2)
        return torch.cat([turned, x[..., R:]], -1)

    page, block = s["touched"] // S, s["touched"] % S
    kept = torch.arange(per, device=row.device)[:, None] < s["kept"][:, None, None, None]  # [n, 1, per, 1]

    def write(x, cache, scale):
        byte = scale.view(torch.uint8)
        old = byte[page, :, block].int()  # [n, hk]
        most = torch.zeros(old.shape, device=row.device).index_reduce_(0, s["of"], x.abs().amax(-1), "amax")
        e = torch.where(s["kept"][:, None] > 0, torch.maximum(old, _exponent(most)), _exponent(most))
        rows = block[:, None] * per + torch.arange(per, device=row.device)
        codes = cache.view(torch.uint8)[page[:, None], :, rows].view(E4M3).float().transpose(1, 2)  # [n, hk, per, D]
        codes = torch.where(kept, torch.ldexp(codes, (old - e)[..., None, None]), codes).to(E4M3).transpose(1, 2)
        cache.view(torch.uint8)[page[:, None], :, rows] = codes.contiguous().view(torch.uint8)
        byte[page, :, block] = e.to(torch.uint8)
        new = torch.ldexp(x, 127 - e[s["of"]][..., None]).to(E4M3)
        cache.view(torch.uint8)[s["slots"] // bs, :, s["slots"] % bs] = new.view(torch.uint8)

    write(rotate(s["k"]), s["k_cache"], s["k_scale"])
    write(s["v"].float().reshape(-1, hk, D), s["v_cache"], s["v_scale"])
    q = rotate(s["q"]).to(DTYPES[case["dtype"]])
    return q.reshape(q.shape[0], -1), s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _plain_attend(s):
    """The whole batch at once, padded to its longest sequence."""
    case, dev = s["case"], s["q"].device
    hq, hk, D, bs, S, P = (case[k] for k in ("hq", "hk", "head", "block", "scales", "prefix"))
    G, B, n, own_max = hq // hk, case["seqs"], s["new_max"], s["own_max"]
    new = s["starts"][1:] - s["starts"][:-1]
    token = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(s["starts"], token, right=True) - 1
    there = seq, token - s["starts"][seq]  # the place of every token in the padded batch
    q = torch.zeros(B, n, hk, G, D, device=dev)
    q[there] = s["q"].float().reshape(-1, hk, G, D) * D ** -0.5
    position = s["seq_lens"][:, None] - new[:, None] + torch.arange(n, device=dev)  # [B, n]

    def values(cache, scale, pages):  # [..., hk, bs, D]
        x = cache.view(torch.uint8)[pages].view(E4M3).float()
        f = scale.view(torch.uint8)[pages].view(E8M0).float()
        return x * f.repeat_interleave(bs // S, -1)[..., None]

    pages = s["block_table"][:, :-(-own_max // bs)]

    def own_part(cache, scale):  # [B, hk, own_max, D]
        return values(cache, scale, pages).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, D)[:, :, :own_max]

    def prefix_part(cache, scale):  # [hk, P, D]
        return values(cache, scale, s["prefix_blocks"]).permute(1, 0, 2, 3).reshape(hk, -1, D)[:, :P]

    qo = q.permute(0, 2, 1, 3, 4).reshape(B, hk, n * G, D)
    so = torch.matmul(qo, own_part(s["k_cache"], s["k_scale"]).transpose(-1, -2)).reshape(B, hk, n, G, own_max)
    seen = (P + torch.arange(own_max, device=dev)) <= position[..., None]  # [B, n, own_max]
    so = so.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = so.amax(-1)  # [B, hk, n, G]
    if P:
        qp = q.permute(2, 0, 1, 3, 4).reshape(hk, B * n * G, D)
        sp = torch.matmul(qp, prefix_part(s["k_cache"], s["k_scale"]).transpose(-1, -2)).reshape(hk, B, n, G, P)
        top = torch.maximum(top, sp.amax(-1).permute(1, 0, 2, 3))
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    so = torch.exp(so - top[..., None])
    total = so.sum(-1)
    o = torch.matmul(so.reshape(B, hk, n * G, own_max), own_part(s["v_cache"], s["v_scale"])).reshape(B, hk, n, G, D)
    if P:
        sp = torch.exp(sp - top.permute(1, 0, 2, 3)[..., None])
        total = total + sp.sum(-1).permute(1, 0, 2, 3)
        op = torch.matmul(sp.reshape(hk, B * n * G, P), prefix_part(s["v_cache"], s["v_scale"]))
        o = o + op.reshape(hk, B, n, G, D).permute(1, 0, 2, 3, 4)
    o = (o / total[..., None]).permute(0, 2, 1, 3, 4)[there]
    lse = (total.log() + top).permute(0, 2, 1, 3)[there]
    return o.reshape(-1, hq * D).to(DTYPES[case["dtype"]]), lse.reshape(-1, hq)


def _copy(s, src, dst):
    """The first pages that are named, in every cache."""
    at = torch.nonzero(src >= 0)[:, 0]
    for c in s["caches"]:
        raw = c.view(torch.uint8)
        raw[dst[at]] = raw[src[at]]


def _plain_fork(s):
    case = s["case"]
    bs, table, dev = case["block"], s["block_table"], s["block_table"].device
    B, W = table.shape
    blocks, rows = len(s["refs"]), len(s["parents"])
    col = torch.arange(W, device=dev)
    held = col < ((s["seq_lens"] + bs - 1) // bs)[:, None]
    # all old sequences let go of their pages ...
    refs = s["refs"].clone()
    refs.index_add_(0, table.flatten(), -held.flatten().int())
    # ... and the new ones take the whole pages of their parents; a page that is written on is the first child's
    is_row = s["parents"] >= 0
    p = s["parents"].clamp(min=0)
    old = torch.where(is_row, s["seq_lens"][p], 0)
    full, rest = old // bs, old % bs
    row = torch.arange(rows, device=dev)
    first = torch.full((B + 1,), rows, device=dev).scatter_reduce_(0, torch.where(is_row, p, B), row, "amin")[p] == row
    entry = table[p]
    last = entry.gather(1, full.clamp(max=W - 1)[:, None])[:, 0]
    keeps = (rest > 0) & first & (refs[last] == 0)
    copies = (rest > 0) & ~keeps
    taken = (col < full[:, None]) | ((col == full[:, None]) & keeps[:, None])
    refs.index_add_(0, entry.flatten(), taken.flatten().int())
    # free pages, lowest first, row after row
    new_lens = old + s["room"]
    have = full + keeps
    need = (new_lens + bs - 1) // bs - have
    start = torch.cumsum(need, 0) - need
    free = refs == 0
    rank = torch.cumsum(free, 0) - 1
    by_rank = torch.full((blocks + 1,), -1, device=dev).scatter_(
        0, torch.where(free, rank, blocks), torch.arange(blocks, device=dev))
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    s["new_table"].copy_(torch.where(taken, entry, torch.where(
        fresh, by_rank[(start[:, None] + col - have[:, None]).clamp(0, blocks)], s["new_table"])))
    s["new_refs"].copy_(torch.where(free & (rank < need.sum()), 1, refs))
    s["new_lens"].copy_(new_lens)
    pair = torch.where(copies, torch.cumsum(copies, 0) - 1, rows)
    src, dst = (torch.full((rows + 1,), -1, device=dev) for _ in range(2))
    src[pair], dst[pair] = last, by_rank[start.clamp(max=blocks)]
    s["src"].copy_(src[:-1].where(row < copies.sum(), -1))
    s["dst"].copy_(dst[:-1].where(row < copies.sum(), -1))
    s["counts"].copy_(torch.stack([copies.sum(), free.sum() - need.sum()]))
    _copy(s, s["src"], s["dst"])
    return (s["new_table"], s["new_lens"], s["new_refs"], s["src"], s["dst"], s["counts"], s["caches"])


def _plain_compact(s):
    case = s["case"]
    bs, P, table, dev = case["block"], case["prefix"], s["block_table"], s["block_table"].device
    blocks = len(s["refs"])
    page = torch.arange(blocks, device=dev)
    live = s["refs"] > 0
    count = live.sum()
    hole, mover = ~live & (page < count), live & (page >= count)
    by_rank = torch.full((blocks + 1,), -1, device=dev).scatter_(
        0, torch.where(hole, torch.cumsum(hole, 0) - 1, blocks), page)
    rank = torch.cumsum(mover, 0) - 1
    to = torch.where(mover, by_rank[rank.clamp(min=0)], page)
    s["new_refs"].zero_().index_add_(0, to, torch.where(live, s["refs"], 0))
    held = torch.arange(table.shape[1], device=dev) < ((s["seq_lens"] - P + bs - 1) // bs)[:, None]
    s["new_table"].copy_(torch.where(held, to[table], s["new_table"]))
    if P:
        s["new_prefix"].copy_(to[s["prefix_blocks"]])
    src = torch.full((blocks + 1,), -1, device=dev).scatter_(0, torch.where(mover, rank, blocks), page)
    most, moved = len(s["src"]), mover.sum()
    s["src"].copy_(src[:most].where(page[:most] < moved, -1))
    s["dst"].copy_(by_rank[:most].where(page[:most] < moved, -1))
    s["counts"].copy_(torch.stack([moved, count]))
    _copy(s, s["src"], s["dst"])
    return (s["new_table"], s["new_prefix"], s["new_refs"], s["src"], s["dst"], s["counts"], s["caches"])


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["kind"] == "append":
        e, te = SIZE[case["dtype"]], 4 if case["table"] == "f32" else SIZE[case["dtype"]]
        new, held = _appended(case)
        T, D, R, hq, hk = sum(new), case["head"], case["rotary"], case["hq"], case["hk"]
        per = case["block"] // case["scales"]
        blocks = sum((a + b - 1) // per - b // per + 1 for a, b in zip(new, held))
        return {"bytes": T * ((2 * hq + 2 * hk) * D * e + 2 * hk * D + R * te + 16) + 2 * 2 * hk * blocks,
                "flops": T * ((hq + hk) * R * 3 + 2 * hk * D * 2)}
    if case["kind"] == "attend":
        e = SIZE[case["dtype"]]
        q, own_len = _lengths(case)
        P, D, per = case["prefix"], case["head"], case["block"] // case["scales"]
        T = sum(q)
        keys = P + sum(own_len)
        seen = sum(a * P + a * b - a * (a - 1) // 2 for a, b in zip(q, own_len))
        blocks = -(-P // case["block"]) + sum(-(-b // case["block"]) for b in own_len)
        scales = -(-P // per) + sum(-(-b // per) for b in own_len)
        return {"bytes": 2 * T * case["hq"] * D * e + 4 * T * case["hq"] + 2 * keys * case["hk"] * D
                + 2 * scales * case["hk"] + 8 * (blocks + 2 * len(q) + 1), "flops": 4 * D * case["hq"] * seen}
    bs = case["block"]
    page = case["layers"] * 2 * case["hk"] * (bs * case["head"] + case["scales"])
    held = _held(case)
    entries = sum(-(-n // bs) for n in held)
    if case["kind"] == "fork":
        blocks, n = entries + case["spare"], max(1, case["beams"])
        rows = case["seqs"] * n
        ragged = sum(1 for v in held if v % bs)
        copied = ragged * (n - 1) if case["beams"] > 0 else ragged * 0.3
        return {"bytes": 8 * entries * (1 + n) + 8 * (case["seqs"] + 3 * rows) + 8 * blocks + 2 * copied * page, "flops": 0}
    live = -(-case["prefix"] // bs) + entries
    blocks = max(live, int(round(live * 100 / (100 - case["holes"]))))
    return {"bytes": 16 * live + 8 * case["seqs"] + 8 * blocks + 2 * page * live * (1 - live / blocks), "flops": 0}


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions, one scale block, token or sequence after the other
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["kind"] in ("fork", "compact"):
        return None  # pages and their numbers: nothing is computed
    s = prepare(case, seed)
    return _exact_append(case, s) if case["kind"] == "append" else _exact_attend(case, s)


def _exact_append(case, s):
    """Cached values as code and scale would have them without the code's rounding."""
    T, D, R, bs, S, hk = len(s["positions"]), case["head"], case["rotary"], case["block"], case["scales"], case["hk"]
    h, per = R // 2, bs // S
    table = s["table"].to(torch.float64)[s["positions"]]
    z = torch.complex(table[:, :h], table[:, h:]).reshape(T, 1, h)

    def turned(x):
        y = x.to(torch.float64).reshape(T, -1, D).clone()
        real = torch.arange(h, device="cuda") * (1 if case["neox"] else 2)
        imag = real + (h if case["neox"] else 1)
        w = torch.complex(y[:, :, real], y[:, :, imag]) * z
        y[:, :, real], y[:, :, imag] = w.real, w.imag
        return y

    slots = s["slots"].tolist()
    runs = [0] + [t for t in range(1, T) if slots[t] != slots[t - 1] + 1 or slots[t] % per == 0] + [T]
    found = []
    for x, cache, scale in ((turned(s["k"]), s["k_cache"], s["k_scale"]),
                            (s["v"].to(torch.float64).reshape(T, -1, D), s["v_cache"], s["v_scale"])):
        codes, power = cache.to(torch.float64), scale.view(torch.uint8).to(torch.float64) - 127
        most = x.abs().amax(-1)
        for a, b in zip(runs, runs[1:]):
            page, at = divmod(slots[a], bs)
            block, before = divmod(at, per)
            e = torch.ceil(torch.log2(most[a:b].amax(0) / 448))
            if before:
                e = torch.maximum(e, power[page, :, block])
                codes[page, :, at - before:at] *= torch.pow(2.0, power[page, :, block] - e)[:, None, None]
            power[page, :, block] = e
            codes[page, :, at:at + b - a] = (x[a:b] * torch.pow(2.0, -e)[:, None]).transpose(0, 1)
        found += [codes, torch.pow(2.0, power)]
    return turned(s["q"]).reshape(T, -1), found[0], found[2], found[1], found[3]


def _exact_attend(case, s):
    hq, hk, D, bs, P, per = *(case[k] for k in ("hq", "hk", "head", "block", "prefix")), case["block"] // case["scales"]
    group = hq // hk
    starts, lens = s["starts"].tolist(), s["seq_lens"].tolist()
    outs, lses = [], []
    for b in range(case["seqs"]):
        new, total = starts[b + 1] - starts[b], lens[b]
        own_at = torch.arange(total - P, device="cuda")
        page, row = s["block_table"][b, own_at // bs], own_at % bs
        if P:
            at = torch.arange(P, device="cuda")
            page, row = torch.cat([s["prefix_blocks"][at // bs], page]), torch.cat([at % bs, row])
        q = s["q"][starts[b]:starts[b + 1]].to(torch.float64).reshape(new, hq, D).transpose(0, 1)
        late = torch.arange(total, device="cuda")[None, :] > (total - new + torch.arange(new, device="cuda"))[:, None]
        o, l = [], []
        for h in range(hk):
            k, v = (c.view(torch.uint8)[page, h, row].view(E4M3).to(torch.float64)
                    * torch.pow(2.0, f.view(torch.uint8)[page, h, row // per].to(torch.float64) - 127)[:, None]
                    for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            score = q[h * group:(h + 1) * group] @ k.T / math.sqrt(D)
            score.masked_fill_(late, -math.inf)
            o.append(torch.softmax(score, -1) @ v)
            l.append(torch.logsumexp(score, -1))
        outs.append(torch.cat(o).transpose(0, 1).reshape(new, hq * D))
        lses.append(torch.cat(l).T)
    return torch.cat(outs), torch.cat(lses)
