"""Cases of the operators that make rotary tables, append to a paged cache and attend over it.

Three kinds of case, in the order in which a serving program meets them:

* ``table``: the cos/sin rows of positions under a long-context scaling;
* ``append``: queries and keys rotated, keys and values written to their cache slots;
* ``attend``: attention of a batch's new tokens over the paged cache, whose sequences
  may share the pages of a long prefix.

``run`` computes them with elementary torch operations in 32 bits (angles in 64)
where ``own`` is false, and with this package's operators where it is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _table(name, dtype, rows, dim, scaling, layout, base=10000.0, first=0, packed=False):
    return {"name": name, "kind": "table", "dtype": dtype, "rows": rows, "dim": dim, "scaling": scaling,
            "layout": layout, "base": base, "first": first, "packed": packed}


def _append(name, dtype, tokens, hq, hk, head, rotary, neox, block, sections="", table="same", fused=True):
    return {"name": name, "kind": "append", "dtype": dtype, "tokens": tokens, "hq": hq, "hk": hk, "head": head,
            "rotary": rotary, "neox": neox, "block": block, "sections": sections, "table": table, "fused": fused}


def _attend(name, dtype, seqs, new, prefix, own_max, hq, hk, head, block):
    """``seqs`` sequences with 1..``new`` new tokens each (all ``new`` where it is given negative), on top of up to
    ``own_max`` tokens of their own (new ones included) after ``prefix`` shared ones."""
    return {"name": name, "kind": "attend", "dtype": dtype, "seqs": seqs, "new": new, "prefix": prefix,
            "own_max": own_max, "hq": hq, "hk": hk, "head": head, "block": block}


def listed():
    return [
        # cos and sin of a packed training batch in 32 bits, for the in-place rotation of a slice of 64 columns
        _table("table_f32_packed_2048x64", "f32", 2048, 64, "linear", "half", packed=True),
        # the whole cos/sin cache of a 128-column rotation stretched to a long context, made at load
        _table("table_bf16_cache_131072x128", "bf16", 131072, 128, "yarn", "cache", base=1000000.0),
        # one decoding step of 64 requests: latency
        _append("append_bf16_64tok_32q8k_h128", "bf16", 64, 32, 8, 128, 128, True, 16),
        # a prompt chunk of 16384 tokens, q, k and v being column ranges of one projection, table in 32 bits
        _append("append_bf16_16384tok_32q8k_h128", "bf16", 16384, 32, 8, 128, 128, True, 16, table="f32"),
        # the interleaved layout on the first 64 of 256 columns, all heads their own keys
        _append("append_f16_8192tok_16q16k_h256_r64", "f16", 8192, 16, 16, 256, 64, False, 32),
        # image and text positions in three sections, 32 bits, an odd token count and an odd page
        _append("append_f32_mrope_1003tok_28q4k_h128", "f32", 1003, 28, 4, 128, 128, True, 12, sections="16,24,24",
                fused=False),
        # one decoding step of 4 short requests: latency
        _attend("attend_bf16_4seq_decode_300", "bf16", 4, -1, 0, 300, 32, 8, 128, 16),
        # one decoding step of 64 requests of up to 8192 tokens, nothing shared: bound by the cache's bytes
        _attend("attend_bf16_64seq_decode_8192", "bf16", 64, -1, 0, 8192, 32, 8, 128, 16),
        # one decoding step of 128 requests behind one long shared prompt
        _attend("attend_bf16_128seq_decode_p16384", "bf16", 128, -1, 16384, 1024, 32, 8, 128, 16),
        # prompt chunks of 1984 tokens behind a shared prompt of 4096: bound by the matrix units
        _attend("attend_bf16_4seq_chunks_p4096", "bf16", 4, -1984, 4096, 1984, 32, 8, 128, 16),
        # up to 5 drafted tokens a request to be verified, heads of 256, pages that are no power of two
        _attend("attend_f16_32seq_draft5_p2048_h256", "f16", 32, 5, 2048, 517, 16, 16, 256, 12),
        # 32 bits, ragged in everything
        _attend("attend_f32_6seq_ragged_p101_h64", "f32", 6, 40, 101, 333, 4, 2, 64, 17),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One case of the listed ones' ranges."""
    kind = rng.choice(["table", "append", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "table":
        c = _table("", dtype, _log(rng, 1, 131072), 2 * _log(rng, 8, 64), rng.choice(["none", "linear", "base", "yarn", "wavelength"]),
                   rng.choice(["cache", "half", "interleave"]), rng.choice([10000.0, 500000.0, 1000000.0]),
                   rng.choice([0, _log(rng, 1, 1000000)]), rng.random() < 0.5)
    elif kind == "append":
        hk = rng.choice([1, 2, 3, 4, 8])
        head = 32 * rng.randint(2, 8)
        sections = rng.choice(["", "", "16,24,24", "8,12,12", "16,16,16,16"])
        rotary = 2 * sum(int(v) for v in sections.split(",")) if sections else min(head, 32 * rng.randint(1, 8))
        head = max(head, rotary)
        c = _append("", dtype, _log(rng, 1, 8192), hk * rng.choice([1, 2, 4, 5, 7]), hk, head, rotary, rng.random() < 0.7,
                    rng.choice([1, 12, 16, 17, 32, 64, 128]), sections, rng.choice(["same", "f32"]), rng.random() < 0.5)
    else:
        most = work(listed()[9])["flops"]
        while True:
            hk = rng.choice([1, 2, 4, 8])
            head = rng.choice([64, 64, 96, 128, 128, 128, 160, 256])
            new = rng.choice([-1, -1, 8, -_log(rng, 2, 64), _log(rng, 2, 2048)])
            c = _attend("", dtype, _log(rng, 1, 128), new, rng.choice([0, _log(rng, 1, 16384)]),
                        abs(new) + _log(rng, 1, 4096), hk * rng.choice([1, 2, 4, 5, 8]), hk, head,
                        rng.choice([12, 16, 17, 32, 64, 128]))
            # no more than the largest listed one costs either side; the plain form's scores stay a few GB
            scores = c["seqs"] * abs(new) * c["hq"] * (c["prefix"] + c["own_max"])
            pages = c["seqs"] * c["own_max"] * hk * head
            if work(c)["flops"] < most / (8 if dtype == "f32" else 1) and scores < 1.5e9 and pages < 3e8:
                break
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lengths(case):
    """(new tokens, own tokens) of every sequence: ragged over the whole range, the same for every seed."""
    n, new = case["seqs"], case["new"]
    spread = [((i * 7919 + 3) % 9973) / 9973.0 for i in range(n)]
    q = [-new if new < 0 else 1 + int(s * new) for s in spread]
    own_len = [max(a, int(round(case["own_max"] * (1.0 - 0.97 * ((i * 0.6180339887) % 1.0))))) for i, a in enumerate(q)]
    return q, own_len


def _frequencies(case):
    """Scaling as a program's configuration names it."""
    kind = case["scaling"]
    if kind in ("linear", "base"):
        return {"kind": kind, "factor": 4.0}
    if kind == "yarn":
        return {"kind": "yarn", "factor": 8.0, "original_length": 16384}
    if kind == "wavelength":
        return {"kind": "wavelength", "factor": 8.0, "low": 1.0, "high": 4.0, "original_length": 8192}
    return None


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32 if dtype == torch.float32 else dtype)

    if case["kind"] == "table":
        rows, dim = case["rows"], case["dim"]
        s["scaling"] = _frequencies(case)
        # the seed moves the positions: another window of the context, or another packing of sequences
        s["first"] = case["first"] + int(torch.randint(0, 4096, (1,), generator=g, device=dev))
        s["positions"] = None
        if case["packed"]:
            s["positions"] = torch.randint(0, 131072, (rows,), generator=g, device=dev)
        if case["layout"] == "cache":
            s["cache"] = torch.empty(rows, dim, device=dev, dtype=dt)
        else:
            s["cos"] = torch.empty(1, rows, 1, dim, device=dev, dtype=dt)
            s["sin"] = torch.empty(1, rows, 1, dim, device=dev, dtype=dt)
        return s

    if case["kind"] == "append":
        T, hq, hk, D, R, bs = (case[k] for k in ("tokens", "hq", "hk", "head", "rotary", "block"))
        if case["fused"]:
            qkv = normal(T, (hq + 2 * hk) * D)
            s["q"], s["k"], s["v"] = qkv[:, :hq * D], qkv[:, hq * D:(hq + hk) * D], qkv[:, (hq + hk) * D:]
        else:
            s["q"], s["k"], s["v"] = normal(T, hq * D), normal(T, hk * D), normal(T, hk * D)
        length = 32768
        tdt = torch.float32 if case["table"] == "f32" else dt
        angle = torch.arange(length, device=dev, dtype=torch.float64)[:, None] * torch.pow(
            torch.tensor(10000.0, device=dev, dtype=torch.float64),
            -torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).to(tdt)
        m = len(case["sections"].split(",")) if case["sections"] else 0
        s["sections"] = [int(v) for v in case["sections"].split(",")] if m else None
        s["positions"] = torch.randint(0, length, (m, T) if m else (T,), generator=g, device=dev)
        blocks = -(-T // bs) + 3
        order = torch.randperm(blocks * bs, generator=g, device=dev)[:T]
        padding = torch.arange(T) % 61 == 60  # a program knows which of its tokens are padding
        s["slots"] = torch.where(padding.to(dev), torch.full_like(order, -1), order)
        s["kept"] = torch.nonzero(~padding)[:, 0].to(dev)
        s["k_cache"], s["v_cache"] = normal(blocks, hk, bs, D), normal(blocks, hk, bs, D)
        s["q_out"] = torch.empty(T, hq * D, device=dev, dtype=dt)
        return s

    q, own_len = _lengths(case)
    hq, hk, D, bs, P = (case[k] for k in ("hq", "hk", "head", "block", "prefix"))
    order = torch.randperm(len(q), generator=torch.Generator().manual_seed(seed)).tolist()  # the seed shuffles the sequences
    q, own_len = [q[i] for i in order], [own_len[i] for i in order]
    T = sum(q)
    s["new_max"], s["own_max"] = max(q), max(own_len)  # a program knows these when it makes up the batch
    s["q"] = normal(T, hq * D)
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
    s["k_cache"], s["v_cache"] = normal(blocks, hk, bs, D), normal(blocks, hk, bs, D)
    s["out"] = torch.empty(T, hq * D, device=dev, dtype=dt)
    s["lse"] = torch.empty(T, hq, device=dev, dtype=torch.float32)
    return s


# ---------------------------------------------------------------------------
# The calls, and the plain forms
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        import transformer_rope_positional_gb300 as R

        if case["kind"] == "table":
            inv, scale = R.rope_frequencies(case["dim"], case["base"], s["scaling"])
            if case["layout"] == "cache":
                R.scaled_cos_sin_cache(s["cache"], inv, scale, positions=s["positions"], first_position=s["first"])
                return s["cache"]
            R.scaled_cos_sin(s["cos"], s["sin"], inv, scale, case["layout"], positions=s["positions"],
                             first_position=s["first"])
            return s["cos"], s["sin"]
        if case["kind"] == "append":
            R.append_paged_kv(s["positions"], s["q"], s["k"], s["v"], s["table"], s["slots"], s["k_cache"], s["v_cache"],
                              case["head"], is_neox=case["neox"], mrope_section=s["sections"], query_out=s["q_out"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        R.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["starts"], s["out"],
                          scale=case["head"] ** -0.5, prefix_blocks=s["prefix_blocks"], prefix_len=case["prefix"],
                          lse=s["lse"])
        return s["out"], s["lse"]
    if case["kind"] == "table":
        return _plain_table(s)
    return _plain_append(s) if case["kind"] == "append" else _plain_attend(s)


def _plain_table(s):
    case, dev = s["case"], torch.device("cuda")
    dim, base, sc = case["dim"], case["base"], s["scaling"]
    i = torch.arange(0, dim, 2, device=dev, dtype=torch.float64)
    scale = 1.0
    if sc is not None and sc["kind"] == "base":
        base = base * sc["factor"] ** (dim / (dim - 2))
    f = base ** (-i / dim)
    if sc is not None and sc["kind"] == "linear":
        f = f / sc["factor"]
    elif sc is not None and sc["kind"] == "yarn":
        def turns(n):  # the frequency index that makes n turns over the original length
            return dim * math.log(sc["original_length"] / (2 * math.pi * n)) / (2 * math.log(base))

        low, high = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), dim - 1)
        ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / sc["factor"] * ramp + f * (1 - ramp)
        scale = 0.1 * math.log(sc["factor"]) + 1.0
    elif sc is not None and sc["kind"] == "wavelength":
        turned = sc["original_length"] * f / (2 * math.pi)
        keep = ((turned - sc["low"]) / (sc["high"] - sc["low"])).clamp(0, 1)
        f = f * keep + f / sc["factor"] * (1 - keep)
    pos = s["first"] + (s["positions"] if s["positions"] is not None else torch.arange(case["rows"], device=dev))
    angle = pos.double()[:, None] * f
    cos, sin = (angle.cos() * scale).to(DTYPES[case["dtype"]]), (angle.sin() * scale).to(DTYPES[case["dtype"]])
    if case["layout"] == "cache":
        return torch.cat([cos, sin], 1)
    if case["layout"] == "half":
        cos, sin = torch.cat([cos, cos], 1), torch.cat([sin, sin], 1)
    else:
        cos, sin = cos.repeat_interleave(2, 1), sin.repeat_interleave(2, 1)
    return cos[None, :, None, :], sin[None, :, None, :]


def _plain_append(s):
    case = s["case"]
    D, R, bs = case["head"], case["rotary"], case["block"]
    row = s["table"][s["positions"]].float()  # [T, R] or [m, T, R]
    cos, sin = row[..., :R // 2], row[..., R // 2:]
    if s["sections"] is not None:
        which = torch.repeat_interleave(torch.arange(len(s["sections"]), device=row.device),
                                        torch.tensor(s["sections"], device=row.device))
        col = torch.arange(R // 2, device=row.device)
        cos, sin = cos[which, :, col].T, sin[which, :, col].T
    cos, sin = cos[:, None, :], sin[:, None, :]

    def rotate(x):
        x = x.float().reshape(x.shape[0], -1, D)
        a, b = (x[..., :R // 2], x[..., R // 2:R]) if case["neox"] else (x[..., 0:R:2], x[..., 1:R:2])
        first, second = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat([first, second], -1) if case["neox"] else torch.stack([first, second], -1).flatten(-2)
        return torch.cat([turned, x[..., R:]], -1).to(DTYPES[case["dtype"]])

    q, k = rotate(s["q"]), rotate(s["k"])
    v = s["v"].reshape(s["v"].shape[0], -1, D)
    slot = s["slots"][s["kept"]]
    s["k_cache"][slot // bs, :, slot % bs] = k[s["kept"]]
    s["v_cache"][slot // bs, :, slot % bs] = v[s["kept"]]
    return q.reshape(q.shape[0], -1), s["k_cache"], s["v_cache"]


def _plain_attend(s):
    """The whole batch at once, padded to its longest sequence."""
    case, dev = s["case"], s["q"].device
    hq, hk, D, bs, P = (case[k] for k in ("hq", "hk", "head", "block", "prefix"))
    G, B, n, own_max = hq // hk, case["seqs"], s["new_max"], s["own_max"]
    new = s["starts"][1:] - s["starts"][:-1]
    token = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(s["starts"], token, right=True) - 1
    there = seq, token - s["starts"][seq]  # the place of every token in the padded batch
    q = torch.zeros(B, n, hk, G, D, device=dev)
    q[there] = s["q"].float().reshape(-1, hk, G, D) * D ** -0.5
    position = s["seq_lens"][:, None] - new[:, None] + torch.arange(n, device=dev)  # [B, n]

    pages = s["block_table"][:, :-(-own_max // bs)]

    def own_part(cache):  # [B, hk, own_max, D]
        return cache[pages].permute(0, 2, 1, 3, 4).reshape(B, hk, -1, D)[:, :, :own_max].float()

    def prefix_part(cache):  # [hk, P, D]
        return cache[s["prefix_blocks"]].permute(1, 0, 2, 3).reshape(hk, -1, D)[:, :P].float()

    qo = q.permute(0, 2, 1, 3, 4).reshape(B, hk, n * G, D)
    so = torch.matmul(qo, own_part(s["k_cache"]).transpose(-1, -2)).reshape(B, hk, n, G, own_max)
    seen = (P + torch.arange(own_max, device=dev)) <= position[..., None]  # [B, n, own_max]
    so = so.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = so.amax(-1)  # [B, hk, n, G]
    if P:
        qp = q.permute(2, 0, 1, 3, 4).reshape(hk, B * n * G, D)
        sp = torch.matmul(qp, prefix_part(s["k_cache"]).transpose(-1, -2)).reshape(hk, B, n, G, P)
        top = torch.maximum(top, sp.amax(-1).permute(1, 0, 2, 3))
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    so = torch.exp(so - top[..., None])
    total = so.sum(-1)
    o = torch.matmul(so.reshape(B, hk, n * G, own_max), own_part(s["v_cache"])).reshape(B, hk, n, G, D)
    if P:
        sp = torch.exp(sp - top.permute(1, 0, 2, 3)[..., None])
        total = total + sp.sum(-1).permute(1, 0, 2, 3)
        op = torch.matmul(sp.reshape(hk, B * n * G, P), prefix_part(s["v_cache"]))
        o = o + op.reshape(hk, B, n, G, D).permute(1, 0, 2, 3, 4)
    o = (o / total[..., None]).permute(0, 2, 1, 3, 4)[there]
    lse = (total.log() + top).permute(0, 2, 1, 3)[there]
    return o.reshape(-1, hq * D).to(DTYPES[case["dtype"]]), lse.reshape(-1, hq)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = SIZE[case["dtype"]]
    if case["kind"] == "table":
        values = case["rows"] * case["dim"]
        wide = 1 if case["layout"] == "cache" else 2
        return {"bytes": values * wide * e + (8 * case["rows"] if case["packed"] else 0), "flops": values * 10}
    if case["kind"] == "append":
        T, D, R = case["tokens"], case["head"], case["rotary"]
        heads = case["hq"] + 2 * case["hk"]
        te = 4 if case["table"] == "f32" else e
        m = len(case["sections"].split(",")) if case["sections"] else 1
        return {"bytes": T * (2 * heads * D * e + R * te + 8 * m + 8), "flops": T * (case["hq"] + case["hk"]) * R * 3}
    q, own_len = _lengths(case)
    P, D = case["prefix"], case["head"]
    T = sum(q)
    keys = P + sum(own_len)
    seen = sum(a * P + a * b - a * (a - 1) // 2 for a, b in zip(q, own_len))
    blocks = -(-P // case["block"]) + sum(-(-b // case["block"]) for b in own_len)
    return {"bytes": 2 * T * case["hq"] * D * e + 4 * T * case["hq"] + 2 * keys * case["hk"] * D * e + 8 * (blocks + 2 * len(q) + 1),
            "flops": 4 * D * case["hq"] * seen}


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions, one position, token or sequence after the other
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "table":
        return _exact_table(case, s)
    return _exact_append(case, s) if case["kind"] == "append" else _exact_attend(case, s)


def _exact_table(case, s):
    dim, sc = case["dim"], s["scaling"]
    kind = sc["kind"] if sc else "none"
    f, gain = [], 1.0
    for k in range(dim // 2):
        base = case["base"]
        if kind == "base":
            base *= math.pow(sc["factor"], dim / (dim - 2.0))
        w = math.exp(-2.0 * k / dim * math.log(base))
        if kind == "linear":
            w /= sc["factor"]
        elif kind == "yarn":
            # between 32 turns over the original length (kept) and one (stretched) the two are mixed linearly in k
            edge = [dim / 2.0 * math.log(sc["original_length"] / (n * 2.0 * math.pi)) / math.log(base) for n in (32.0, 1.0)]
            lo, hi = max(0, math.floor(edge[0])), min(dim - 1, math.ceil(edge[1]))
            mix = min(1.0, max(0.0, (k - lo) / max(hi - lo, 0.001)))
            w = w * (1.0 - mix) + w / sc["factor"] * mix
            gain = 1.0 + 0.1 * math.log(sc["factor"])
        elif kind == "wavelength":
            wave = 2.0 * math.pi / w
            if wave > sc["original_length"] / sc["low"]:
                w /= sc["factor"]
            elif wave >= sc["original_length"] / sc["high"]:
                t = (sc["original_length"] / wave - sc["low"]) / (sc["high"] - sc["low"])
                w = (1.0 - t) * w / sc["factor"] + t * w
        f.append(w)
    at = s["positions"] if s["positions"] is not None else torch.arange(case["rows"], device="cuda")
    turn = torch.outer((at + s["first"]).to(torch.float64), torch.tensor(f, dtype=torch.float64, device="cuda"))
    # the angle less its whole turns, then e^(i angle)
    z = gain * torch.polar(torch.ones_like(turn), torch.remainder(turn, 2.0 * math.pi))
    c, n = z.real, z.imag
    if case["layout"] == "cache":
        return torch.hstack([c, n])
    shape = (1, case["rows"], 1, dim)
    order = torch.arange(dim, device="cuda") % (dim // 2) if case["layout"] == "half" else torch.arange(dim, device="cuda") // 2
    return c[:, order].reshape(shape), n[:, order].reshape(shape)


def _exact_append(case, s):
    T, D, R, bs = case["tokens"], case["head"], case["rotary"], case["block"]
    h = R // 2
    pos = s["positions"] if s["sections"] else s["positions"][None]
    ends = torch.tensor(s["sections"] or [h], device="cuda").cumsum(0)
    row_of = torch.bucketize(torch.arange(h, device="cuda"), ends, right=True)
    table = s["table"].to(torch.float64)
    token_pos = pos[row_of]  # [h, T]
    z = torch.complex(table[token_pos, torch.arange(h, device="cuda")[:, None]],
                      table[token_pos, h + torch.arange(h, device="cuda")[:, None]]).T.reshape(T, 1, h)

    def turned(x):
        y = x.to(torch.float64).reshape(T, -1, D).clone()
        real = torch.arange(h, device="cuda") * (1 if case["neox"] else 2)
        imag = real + (h if case["neox"] else 1)
        w = torch.complex(y[:, :, real], y[:, :, imag]) * z
        y[:, :, real], y[:, :, imag] = w.real, w.imag
        return y

    kc, vc = s["k_cache"].to(torch.float64), s["v_cache"].to(torch.float64)
    k, v = turned(s["k"]), s["v"].to(torch.float64).reshape(T, -1, D)
    to = [t for t, slot in enumerate(s["slots"].tolist()) if slot >= 0]
    slot = s["slots"][to]
    flat_k, flat_v = kc.transpose(1, 2).contiguous().view(-1, case["hk"], D), vc.transpose(1, 2).contiguous().view(-1, case["hk"], D)
    flat_k[slot], flat_v[slot] = k[to], v[to]
    back = lambda f: f.view(-1, bs, case["hk"], D).transpose(1, 2).contiguous()  # noqa: E731
    return turned(s["q"]).reshape(T, -1), back(flat_k), back(flat_v)


def _exact_attend(case, s):
    hq, hk, D, bs, P = (case[k] for k in ("hq", "hk", "head", "block", "prefix"))
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
            k, v = s["k_cache"][page, h, row].to(torch.float64), s["v_cache"][page, h, row].to(torch.float64)
            score = q[h * group:(h + 1) * group] @ k.T / math.sqrt(D)
            score.masked_fill_(late, -math.inf)
            o.append(torch.softmax(score, -1) @ v)
            l.append(torch.logsumexp(score, -1))
        outs.append(torch.cat(o).transpose(0, 1).reshape(new, hq * D))
        lses.append(torch.cat(l).T)
    return torch.cat(outs), torch.cat(lses)
