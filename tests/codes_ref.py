"""Inputs, 64-bit references and error bounds of the operators on a paged cache of 8-bit codes, and plain
references of those on its pages, for their tests.

A cached value is code * 2^(byte - 127), 0 times the code for byte 0, exact in binary64.  Bounds beside those of serving_ref.py (e = 2^-24):

* append: a code is the nearest of E4M3's values to x' = fl(a c - fl(b s)), whose two roundings are off by e |b s| and
  e |a c - b s| (1 + e): |value - x| <= step(x) / 2 + 4 e (|a c| + |b s|), step being that of E4M3 at x in units of the
  scale (2^-3 of the power of two below, 2^-9 at least).  With |a|, |b| <= the row's largest magnitude r and
  |c|, |s| <= the table's t (r and t are those of the case) the terms are at most 2 r t; values are copied (one term).  The scale byte is a step function of the largest
  magnitude: a reference within 2^-20 of a step's edge may come out on either side.
* attention: the cache's values are exact, so the bounds are those of serving_ref.attend_reference.
"""
import math

import torch

from serving_ref import E32, append_case, append_reference, attend_case, attend_reference

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def bytes_of(t):
    return t.view(torch.uint8)


def e8m0(t):
    return t.to(torch.uint8).view(E8M0)


def values_of(codes, scale):
    """[NB, H, BS, D] codes and [NB, H, S] scales as float64 values."""
    b = bytes_of(scale).double()
    f = torch.where(b == 255, torch.nan, torch.where(b == 0, 0.0, torch.pow(2.0, b - 127)))
    return bytes_of(codes).view(E4M3).double() * f.repeat_interleave(codes.shape[2] // scale.shape[2], 2)[..., None]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def coded_case(seed, dtype, new, own, S=1, spread=3, extreme=None, **kw):
    """serving_ref.attend_case with its keys and values as codes: every scale block in units of its own, from
    2^-(7 + spread) to 2^(spread - 7) of values of about one.  Rows that hold no token are NaN codes, scales of blocks
    without any are NaN."""
    c = attend_case(seed, torch.float64, new, own, **kw)
    c["q"] = c["q"].to(dtype)
    g = torch.Generator().manual_seed(seed + 1000)
    per = c["bs"] // S
    for name in ("k", "v"):
        x = c[name]
        NB, H, BS, D = x.shape
        there = ~torch.isnan(x).all(-1).all(1)  # [NB, BS]
        byte = torch.randint(120 - spread, 121 + spread, (NB, H, S), generator=g)
        if extreme:
            byte = byte + extreme[name]
        empty = ~there.reshape(NB, S, per).any(-1)
        byte[empty[:, None].expand(NB, H, S)] = 255
        # codes: values of about one in units of 2^-7
        codes = (x * 64).float().clamp(-448, 448).to(E4M3)
        c[name + "_codes"], c[name + "_scale"] = codes, e8m0(byte)
        c[name] = values_of(codes, c[name + "_scale"])
    c["S"] = S
    return c


def run_coded(R, c, guards=None, lse=True, stream=None, prepared=False, **kw):
    """(out, lse) of the operator on guarded device copies; rows past the last token hold the canary pattern before
    the call."""
    from guard import Guards
    g = guards or Guards()
    q = g.put(c["q"], "q")[:, :c["width"]]
    rows = c["q"].shape[0]
    out = g.empty((rows, c["width"]), c["q"].dtype, "out")
    ls = g.empty((rows, c["hq"]), torch.float32, "lse") if lse else None
    call = R.prepare_paged_attention_8bit if prepared else R.paged_attention_8bit
    caches = [g.put(bytes_of(c[n]), n).view(c[n].dtype) for n in ("k_codes", "v_codes", "k_scale", "v_scale")]
    r = call(q, *caches, g.put(c["table"], "table"), g.put(c["lens"], "lens"), g.put(c["starts"], "starts"), out,
             scale=c["scale"], prefix_blocks=g.put(c["prefix"], "prefix") if c["P"] else None, prefix_len=c["P"], lse=ls,
             stream=stream, **kw)
    if prepared:
        r()
    g.check()
    return out.cpu(), None if ls is None else ls.cpu()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def codes_append_case(seed, dtype, new, held, bs, S, hq=4, hk=2, D=64, R=None, hv=None, pad=0, scale=1.0, **kw):
    """``new[b]`` tokens for sequences that hold ``held[b]``, in pages somewhere in a cache of codes; ``pad`` padding
    tokens after every sequence."""
    T = sum(new) + pad * len(new)
    c = append_case(seed, dtype, T, hq, hk, D, R or D, bs, hv=hv, pad_every=0, NB=1, **kw)
    hv = c["hv"]
    g = torch.Generator().manual_seed(seed + 2000)
    need = [-(-(n + h) // bs) for n, h in zip(new, held)]
    NB = sum(need) + 2
    pages = torch.randperm(NB, generator=g).tolist()
    slots, at = [], 0
    for b in range(len(new)):
        mine = pages[at:at + need[b]]
        at += need[b]
        slots += [mine[j // bs] * bs + j % bs for j in range(held[b], held[b] + new[b])] + [-1] * pad
    c["slots"] = torch.tensor(slots, dtype=torch.int64)
    c["S"], c["hv"] = S, hv
    if scale != 1.0:  # blocks of different sizes
        for n in ("k", "v"):
            f = torch.pow(torch.tensor(scale), torch.randn(T, 1, generator=g))
            c[n] = (c[n].float() * f).to(dtype)
    for n, h in (("k", hk), ("v", hv)):
        codes = torch.randint(0, 256, (NB, h, bs, D), generator=g)
        codes[(codes & 0x7f) == 0x7f] = 0x22
        c[n + "c"] = codes.to(torch.uint8).view(E4M3)
        c[n + "s"] = e8m0(torch.randint(115, 124, (NB, h, S), generator=g))
    return c


def coded(x64, byte):
    """The nearest E4M3 code of x64 / 2^(byte - 127) and the value before."""
    y = x64 * 2.0 ** (127 - byte)
    return y


def codes_append_reference(c):
    """(q_out, [(name, codes' uncoded values per row or None)], ...): for K and V a dict with the expected scale bytes
    [NB, H, S], whether a byte's edge is near, which rows were written (with their exact values in units of the scale)
    and the expected codes of all others."""
    d = dict(c, kc=torch.zeros(1, c["hk"], c["bs"], c["D"]), vc=torch.zeros(1, c["hv"], c["bs"], c["D"]))
    T, D, bs, S = c["q"].shape[0], c["D"], c["bs"], c["S"]
    per = bs // S
    # the rotation, from the reference of the plain append: one page that all tokens go through
    d["slots"] = torch.full((T,), -1, dtype=torch.int64)
    q_out, _, _, skipped = append_reference(d)
    dk = dict(d, q=c["k"], hq=c["hk"])
    k_rot = append_reference(dk)[0].reshape(T, c["hk"], D)
    out = []
    largest = float(c["table"].double().abs().max())
    for n, x, H in (("k", k_rot, c["hk"]), ("v", c["v"].double().reshape(T, c["hv"], D), c["hv"])):
        codes, scale = bytes_of(c[n + "c"]).clone(), bytes_of(c[n + "s"]).clone().int()
        value = torch.full(codes.shape, math.nan, dtype=torch.float64)  # of written rows, in units of the scale
        written = torch.zeros(codes.shape[:3], dtype=torch.bool)
        near = torch.zeros(scale.shape, dtype=torch.bool)
        terms = torch.zeros(codes.shape[:3], dtype=torch.float64)
        slots = c["slots"].tolist()
        t = 0
        total = codes.shape[0] * bs
        while t < T:
            if not 0 <= slots[t] < total:
                t += 1
                continue
            m = 1
            while t + m < T and slots[t + m] == slots[t] + m and slots[t + m] % per:
                m += 1
            page, at = divmod(slots[t], bs)
            part, first = divmod(at, per)
            use = [i for i in range(t, t + m) if i not in skipped]
            for h in range(H):
                if not use:
                    break
                v = x[use, h]
                finite = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))
                most = float(finite.max())
                byte = 0
                if most > 0:
                    e = math.ceil(math.log2(most / 448))
                    while most > 448 * 2.0 ** e:
                        e += 1
                    while most <= 448 * 2.0 ** (e - 1):
                        e -= 1
                    byte = min(max(e + 127, 1), 254)
                    ratio = most / (448 * 2.0 ** (byte - 127))
                    near[page, h, part] = ratio > 1 - 2.0 ** -20 or ratio < 0.5 * (1 + 2.0 ** -20)
                old = int(scale[page, h, part])
                if first and old >= byte:
                    byte = old
                    near[page, h, part] = False
                elif first:
                    rows = codes[page, h, at - first:at].view(E4M3).double() * 2.0 ** (old - byte)
                    codes[page, h, at - first:at] = bytes_of(rows.float().to(E4M3))
                scale[page, h, part] = byte
                for i in use:
                    value[page, h, at + i - t] = x[i, h] * 2.0 ** (127 - byte)
                    if n == "k":
                        raw = c["k"].double().reshape(T, H, D)[i, h].abs()
                        raw = float(torch.where(torch.isfinite(raw), raw, torch.zeros_like(raw)).max())
                        terms[page, h, at + i - t] = 2 * raw * largest * 2.0 ** (127 - byte)
                    written[page, h, at + i - t] = True
            t += m
        out.append({"codes": codes, "scale": scale, "value": value, "written": written, "near": near, "terms": terms})
    return q_out, skipped, out


def check_codes(got_codes, got_scale, want, what):
    codes, scale = bytes_of(got_codes).cpu(), bytes_of(got_scale).cpu().int()
    S = scale.shape[2]
    near = want["near"]
    same = (scale == want["scale"]) | (near & ((scale - want["scale"]).abs() <= 1))
    assert bool(same.all()), (what, "scale", scale[~same], want["scale"][~same])
    sure = (scale == want["scale"]).repeat_interleave(codes.shape[2] // S, 2)
    w = want["written"] & sure
    kept = ~want["written"] & sure
    assert torch.equal(codes[kept], want["codes"][kept]), what + " rows that stay"
    v, g = want["value"][w], codes[w].view(E4M3).double()
    terms = want["terms"][w][:, None].expand_as(v)
    bad = ~torch.isfinite(v)
    assert bool(torch.isnan(g[bad]).all()), what + " values that are not finite"
    v, g, terms = v[~bad], g[~bad], terms[~bad]
    step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    err = (g - v).abs()
    assert bool((err <= step / 2 + 4 * E32 * (v.abs() + terms)).all()), (what, float((err - step / 2).max()))


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def pages_case(seed, lens, bs, P=0, spare=7, share=True, spare_columns=2):
    """Tables of sequences of ``lens`` own tokens behind a prefix of P; every third shares whole pages with the one
    before it."""
    g = torch.Generator().manual_seed(seed)
    shared = -(-P // bs)
    held = [-(-n // bs) for n in lens]
    NB = shared + sum(held) + spare
    pages = torch.randperm(NB, generator=g).tolist()
    W = max(held + [1]) + spare_columns
    table = torch.full((len(lens), W), 1 << 40, dtype=torch.int64)
    refs = torch.zeros(NB, dtype=torch.int32)
    prefix, at = pages[:shared], shared
    for p in prefix:
        refs[p] += 1
    for b, n in enumerate(held):
        mine = pages[at:at + n]
        at += n
        if share and b % 3 == 2:
            same = min(lens[b] // bs, lens[b - 1] // bs) // 2
            mine[:same] = table[b - 1, :same].tolist()
        for j, p in enumerate(mine):
            table[b, j] = p
            refs[p] += 1
    return {"table": table, "lens": torch.tensor([P + n for n in lens], dtype=torch.int64), "refs": refs, "bs": bs, "P": P,
            "prefix": torch.tensor(prefix, dtype=torch.int64), "NB": NB}


def rearrange_reference(c, parents, room=None, new_W=None, canary=-77):
    """What rope_rearrange_sequences says, row by row."""
    bs, P, NB = c["bs"], c["P"], c["NB"]
    refs = c["refs"].tolist()
    table, lens = c["table"].tolist(), c["lens"].tolist()
    W = c["table"].shape[1]
    new_W = new_W or W
    held = lambda n: -(-max(n - P, 0) // bs)  # noqa: E731
    for b in range(len(lens)):
        for j in range(min(held(lens[b]), W)):
            refs[table[b][j]] -= 1
    new, new_lens, need, pairs, claimed = [], [], [], [], set()
    own_of = [max(lens[p] - P, 0) if p >= 0 else 0 for p in parents]
    keeps = []
    for i, p in enumerate(parents):  # whole pages first: who holds one keeps others from writing on it
        for j in range(own_of[i] // bs):
            refs[table[p][j]] += 1
    for i, p in enumerate(parents):
        full, rest = divmod(own_of[i], bs)
        k = False
        if rest:
            last = table[p][full]
            k = refs[last] == 0 and last not in claimed
            claimed |= {last} if k else set()
        keeps.append(k)
    for i, p in enumerate(parents):
        full, rest = divmod(own_of[i], bs)
        row = [table[p][j] for j in range(full + keeps[i])] if p >= 0 else []
        if keeps[i]:
            refs[row[-1]] += 1
        new.append(row)
        grown = own_of[i] + (room[i] if room is not None else 0)
        new_lens.append(P + grown)
        need.append(-(-grown // bs) - len(row))
    free = [j for j in range(NB) if refs[j] == 0]
    for i, p in enumerate(parents):
        if own_of[i] % bs and not keeps[i]:
            pairs.append((table[p][own_of[i] // bs], free[0] if free else -1))
        for _ in range(need[i]):
            if free:
                refs[free[0]] = 1
                new[i].append(free.pop(0))
            else:
                new[i].append(-1)
    rows = len(parents)
    out = torch.full((rows, new_W), canary, dtype=torch.int64)
    for i in range(rows):
        out[i, :len(new[i])] = torch.tensor(new[i], dtype=torch.int64)
    src = [s for s, _ in pairs] + [-1] * (rows - len(pairs))
    dst = [d for _, d in pairs] + [-1] * (rows - len(pairs))
    return {"new_table": out, "new_lens": torch.tensor(new_lens, dtype=torch.int64), "new_refs": torch.tensor(refs, dtype=torch.int32),
            "src": torch.tensor(src, dtype=torch.int64), "dst": torch.tensor(dst, dtype=torch.int64),
            "counts": torch.tensor([len(pairs), len(free)], dtype=torch.int64)}


def compact_reference(c, pairs, canary=-77):
    refs = c["refs"].tolist()
    NB, bs, P = c["NB"], c["bs"], c["P"]
    live = [j for j in range(NB) if refs[j] > 0]
    L = len(live)
    holes = [j for j in range(L) if refs[j] <= 0]
    movers = [j for j in live if j >= L]
    to = dict(zip(movers, holes))
    new_refs = [0] * NB
    for j in live:
        new_refs[to.get(j, j)] = refs[j]
    table = torch.full_like(c["table"], canary)
    for b in range(table.shape[0]):
        for j in range(-(-max(int(c["lens"][b]) - P, 0) // bs)):
            p = int(c["table"][b, j])
            table[b, j] = to.get(p, p)
    pad = [-1] * (pairs - len(movers))
    return {"new_table": table, "new_refs": torch.tensor(new_refs, dtype=torch.int32),
            "new_prefix": torch.tensor([to.get(p, p) for p in c["prefix"].tolist()], dtype=torch.int64),
            "src": torch.tensor(movers + pad, dtype=torch.int64), "dst": torch.tensor(holes + pad, dtype=torch.int64),
            "counts": torch.tensor([len(movers), L], dtype=torch.int64)}
