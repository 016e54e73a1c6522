"""Inputs, 64-bit references and error bounds of the serving operators (scaled rotary
tables, append to a paged cache, paged attention), for their tests.

Bounds, u = torch.finfo(dtype).eps / 2 being half a step of the output type and
e = 2^-24 half a step of binary32:

* tables: the binary32 value is within 4 e |value| of scale * sin or cos (angle exact to
  2^-64 turns, 2 units of the polynomial and its argument, one product with scale), the
  reference's angle p * f has an error of 2^-53 |angle|:   u |r| + 4 e |r| + 2^-52 |angle|.
* append: one correctly rounded FMA or a compensated difference (2 e |r|), rounded once:
  u |r| + 4 e |r|.
* attention: scores are binary32 sums of D products, off by at most
  d = scale * 2 (D + 4) e * max_j sum_i |q_i k_ji| (a factor 2 for sums that truncate); a weight
  e^(s - m) is then off by the factor e^(d + 8 e), and rounded to the data's type (u); sums over
  n keys are off by n e relative to their terms.  With A = sum_j w_j |v_j|:
      out: u |o| + (u_w + 2 d + (4 n + 64) e) A,   u_w = u, or 0 for binary32
      lse: d + (n + 64) e + 4 e |lse|
  Values below the normal range are off by up to half the smallest step (tiny).
"""
import math

import torch

E32 = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def assert_close(got, ref, tol, what):
    """Every element of got within tol of the float64 ref (NaN and infinities must match)."""
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    same = (torch.isnan(g) & torch.isnan(ref)) | (g == ref)
    err = (g - ref).abs()
    ok = same | (err <= tol)
    if not bool(ok.all()):
        bad = (~ok).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError("%s: %d of %d elements outside the bound, first at %s: got %r, expected %r, bound %r"
                             % (what, len(bad), ok.numel(), i, float(g[i]), float(ref[i]), float(tol[i])))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attend_case(seed, dtype, new, own, P=0, hq=4, hk=2, D=64, bs=16, spare_pages=1, spare_rows=0, stride_pad=0,
                fill=float("nan"), q_scale=1.0):
    """A batch on the CPU: ``new[b]`` new tokens as the last of ``own[b]`` own tokens after P
    shared ones.  Cache rows that hold no token are ``fill``."""
    g = torch.Generator().manual_seed(seed)
    B, T = len(new), sum(new)
    held = [-(-n // bs) for n in own]
    shared = -(-P // bs)
    NB = shared + sum(held) + 2
    pages = torch.randperm(NB, generator=g)
    W = max(max(held), 1) + spare_pages
    table = torch.full((B, W), 1 << 40, dtype=torch.int64)  # entries past a sequence's pages are never read
    at = shared
    for b in range(B):
        table[b, :held[b]] = pages[at:at + held[b]]
        at += held[b]
    prefix = pages[:shared].clone()
    k = torch.full((NB, hk, bs, D), fill, dtype=dtype)
    v = torch.full((NB, hk, bs, D), fill, dtype=dtype)
    for j in range(P):
        k[prefix[j // bs], :, j % bs] = torch.randn(hk, D, generator=g).to(dtype)
        v[prefix[j // bs], :, j % bs] = torch.randn(hk, D, generator=g).to(dtype)
    for b in range(B):
        for j in range(own[b]):
            k[table[b, j // bs], :, j % bs] = torch.randn(hk, D, generator=g).to(dtype)
            v[table[b, j // bs], :, j % bs] = torch.randn(hk, D, generator=g).to(dtype)
    width = hq * D
    q = (torch.randn(T + spare_rows, width + stride_pad, generator=g) * q_scale).to(dtype)
    return {"q": q, "width": width, "k": k, "v": v, "table": table,
            "lens": torch.tensor([P + n for n in own], dtype=torch.int64),
            "starts": torch.tensor([0] + list(new), dtype=torch.int64).cumsum(0),
            "prefix": prefix, "P": P, "hq": hq, "hk": hk, "D": D, "bs": bs, "T": T, "scale": D ** -0.5}


def attend_reference(c):
    """(out, lse, out bound, lse bound) in float64, a row at a time where a row sees other keys."""
    hq, hk, D, bs, P = (c[x] for x in ("hq", "hk", "D", "bs", "P"))
    G, rows = hq // hk, c["q"].shape[0]
    dtype = c["q"].dtype
    uw = 0.0 if dtype == torch.float32 else half_step(dtype)
    out = torch.zeros(rows, hq, D, dtype=torch.float64)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(len(c["lens"])):
        t0, t1, n = int(c["starts"][b]), int(c["starts"][b + 1]), int(c["lens"][b])
        if t1 == t0:
            continue
        ks, vs = [], []
        for j in range(max(0, n)):
            page = int(c["prefix"][j // bs]) if j < P else (
                int(c["table"][b, (j - P) // bs]) if (j - P) // bs < c["table"].shape[1] else -1)
            if not 0 <= page < c["k"].shape[0]:
                ks.append(None)
                vs.append(None)
                continue
            r = j % bs if j < P else (j - P) % bs
            ks.append(c["k"][page, :, r].double())
            vs.append(c["v"][page, :, r].double())
        for t in range(t0, t1):
            seen = [j for j in range(n - (t1 - t) + 1) if ks[j] is not None]
            if not seen:
                continue
            k = torch.stack([ks[j] for j in seen])  # [n, hk, D]
            v = torch.stack([vs[j] for j in seen])
            q = c["q"][t, :c["width"]].double().reshape(hk, G, D)
            s = torch.einsum("kgd,nkd->kgn", q, k) * c["scale"]
            big = torch.einsum("kgd,nkd->kgn", q.abs(), k.abs()).amax(-1) * c["scale"]
            ls = torch.logsumexp(s, -1)
            w = torch.softmax(s, -1)
            o = torch.einsum("kgn,nkd->kgd", w, v)
            A = torch.einsum("kgn,nkd->kgd", w, v.abs())
            d = 2 * (D + 4) * E32 * big
            m = len(seen)
            out[t], lse[t] = o.reshape(hq, D), ls.reshape(hq)
            tol[t] = (half_step(dtype) * o.abs() + (uw + 2 * d[..., None] + (4 * m + 64) * E32) * A
                      + TINY[dtype]).reshape(hq, D)
            ltol[t] = (d + (m + 64) * E32 + 4 * E32 * ls.abs()).reshape(hq)
    return out.reshape(rows, -1), lse, tol.reshape(rows, -1), ltol


def run_attend(R, c, guards=None, lse=True, stream=None, prepared=False, **kw):
    """(out, lse) of the operator on guarded device copies; rows past the last token hold the
    canary pattern before the call."""
    from guard import Guards
    g = guards or Guards()
    q = g.put(c["q"], "q")[:, :c["width"]]
    rows = c["q"].shape[0]
    out = g.empty((rows, c["width"]), c["q"].dtype, "out")
    ls = g.empty((rows, c["hq"]), torch.float32, "lse") if lse else None
    call = R.prepare_paged_attention if prepared else R.paged_attention
    r = call(q, g.put(c["k"], "k"), g.put(c["v"], "v"), g.put(c["table"], "table"), g.put(c["lens"], "lens"),
             g.put(c["starts"], "starts"), out, scale=c["scale"],
             prefix_blocks=g.put(c["prefix"], "prefix") if c["P"] else None, prefix_len=c["P"], lse=ls, stream=stream,
             **kw)
    if prepared:
        r()
    g.check()
    return out.cpu(), None if ls is None else ls.cpu()


def widened(c):
    """The case with a block table of 200000 keys' pages, the added ones outside the cache: with more than 16 rows
    a key head, which kernel runs goes by how many keys there may be."""
    B, W = c["table"].shape
    more = max(0, -(-200000 // c["bs"]) - W)
    return dict(c, table=torch.cat([c["table"], torch.full((B, more), 1 << 40, dtype=torch.int64)], 1))


def check_attend(R, c, what="", **kw):
    """The case as it is and widened; (out, lse) of the first."""
    ro, rl, to, tl = attend_reference(c)
    T = int(c["starts"][-1])
    first = None
    for case in (c, widened(c)):
        out, lse = run_attend(R, case, **kw)
        assert_close(out[:T], ro[:T], to[:T], what + " out")
        if lse is not None:
            assert_close(lse[:T], rl[:T], tl[:T], what + " lse")
        canary = torch.full_like(out[T:].view(torch.int16), 0x7FA5)
        assert torch.equal(out[T:].view(torch.int16), canary), what + ": rows past the last token changed"
        assert R.get_device_error() == 0
        first = first or (out, lse)
        if c["T"] * (c["hq"] // c["hk"]) <= 16 * len(c["lens"]):
            break  # 16 rows at most: the same kernel
    return first


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def append_case(seed, dtype, T, hq, hk, D, R, bs, neox=True, sections=None, cache_mode=0, table_dtype=None,
                fused=False, hv=None, max_seq=97, pad_every=5, NB=None):
    g = torch.Generator().manual_seed(seed)
    hv = hk if hv is None else hv
    table_dtype = table_dtype or dtype
    if fused:
        buf = torch.randn(T, (hq + hk + hv) * D, generator=g).to(dtype)
        q, k, v = buf[:, :hq * D], buf[:, hq * D:(hq + hk) * D], buf[:, (hq + hk) * D:]
    else:
        q, k, v = (torch.randn(T, h * D, generator=g).to(dtype) for h in (hq, hk, hv))
    table = torch.randn(max_seq, R, generator=g).to(table_dtype)
    m = len(sections) if sections else 0
    pos = torch.randint(0, max_seq, (m, T) if m else (T,), generator=g)
    NB = NB or -(-T // bs) + 2
    slots = torch.randperm(NB * bs, generator=g)[:T]
    if pad_every:
        slots[pad_every - 1::pad_every] = -1
    return {"q": q, "k": k, "v": v, "table": table, "pos": pos, "slots": slots, "D": D, "R": R, "neox": neox,
            "sections": sections, "cache_mode": cache_mode, "hq": hq, "hk": hk, "hv": hv, "bs": bs,
            "kc": torch.randn(NB, hk, bs, D, generator=g).to(dtype),
            "vc": torch.randn(NB, hv, bs, D, generator=g).to(dtype), "dtype": dtype}


def append_reference(c):
    """(q, k_cache, v_cache) in float64, and the tokens skipped for their position."""
    T, D, R, bs, half = c["q"].shape[0], c["D"], c["R"], c["bs"], c["R"] // 2
    pos = c["pos"] if c["pos"].dim() == 2 else c["pos"][None]
    kc, vc = c["kc"].double().clone(), c["vc"].double().clone()
    q_out = torch.full((T, c["hq"] * D), math.nan, dtype=torch.float64)
    skipped = []
    for t in range(T):
        if bool(((pos[:, t] < 0) | (pos[:, t] >= c["table"].shape[0])).any()):
            skipped.append(t)
            continue
        rows = c["table"][pos[:, t]].double()
        cos, sin = torch.empty(half, dtype=torch.float64), torch.empty(half, dtype=torch.float64)
        for i in range(half):
            if not c["sections"]:
                r = 0
            elif c["cache_mode"] == 1:
                r = i % 3 if i < 3 * c["sections"][1] else 0
            else:
                r = [i < sum(c["sections"][:s + 1]) for s in range(len(c["sections"]))].index(True)
            cos[i], sin[i] = rows[r, i], rows[r, half + i]

        def rot(x):
            x = x.double().reshape(-1, D).clone()
            ia = torch.arange(half) if c["neox"] else 2 * torch.arange(half)
            ib = ia + (half if c["neox"] else 1)
            a, b = x[:, ia].clone(), x[:, ib].clone()
            x[:, ia], x[:, ib] = a * cos - b * sin, b * cos + a * sin
            return x

        q_out[t] = rot(c["q"][t]).reshape(-1)
        s = int(c["slots"][t])
        if 0 <= s < kc.shape[0] * bs:
            kc[s // bs, :, s % bs] = rot(c["k"][t])
            vc[s // bs, :, s % bs] = c["v"][t].double().reshape(-1, D)
    return q_out, kc, vc, skipped


def append_bound(ref, dtype):
    return (half_step(dtype) + 4 * E32) * ref.abs() + TINY[dtype]


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------
def table_reference(inv, scale, positions, layout):
    """(cos, sin) or the cache, in float64, and their bound per unit of the output's half step."""
    angle = positions.double()[:, None] * torch.as_tensor(inv, dtype=torch.float64)
    c, s = angle.cos() * scale, angle.sin() * scale
    slack = 2.0 ** -52 * angle.abs() * abs(scale)
    if layout == "cache":
        return torch.cat([c, s], 1), torch.cat([slack, slack], 1)
    if layout == "half":
        w = lambda x: torch.cat([x, x], 1)  # noqa: E731
    else:
        w = lambda x: x.repeat_interleave(2, 1)  # noqa: E731
    return w(c), w(s), w(slack)


def table_bound(ref, slack, dtype):
    return (half_step(dtype) + 4 * E32) * ref.abs() + slack + TINY[dtype]
