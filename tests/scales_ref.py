"""A float64 reference of the attention over a cache of 8-bit codes, whatever its scales are, with error bounds.

Bounds, beside those of tests/serving_ref.py: a weight w, relative to the row's largest, of a key whose V scale is 2^-n of
the largest that its kernel has seen is rounded in binary16 with V's scale in it.  Units of 8 and 16 rows take that 2^15 times
as large: half a step of it, or 2^-25 / 2^15 * 2^n = 2^(n - 40), n at most 15 (else the row is computed key by key, or the weight is
at most 2^-30).  Tall units 2^11 times: 2^(n - 36), n at most 10.  So 2^-25 at most; and never more than w, since 0 is a
binary16 value.  With W the row's largest weight:  out: + W sum_j min(w_j / W, 2^-25) |v_j|.
"""
import math

import torch

import transformer_rope_positional_gb300 as R
from codes_ref import bytes_of, run_coded, values_of
from serving_ref import E32, TINY, assert_close, half_step, widened


def place(c, b, j):
    """(page, row) of key j of sequence b."""
    bs, P = c["bs"], c["P"]
    return (int(c["prefix"][j // bs]), j % bs) if j < P else (int(c["table"][b, (j - P) // bs]), (j - P) % bs)


def put(c, name, j, byte=None, code=None, b=None):
    """The scale byte and the codes of key j of every sequence (that has it), or of sequence b."""
    for i in range(len(c["lens"])) if b is None else [b]:
        if j < int(c["lens"][i]):
            page, row = place(c, i, j)
            if byte is not None:
                bytes_of(c[name + "_scale"])[page, :, row] = byte
            if code is not None:
                bytes_of(c[name + "_codes"])[page, :, row] = code


def put_bytes(c, name, bytes_):
    """The scale byte of key j of every sequence (that has it): bytes_[j]."""
    for b, n in enumerate(c["lens"].tolist()):
        n = min(n, len(bytes_))
        page, row = torch.tensor([place(c, b, j) for j in range(n)]).unbind(1)
        bytes_of(c[name + "_scale"])[page, :, row] = torch.as_tensor(bytes_[:n]).to(torch.uint8)[:, None]


def reference(c):
    hq, hk, D = c["hq"], c["hk"], c["D"]
    G, rows, dtype = hq // hk, c["q"].shape[0], c["q"].dtype
    where = "cuda" if torch.cuda.is_available() else "cpu"  # (plain operations in 64 bits: quicker there)
    K, V = (values_of(c[n + "_codes"], c[n + "_scale"]).to(where) for n in ("k", "v"))
    out = torch.zeros(rows, hq, D, dtype=torch.float64, device=where)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=where)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    uw = 0.0 if dtype == torch.float32 else half_step(dtype)
    for b in range(len(c["lens"])):
        t0, t1, n = int(c["starts"][b]), int(c["starts"][b + 1]), int(c["lens"][b])
        if t1 == t0 or n <= 0:
            continue
        page, row = torch.tensor([place(c, b, j) for j in range(n)], device=where).unbind(1)
        k, v = (x[page, :, row].transpose(0, 1) for x in (K, V))  # [hk, n, D]
        q = c["q"][t0:t1, :c["width"]].to(where).double().reshape(t1 - t0, hk, G, D)
        s = torch.einsum("tkgd,knd->tkgn", q, k) * c["scale"]
        big = torch.einsum("tkgd,knd->tkgn", q.abs(), k.abs()) * c["scale"]
        seen = (torch.arange(n)[None] < (n - (t1 - torch.arange(t0, t1)) + 1)[:, None]).to(where)  # [t, n]
        s = s.masked_fill(~seen[:, None, None], -math.inf)
        big = big.masked_fill(~seen[:, None, None], 0.0).amax(-1)
        w = torch.softmax(s, -1).masked_fill(~seen[:, None, None], 0.0)
        ls = torch.logsumexp(s, -1)
        finite = torch.nan_to_num(v, nan=0.0)
        o = torch.einsum("tkgn,knd->tkgd", w, finite)
        bad = torch.einsum("tn,knd->tkd", seen.double(), torch.isnan(v).double()) > 0
        o = torch.where(bad[:, :, None], torch.nan, o)
        A = torch.einsum("tkgn,knd->tkgd", w, finite.abs())
        top = w.amax(-1, keepdim=True)
        low = torch.einsum("tkgn,knd->tkgd", torch.minimum(w, top * 2.0 ** -25), finite.abs())
        d = 2 * (D + 4) * E32 * big
        out[t0:t1], lse[t0:t1] = o.reshape(-1, hq, D), ls.reshape(-1, hq)
        tol[t0:t1] = (half_step(dtype) * o.abs() + (uw + 2 * d[..., None] + (4 * n + 64) * E32) * A + low
                      + TINY[dtype]).reshape(-1, hq, D)
        ltol[t0:t1] = (d + (n + 64) * E32 + 4 * E32 * ls.abs()).reshape(-1, hq)
    return tuple(x.cpu() for x in (out.reshape(rows, -1), lse, tol.reshape(rows, -1), ltol))


def run(c):
    out, lse = run_coded(R, widened(c) if c.get("wide") else c)
    assert R.get_device_error() == 0
    return out, lse


def check(c, what=""):
    ro, rl, to, tl = reference(c)
    out, lse = run(c)
    assert_close(out, ro, to, what + " out")
    assert_close(lse, rl, tl, what + " lse")
    return out, lse
