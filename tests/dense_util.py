"""Oracles in 64 bits for the dense attention entry points and the cache, and their error bounds.

Bound of an attention output. With weights w_j = p_j / l, values v_j, o = sum_j w_j v_j and
A = sum_j w_j |v_j| (both per column):
  * the output is rounded once: half a step, |o| eps / 2 of its type (and half the smallest
    subnormal of fp16);
  * each p_j is rounded to the product's 16-bit type before it meets v_j: eps / 2 relative, so
    at most A eps / 2 (bf16 2^-8, fp16 2^-11; 8-bit caches are multiplied in fp16). An fp16
    value below 2^-14 is off by at most 2^-25: at most 2^-25 sum_j |v_j|, since the largest p_j
    is at least 1 before normalisation (the reference maximum is the score of a key);
    with 8-bit values p_j carries the value's scale over a power of two c <= 2 max_j scale_j, so there
    it is 2^-25 c sum_j |code_j|;
  * the exponentials are within 7.5e-5 of 2^x (the bound of the library's exp2), in p_j and
    in l: 2 x 7.5e-5 A;
  * the logits: products of 16-bit values are exact in 32 bits, their sum of d terms in 32 bits
    is off by at most d 2^-23 T, T = max sum_e |q_e k_e| / sqrt(d) (the tensor core may truncate:
    a whole step); scaling and the subtraction of the maximum add 4 steps of a magnitude
    within 2 T log2(e). A logit off by x moves p_j by x relatively: 2 (d + 12) 2^-23 T A;
  * the sums over n keys in 32 bits: 2 n 2^-23 A at most; the joins of parts are among them.
"""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10}


def attend(q, k, v, limit, mult=None, codes=None, cmax=0.0, dtype=torch.bfloat16, ptype=None):
    """One head in 64 bits: rows q [R, d] that see the first limit[r] of the keys. Returns
    (o, bound); ``ptype`` is the type P is rounded to."""
    R, d = q.shape
    o = torch.zeros_like(q)
    A = torch.zeros_like(q)
    T = 0.0
    sub = torch.zeros(d, dtype=torch.float64, device=q.device)
    n = k.shape[0]
    if n:
        s = q @ k.t() / math.sqrt(d)
        T = float((q.abs() @ k.abs().t()).max()) / math.sqrt(d)
        seen = torch.arange(n, device=q.device)[None, :] < limit[:, None]
        s = torch.where(seen, s, torch.full_like(s, -math.inf))
        m = s.amax(1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
        l = p.sum(1, keepdim=True)
        w = p / torch.where(l == 0, torch.ones_like(l), l)
        o, A = w @ v, w @ v.abs()
        sub = 2.0 ** -25 * (v.abs().sum(0) if codes is None else 2 * cmax * codes.abs().sum(0))
    ptype = ptype or dtype
    bound = o.abs() * EPS[dtype] / 2 + A * (EPS[ptype] / 2 + 1.5e-4 + (2 * (d + 12) * T + 2 * n) * 2.0 ** -23)
    if ptype == torch.float16:
        bound = bound + sub
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25
    return o, bound


def check(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(err[bad].nan_to_num(nan=float("inf")).max()),
                           float(bound[bad].max()))


TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def quantise(x, kind):
    """Codes (as the values they stand for) and scales of rows x [..., d], in 64 bits."""
    x = x.double()
    top = TOP[kind]
    amax = x.abs().amax(-1, keepdim=True)
    scale = (amax / top).float()
    y = torch.where(amax > 0, x * top / torch.where(amax > 0, amax, torch.ones_like(amax)), torch.zeros_like(x))
    if kind == torch.int8:
        return torch.round(y), scale[..., 0]
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448, 448), scale[..., 0]


def make_cache(gen, lens, Hkv, page, d, dtype, kind, spare=3, mul=1.0, device="cuda"):
    """Pages in a random order, a table with -1 behind every sequence's last page, and garbage
    (NaN, or codes with NaN scales) wherever no sequence's token lives."""
    need = [-(-max(x, 0) // page) for x in lens]
    pool, width = sum(need) + spare, max([1] + need)
    perm = torch.randperm(pool, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=device)
    at = 0
    for b, x in enumerate(need):
        table[b, :x] = perm[at:at + x]
        at += x
    live = torch.zeros(pool, page, dtype=torch.bool, device=device)
    for b, L in enumerate(lens):
        pos = torch.arange(L, device=device)
        live[table[b].long()[pos // page], pos % page] = True
    out = []
    for _ in range(2):
        x = torch.randn(pool, Hkv, page, d, generator=gen, device=device) * mul
        dead = ~live[:, None, :].expand(pool, Hkv, page)
        if kind is None:
            x = x.to(dtype)
            x[dead] = float("nan")
            out.append((x, None))
        else:
            codes, scale = quantise(x.to(dtype), kind)
            codes = codes.float().to(kind) if kind != torch.int8 else codes.to(torch.int8)
            scale[dead] = float("nan")
            out.append((codes, scale.contiguous()))
    (k, ks), (v, vs) = out
    return k, v, ks, vs, table


def cached(pages, scale, table, page, L):
    """A sequence's rows [Hkv, L, d] in 64 bits, its codes, and its largest scale."""
    pos = torch.arange(L, device=pages.device)
    at = table.long()[pos // page]
    x = pages.view(torch.uint8).view(*pages.shape[:-1], -1)[at, :, pos % page].contiguous().view(pages.dtype).double().transpose(0, 1)
    if scale is None:
        return x, None, 0.0
    s = scale[at, :, pos % page].double().transpose(0, 1)
    return x * s[..., None], x, float(s.abs().max()) if L else 0.0


def paged_oracle(q, k, v, ks, vs, table, ns, lens, causal, dtype):
    """(o, bound) [total, H, d] of solattn_paged_forward."""
    total, H, d = q.shape
    Hkv, page = k.shape[1], k.shape[2]
    G = H // Hkv
    o = torch.zeros(total, H, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    t0 = 0
    for b, (n, L) in enumerate(zip(ns, lens)):
        if n:
            kk, _, _ = cached(k, ks, table[b], page, L)
            vv, codes, cmax = cached(v, vs, table[b], page, L)
            i = torch.arange(n, device=q.device)
            limit = L - n + i + 1 if causal else torch.full_like(i, L)
            for h in range(H):
                o[t0:t0 + n, h], bound[t0:t0 + n, h] = attend(
                    q[t0:t0 + n, h].double(), kk[h // G], vv[h // G], limit, codes=None if codes is None else codes[h // G],
                    cmax=cmax, dtype=dtype, ptype=torch.float16 if ks is not None else dtype)
        t0 += n
    return o, bound


def cross_oracle(q, k, v, lens, dtype):
    B, H, Nq, d = q.shape
    G = H // k.shape[1]
    o = torch.zeros(B, H, Nq, d, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    for b in range(B):
        L = k.shape[2] if lens is None else lens[b]
        for h in range(H):
            limit = torch.full((Nq,), L, device=q.device)
            o[b, h], bound[b, h] = attend(q[b, h].double(), k[b, h // G, :L].double(), v[b, h // G, :L].double(), limit, dtype=dtype)
    return o, bound


def cu_of(ns, device="cuda"):
    c = [0]
    for x in ns:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device=device)


def ints(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)
