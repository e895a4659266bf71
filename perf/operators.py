"""Cases for measuring the dense attention family that stands beside the Sol-Attn operator:

* cross   attention of a diffusion transformer's tokens to an encoder's states of another length
          (text or image conditioning, padded to the batch's longest prompt);
* chunk   attention of a chunk of new tokens (a video frame, a prompt, one token) over a paged
          key/value cache, in 16 bits or quantised to 8;
* cache   new keys and values quantised into the pages as they are written, and read back;
* read    a long quantised cache read back into 16-bit keys and values.

``run`` computes them in plain torch, in 32 bits, or (``own``) through the library's entry points.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
# Largest code of a quantised row: the row's largest magnitude is mapped onto it.
TOP = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ cases

def cross_case(name, dtype, B, H, Hkv, Nq, Nk, d, ragged, layout):
    return {"name": name, "op": "cross", "dtype": dtype, "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d,
            "ragged": ragged, "layout": layout, "plan": 3}


def chunk_case(name, dtype, kind, B, H, Hkv, d, page, causal, n, L):
    return {"name": name, "op": "chunk", "dtype": dtype, "kind": kind, "B": B, "H": H, "Hkv": Hkv, "d": d, "page": page,
            "causal": causal, "n_lo": n[0], "n_hi": n[1], "L_lo": L[0], "L_hi": L[1], "plan": 3}


def cache_case(name, op, dtype, kind, B, Hkv, d, page, n, L):
    return {"name": name, "op": op, "dtype": dtype, "kind": kind, "B": B, "H": Hkv, "Hkv": Hkv, "d": d, "page": page,
            "causal": False, "n_lo": n[0], "n_hi": n[1], "L_lo": L[0], "L_hi": L[1], "plan": 3}


def listed():
    return [
        # the tiny configuration's tokens against a short caption: one launch, latency counts
        cross_case("cross_tiny", "fp16", 1, 2, 2, 1024, 77, 64, False, "bhnd"),
        # image DiT, a batch of prompts padded to 256, heads as a projection leaves them ([B][N][H][d])
        cross_case("cross_image_padded", "bf16", 8, 16, 16, 4096, 256, 128, True, "bnhd"),
        # 480p video tokens against 512 text states
        cross_case("cross_video480", "bf16", 1, 12, 12, 32760, 512, 128, False, "bhnd"),
        # 720p video tokens against 512 text and 257 image states: an odd length
        cross_case("cross_video720", "bf16", 1, 24, 24, 75600, 769, 128, False, "bhnd"),
        # streaming 480p generation: one latent frame (30 x 52 tokens) against all 21 frames in the cache
        chunk_case("chunk_frame", "bf16", "16", 1, 12, 12, 128, 128, False, (1560, 1560), (32760, 32760)),
        # the same with the cache in 8-bit integers
        chunk_case("chunk_frame_int8", "bf16", "int8", 1, 12, 12, 128, 64, False, (1560, 1560), (32760, 32760)),
        # a batch of prompts of unequal length behind shared prefixes, causal, shared key heads
        chunk_case("chunk_prompts", "fp16", "16", 8, 16, 4, 128, 16, True, (1, 2048), (1, 4096)),
        # single tokens of a batch of sequences of unequal length
        chunk_case("token_batch", "bf16", "16", 32, 16, 4, 128, 64, True, (1, 1), (1, 16384)),
        # one token against a long cache in e4m3 (the long video's length)
        chunk_case("token_long_e4m3", "bf16", "e4m3", 1, 24, 24, 128, 128, True, (1, 1), (118800, 118800)),
        # one new token of each sequence of a batch: latency
        cache_case("cache_tokens", "cache", "bf16", "e4m3", 32, 4, 128, 64, (1, 1), (1, 16384)),
        # one latent frame written and read back
        cache_case("cache_frame", "cache", "bf16", "int8", 1, 12, 128, 64, (1560, 1560), (32760, 32760)),
        # a whole 720p cache read back
        cache_case("cache_read_long", "read", "bf16", "e4m3", 1, 24, 128, 128, (75600, 75600), (75600, 75600)),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype, d = rng.choice(["bf16", "fp16"]), rng.choice([64, 128])
    G = rng.choice([1, 1, 2, 3, 4, 8])
    page, kind = rng.choice([16, 32, 64, 128]), rng.choice(["16", "int8", "e4m3"])
    op = rng.choice(["cross", "cross", "chunk", "chunk", "token", "cache", "read"])
    plan = rng.randrange(1 << 20)
    if op == "cross":
        Hkv, B = rng.randint(1, 12), rng.randint(1, 8)
        c = cross_case("", dtype, B, Hkv * G, Hkv, _log(rng, 1, 40000), _log(rng, 1, 4096), d, rng.random() < 0.5,
                       rng.choice(["bhnd", "bnhd"]))
        while 4.0 * c["B"] * c["H"] * c["Nq"] * c["Nk"] * d > 4e11:
            c["Nq"] = max(1, c["Nq"] * 2 // 3)
    elif op in ("chunk", "token"):
        Hkv, B = rng.randint(1, 8), rng.randint(1, 16)
        hi, L = (1, _log(rng, 1, 60000)) if op == "token" else (_log(rng, 2, 3000), _log(rng, 64, 30000))
        while B > 1 and (4.0 * B * Hkv * G * hi * L * d > 2e11 or B * Hkv * L * d > 3e8):
            B -= 1
        while 4.0 * Hkv * G * hi * L * d > 2e11 or Hkv * L * d > 3e8:
            L = max(1, L * 2 // 3)
        c = chunk_case("", dtype, kind, B, Hkv * G, Hkv, d, page, rng.random() < 0.5, (max(1, hi // 3), hi),
                       (max(1, L // 3), L))
    else:
        Hkv, B = rng.randint(1, 24), rng.randint(1, 16)
        L = _log(rng, 1, 60000)
        while B * Hkv * L * d > 2e8:
            L = max(1, L * 2 // 3)
        hi = L if op == "read" else _log(rng, 1, L)
        c = cache_case("", op, dtype, kind if kind != "16" else "int8", B, Hkv, d, page, (max(1, hi // 2), hi),
                       (max(1, L // 2), L))
    c["plan"] = plan
    del c["name"]
    return c


def plan(case):
    """Lengths of the batch's sequences: those of a serving step, which the case fixes."""
    rng = random.Random(case["plan"])
    if case["op"] == "cross":
        if not case["ragged"]:
            return [case["Nk"]] * case["B"]
        lens = [rng.randint(0, case["Nk"]) for _ in range(case["B"])]
        lens[rng.randrange(case["B"])] = case["Nk"]
        return lens
    n = [rng.randint(case["n_lo"], case["n_hi"]) for _ in range(case["B"])]
    return [(x, max(x, rng.randint(case["L_lo"], case["L_hi"]))) for x in n]


def pairs(case, n, L):
    """(query, key) pairs of a chunk of n tokens that ends a sequence of L."""
    return n * L - (n * (n - 1) // 2 if case["causal"] else 0)


def work(case):
    d, H, Hkv, B = case["d"], case["H"], case["Hkv"], case["B"]
    if case["op"] == "cross":
        lens = plan(case)
        kv = sum(lens) * Hkv * d * 2 * 2
        return {"bytes": 2 * B * H * case["Nq"] * d * 2 + kv, "flops": 4.0 * H * case["Nq"] * d * sum(lens)}
    p = plan(case)
    row = 2 * (d * 2 if case["kind"] == "16" else d + 4)  # one cached token of one head, keys and values
    if case["op"] == "chunk":
        new, old = sum(n for n, _ in p), sum(L for _, L in p)
        return {"bytes": 2 * new * H * d * 2 + old * Hkv * row, "flops": 4.0 * H * d * sum(pairs(case, n, L) for n, L in p)}
    new = sum(n for n, _ in p) * Hkv
    if case["op"] == "cache":
        return {"bytes": new * (2 * row + 2 * 2 * d * 2), "flops": 2.0 * new * 2 * d}
    return {"bytes": new * (row + 2 * d * 2), "flops": 2.0 * new * d}


# ------------------------------------------------------------------ inputs

def _codes(x, kind, dtype):
    """Rows of x [.., d] as a user's pages hold them: (pages, scales)."""
    if kind == "16":
        return x.to(dtype), None
    s = x.abs().amax(-1) / TOP[kind]
    y = x / s.clamp_min(1e-30)[..., None]
    return (y.round().clamp(-127, 127).to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, d, B, H, Hkv = DT[case["dtype"]], case["d"], case["B"], case["H"], case["Hkv"]

    def normal(*shape, mul=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * mul)

    st = {"case": case, "dtype": dtype}
    if case["op"] == "cross":
        def heads(n, h, mul=1.0):  # [B][h][n][d], or the same as a view of [B][n][h][d]
            x = normal(B, n, h, d, mul=mul).to(dtype)
            return x.transpose(1, 2) if case["layout"] == "bnhd" else x.transpose(1, 2).contiguous()
        st.update(q=heads(case["Nq"], H, 2.0), k=heads(case["Nk"], Hkv), v=heads(case["Nk"], Hkv))
        st["out"] = torch.empty_like(st["q"])
        st["len"] = torch.tensor(plan(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        return st
    p, page = plan(case), case["page"]
    n, L = [x[0] for x in p], [x[1] for x in p]
    width = max(-(-x // page) for x in L)
    need = [-(-x // page) for x in L]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")  # -1: no page
    owned = torch.arange(width, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[owned] = order[:sum(need)]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    st.update(table=table, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_n=max(n), total=cu[-1],
              len=torch.tensor(L, dtype=torch.int32, device="cuda"))
    st["k_pages"], st["k_scale"] = _codes(normal(pool, Hkv, page, d), case["kind"], dtype)
    st["v_pages"], st["v_scale"] = _codes(normal(pool, Hkv, page, d), case["kind"], dtype)
    if case["op"] == "chunk":
        st["q"] = normal(cu[-1], H, d, mul=2.0).to(dtype)
        st["out"] = torch.empty_like(st["q"])
    else:
        st["new_k"] = normal(cu[-1], Hkv, d).to(dtype)
        st["new_v"] = normal(cu[-1], Hkv, d, mul=0.5).to(dtype)
        st["out_k"], st["out_v"] = torch.empty_like(st["new_k"]), torch.empty_like(st["new_v"])
    return st


# ------------------------------------------------------------------ plain forms

def _attend(q, k, v, seen, scale):
    """softmax(q k^T scale) v over the keys that `seen` leaves, zero where it leaves none."""
    s = torch.matmul(q, k.transpose(-1, -2)) * scale
    s = s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = s.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    l = e.sum(-1, keepdim=True)
    return torch.matmul(e, v) / l.masked_fill(l == 0, 1.0)


def _plain_cross(st):
    c, q, k, v = st["case"], st["q"], st["k"], st["v"]
    B, H, Hkv, Nq, Nk, d = c["B"], c["H"], c["Hkv"], c["Nq"], c["Nk"], c["d"]
    lens = st["len"] if st["len"] is not None else torch.full((B,), Nk, dtype=torch.int32, device=q.device)
    seen = (torch.arange(Nk, device=q.device)[None, :] < lens[:, None])[:, None, None, :]
    o = _attend(q.float().reshape(B, Hkv, -1, d), k.float(), v.float(), seen, 1.0 / math.sqrt(d))
    return o.reshape(B, H, Nq, d).to(st["dtype"])


def _places(st):
    """Of each new token: its sequence, its position there, its page and its row in the page."""
    cu, t = st["cu"].long(), torch.arange(st["total"], device=st["cu"].device)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    pos = st["len"].long()[b] - (cu[b + 1] - t)
    page = st["case"]["page"]
    return b, pos, st["table"].long()[b, pos // page], pos % page


def _gathered(st, which):
    """A sequence's cached rows in order: [B][Hkv][positions][d] in 32 bits."""
    pages, scale = st[which + "_pages"], st[which + "_scale"]
    at = st["table"].long().clamp_min(0)
    x = pages[at].float() if scale is None else pages[at].float() * scale[at][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_chunk(st):
    c = st["case"]
    H, Hkv, d, B, n = c["H"], c["Hkv"], c["d"], c["B"], st["max_n"]
    k, v = _gathered(st, "k"), _gathered(st, "v")
    b, pos, _, _ = _places(st)
    first = st["len"].long() - (st["cu"][1:] - st["cu"][:-1]).long()
    q = torch.zeros(B, n, H, d, device=k.device)
    q[b, pos - first[b]] = st["q"].float()
    q = q.reshape(B, n, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    at = torch.arange(k.shape[2], device=k.device)
    seen = (at[None, :] < st["len"].long()[:, None])[:, None, :]
    if c["causal"]:
        seen = seen & (at[None, None, :] <= (first[:, None] + torch.arange(n, device=k.device)[None, :])[:, :, None])
    seen = seen.expand(B, n, -1)[:, None].expand(B, H // Hkv, n, -1).reshape(B, 1, -1, k.shape[2])
    o = _attend(q, k, v, seen, 1.0 / math.sqrt(d))
    o = o.reshape(B, Hkv, H // Hkv, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, H, d)
    return o[b, pos - first[b]].to(st["dtype"])


def _write(st, which, at, row):
    # A code is the nearest to x top / amax, the exact ratio: in 64 bits, since ratios lie on the border of two codes.
    x = st["new_" + which].double()
    top = TOP[st["case"]["kind"]]
    amax = x.abs().amax(-1)
    s = (amax / top).float()
    y = x * top / amax.masked_fill(amax == 0, 1.0)[..., None]
    pages = st[which + "_pages"]
    if st["case"]["kind"] == "int8":
        pages[at, :, row] = y.round().clamp(-127, 127).to(torch.int8)
    else:
        pages.view(torch.uint8)[at, :, row] = y.clamp(-top, top).to(torch.float8_e4m3fn).view(torch.uint8)
    st[which + "_scale"][at, :, row] = s


def _read(st, which, at, row):
    codes = st[which + "_pages"].view(torch.uint8)[at, :, row].view(st[which + "_pages"].dtype)
    return (codes.float() * st[which + "_scale"][at, :, row][..., None]).to(st["dtype"])


def _plain_cache(st):
    _, _, at, row = _places(st)
    if st["case"]["op"] == "cache":
        _write(st, "k", at, row)
        _write(st, "v", at, row)
    return _read(st, "k", at, row), _read(st, "v", at, row)


# ------------------------------------------------------------------ one pass

def _lib():
    from block_sparse_online_b200 import solattn
    return solattn


def _own(st):
    lib, c = _lib(), st["case"]
    if c["op"] == "cross":
        if "ws" not in st:
            st["ws"] = lib.alloc_cross_workspace(c["B"], c["H"], c["Hkv"], c["Nq"], c["Nk"], c["d"], st["q"].device)
        return lib.solattn_cross(st["q"], st["k"], st["v"], key_len=st["len"], out=st["out"], workspace=st["ws"])
    if "cache" not in st:  # the handle over the pages that a serving program keeps
        st["cache"] = lib.PagedCache(st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"])
        if c["op"] == "chunk":
            st["ws"] = lib.alloc_paged_workspace(st["cache"], c["B"], c["H"], st["total"], st["q"].device)
        else:
            st["ws"] = lib.alloc_status(st["table"].device)
    args = (st["table"], st["cu"], st["len"])
    if c["op"] == "chunk":
        return lib.solattn_paged_forward(st["q"], st["cache"], *args, max_new=st["max_n"], causal=c["causal"],
                                         out=st["out"], workspace=st["ws"])
    if c["op"] == "cache":
        lib.solattn_cache_append(st["cache"], st["new_k"], st["new_v"], *args, workspace=st["ws"])
    return lib.solattn_cache_read(st["cache"], *args, k_out=st["out_k"], v_out=st["out_v"], workspace=st["ws"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_cross(state) if op == "cross" else _plain_chunk(state) if op == "chunk" else _plain_cache(state)


# ------------------------------------------------------------------ the definition in 64 bits

def _softmax_rows(q, k, v, limit):
    """One sequence and one key head: rows q [R][d] that see the first limit[r] keys."""
    out = torch.zeros_like(q)
    for i in range(0, q.shape[0], 4096):
        lim = limit[i:i + 4096, None]
        s = (q[i:i + 4096] @ k.t()) / math.sqrt(q.shape[1])
        hidden = torch.arange(k.shape[0], device=q.device)[None, :] >= lim
        w = torch.softmax(torch.where(hidden, torch.full_like(s, -1e300), s), 1)
        out[i:i + 4096] = torch.where(lim > 0, torch.where(hidden, torch.zeros_like(w), w) @ v, torch.zeros_like(q[i:i + 4096]))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    c, G = case, case["H"] // case["Hkv"]
    if c["op"] == "cross":
        out = torch.zeros(c["B"], c["H"], c["Nq"], c["d"], dtype=torch.float64, device="cuda")
        for b, m in enumerate(plan(c)):
            for h in range(c["H"] if m else 0):
                k, v = st["k"][b, h // G, :m].double(), st["v"][b, h // G, :m].double()
                limit = torch.full((c["Nq"],), m, device="cuda")
                out[b, h] = _softmax_rows(st["q"][b, h].double(), k, v, limit)
        return out

    def rows(which, b, first, last):
        """Positions first .. last - 1 of sequence b from the pages, [Hkv][rows][d]."""
        pos = torch.arange(first, last, device="cuda")
        at, row = st["table"][b].long()[pos // c["page"]], pos % c["page"]
        pages, scale = st[which + "_pages"], st[which + "_scale"]
        x = pages.view(torch.uint8)[at, :, row].view(pages.dtype) if scale is not None else pages[at, :, row]
        x = x.double()
        return (x if scale is None else x * scale[at, :, row].double()[..., None]).transpose(0, 1)

    p, cu = plan(c), st["cu"].tolist()
    if c["op"] == "chunk":
        out = torch.zeros(st["total"], c["H"], c["d"], dtype=torch.float64, device="cuda")
        for b, (n, L) in enumerate(p):
            k, v = rows("k", b, 0, L), rows("v", b, 0, L)
            i = torch.arange(n, device="cuda")
            limit = L - n + i + 1 if c["causal"] else torch.full_like(i, L)
            for h in range(c["H"]):
                out[cu[b]:cu[b + 1], h] = _softmax_rows(st["q"][cu[b]:cu[b + 1], h].double(), k[h // G], v[h // G], limit)
        return out
    if c["op"] == "read":
        return tuple(torch.cat([rows(w, b, L - n, L) for b, (n, L) in enumerate(p)], 1).transpose(0, 1) for w in ("k", "v"))
    back = []
    for w in ("k", "v"):
        x = st["new_" + w].double()
        # the scale is part of the cache's format: the 32-bit quotient nearest to amax / top
        # and a code is the one nearest to the exact ratio x top / amax, ties to the even one
        amax = x.abs().amax(-1, keepdim=True)
        s = (amax / TOP[c["kind"]]).float().double()  # [..][1]
        y = torch.where(amax > 0, x * TOP[c["kind"]] / torch.where(amax > 0, amax, torch.ones_like(amax)), torch.zeros_like(x))
        if c["kind"] == "int8":
            y = torch.round(y).clamp(-127, 127)
        else:  # nearest value of 1.mmm * 2^e, e >= -6, ties to the even step
            e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))).clamp(-6, 8)
            y = (torch.round(y / torch.exp2(e - 3)) * torch.exp2(e - 3)).clamp(-448, 448)
        back.append(y * s)
    return tuple(back)
