"""Measured cases of the 8-bit paged cache and of the rotary positions: their plain forms, the
calls a program makes of this package, and their values in 64 bits.

Four operators. ``rope`` turns the queries and keys of packed tokens by their positions (and,
backward, their gradients back). ``write`` quantises the keys and values of new tokens into a paged
cache of 8-bit codes with one scale for every ``G`` consecutive tokens of a head, and reads the
touched groups back (what is held in 8 bits is compared as the values it stands for). ``read``
gathers a cache's tokens as packed rows. ``attn`` is attention of packed queries over that cache.

A cache: codes [pages, page_size, Hkv, D] (int8 or float8_e4m3fn), scales float32 [pages, Hkv,
page_size / G]. Token j of sequence s is row j % page_size of page table[s][j // page_size].
"""
import math

import numpy as np
import torch

own = False  # False: the plain forms below; True: the package's kernels

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
FLOOR = 2.0 ** -100  # the smallest scale


# ----------------------------------------------------------------------------- cases
def _rope(name, tokens, hq, hk, d, rot, layout, dtype, top, scaling, back=False):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rot, "layout": layout,
            "dtype": dtype, "top": top, "scaling": scaling, "back": back}


def _cache(name, op, dtype, code, seqs, hq, hkv, d, page, g, ctx_lo, ctx_hi, q_lo, q_hi, meta, causal=True):
    return {"name": name, "op": op, "dtype": dtype, "code": code, "seqs": seqs, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "g": g, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "q_lo": q_lo, "q_hi": q_hi, "meta": meta,
            "causal": causal}


def listed():
    return [
        # one serving step of 64 sequences, 32 query and 8 key heads (the repository's paged decode workload)
        _rope("rope_step", 64, 32, 8, 128, 128, "half", "bf16", 8192, "none"),
        # a long document: half of each head turned, neighbouring pairs, frequencies scaled by parts
        _rope("rope_long_f16", 8191, 32, 8, 128, 64, "interleaved", "f16", 1 << 20, "by_parts"),
        # the gradient of a training batch of 4 x 4096 tokens (the repository's causal 4k workload)
        _rope("rope_grad_f32", 16384, 32, 32, 128, 128, "half", "f32", 4096, "none", True),
        # the same serving step appends one token to each of 64 sequences, part-filled groups of 16
        _cache("write_step_int8", "write", "bf16", "int8", 64, 32, 8, 128, 64, 16, 1024, 8192, 1, 1, 20),
        # prompts of 500 to 2000 tokens enter the cache, one scale for a page of 64
        _cache("write_prompts_e4m3", "write", "f16", "e4m3", 32, 32, 8, 128, 64, 64, 500, 2000, 500, 2000, 21),
        # a few short prefixes come back for a dense pass
        _cache("read_prefix_int8", "read", "bf16", "int8", 3, 8, 2, 64, 16, 1, 37, 300, 0, 0, 22),
        # every sequence of the serving step leaves the cache (a change of format)
        _cache("read_all_e4m3", "read", "f32", "e4m3", 64, 32, 8, 128, 64, 16, 1024, 8192, 0, 0, 20),
        # one chat just begun: latency
        _cache("attn_first_f16", "attn", "f16", "int8", 1, 8, 2, 64, 16, 1, 201, 201, 1, 1, 23),
        # the repository's paged decode workload on an 8-bit cache
        _cache("attn_step_bf16", "attn", "bf16", "e4m3", 64, 32, 8, 128, 64, 64, 1024, 8192, 1, 1, 20),
        # 5 drafted tokens of 12 sequences are scored at once, groups of 7 heads
        _cache("attn_drafts_f16", "attn", "f16", "int8", 12, 28, 4, 128, 32, 16, 3000, 16000, 5, 5, 24),
        # one question to a long document
        _cache("attn_document_bf16", "attn", "bf16", "int8", 1, 32, 8, 128, 128, 32, 130001, 130001, 1, 1, 25),
        # the repository's chunked prefill workload on an 8-bit cache
        _cache("attn_prefill_bf16", "attn", "bf16", "e4m3", 16, 32, 8, 128, 64, 16, 512, 4096, 128, 512, 21),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "write", "read", "attn", "attn"))
    dtype = rng.choice(("bf16", "f16"))
    if op == "rope":
        d = rng.choice((64, 128))
        return {k: v for k, v in _rope("", _log(rng, 1, 12000), rng.choice((8, 14, 32)), rng.choice((1, 2, 8)), d,
                                       rng.choice((d, d // 2, d // 4 * 3)), rng.choice(("half", "interleaved")),
                                       rng.choice(("f32", "f16", "bf16")), _log(rng, 512, 1 << 20),
                                       rng.choice(("none", "linear", "ntk", "by_parts")),
                                       rng.choice((False, True))).items() if k != "name"}
    page = rng.choice((16, 32, 64, 128))
    g = rng.choice((1, 8, 16, page))
    hkv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 3, 4, 7, 8))
    d = rng.choice((64, 128))
    code = rng.choice(("int8", "e4m3"))
    seqs = _log(rng, 1, 48)
    hi = _log(rng, 33, 8000)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    if op == "attn" and rng.random() < 0.4:  # a chunk of a prompt
        seqs, hi = _log(rng, 1, 12), _log(rng, 65, 4000)
        lo = max(64, int(hi * rng.uniform(0.3, 1.0)))
        q_hi = min(lo, _log(rng, 16, 480))
        q_lo = max(1, int(q_hi * rng.uniform(0.3, 1.0)))
        group = rng.choice((1, 4, 7, 8)) if hkv < 8 else rng.choice((1, 4))
    elif op == "write":
        q_hi = min(hi, _log(rng, 1, 1500))
        q_lo = max(1, int(q_hi * rng.uniform(0.3, 1.0)))
    else:
        q_lo = q_hi = rng.choice((1, 1, 1, 2, 4))
    c = _cache("", op, dtype, code, seqs, hkv * group, hkv, d, page, g, lo, hi, q_lo, q_hi, rng.randrange(1 << 20),
               rng.random() < 0.8)
    return {k: v for k, v in c.items() if k != "name"}


# ----------------------------------------------------------------------------- inputs
def _frequencies(c):
    """float64 [rot / 2] angular frequencies and the factor on cos and sin."""
    rot, i = c["rot"], np.arange(0, c["rot"], 2, dtype=np.float64)
    base, f = 10000.0, 8.0
    if c["scaling"] == "ntk":
        base *= f ** (rot / (rot - 2.0))
    w = base ** (-i / rot)
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "by_parts":  # fast turns stay, slow ones are divided, between 1 and 32 turns a ramp
        turns = 4096 * w / (2 * math.pi)
        keep = np.clip((turns - 1.0) / 31.0, 0.0, 1.0)
        w = w * keep + w / f * (1.0 - keep)
        return w, 0.1 * math.log(f) + 1.0
    return w, 1.0


def _lengths(c):
    """Tokens and new tokens of each sequence: by the case alone, so that work() knows them."""
    r = np.random.RandomState(c["meta"])
    lens = r.randint(c["ctx_lo"], c["ctx_hi"] + 1, c["seqs"])
    new = np.minimum(lens, r.randint(c["q_lo"], c["q_hi"] + 1, c["seqs"]))
    if c["op"] == "write" and c["ctx_lo"] == c["q_lo"] and c["q_hi"] == c["ctx_hi"]:
        new = lens.copy()  # whole prompts
    return lens, new


def _normal(gen, shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _rows(gen, n, heads, d, dtype):
    """Keys or values as a model makes them: some channels and some tokens larger than the rest."""
    channel = 1.0 + 3.0 * (torch.rand((heads, d), generator=gen, device="cuda") < 0.05).float()
    token = torch.exp(0.4 * _normal(gen, (n, heads, 1)))
    return (_normal(gen, (n, heads, d)) * channel * token).to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[c["dtype"]]
    if c["op"] == "rope":
        # q and k lie side by side, with the values, in one projection's output
        x = _rows(gen, c["tokens"], c["hq"] + 2 * c["hk"], c["d"], dt)
        q, k = x[:, :c["hq"]], x[:, c["hq"]:c["hq"] + c["hk"]]
        w, m = _frequencies(c)
        pos = torch.randint(0, c["top"], (c["tokens"],), generator=gen, device="cuda", dtype=torch.int32)
        return {"case": c, "q": q, "k": k, "pos": pos, "freq": torch.from_numpy(w).cuda(), "m": m}
    lens, new = _lengths(c)
    P, G, H, D = c["page"], c["g"], c["hkv"], c["d"]
    need = -(-lens // P)
    pages = int(need.sum()) + 3
    perm = np.random.RandomState(c["meta"] + 1 + seed % 1000).permutation(pages).astype(np.int32)
    table = np.full((c["seqs"], int(need.max())), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    off = lambda n: torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()  # noqa: E731
    s = {"case": c, "table": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(lens.astype(np.int32)).cuda(),
         "q_off": off(new), "max_q": int(new.max())}
    kc, ks = _fill(gen, pages, P, G, H, D, c["code"], dt)
    vc, vs = _fill(gen, pages, P, G, H, D, c["code"], dt)
    s.update(kc=kc, vc=vc, ks=ks, vs=vs)
    total = int(new.sum())
    if c["op"] == "attn":
        s["q"] = (2.0 * _normal(gen, (total, c["hq"], D))).to(dt)
        s["max_l"] = int(lens.max())
    elif c["op"] == "write":
        x = _rows(gen, total, c["hq"] + 2 * H, D, dt)  # k and v beside the queries
        s["k"], s["v"] = x[:, c["hq"]:c["hq"] + H], x[:, c["hq"] + H:]
        start = (lens - new) // G * G  # the groups the new tokens touch, from their first token
        s["starts"] = torch.from_numpy(start.astype(np.int32)).cuda()
        s["r_off"], s["rows"] = off(lens - start), int((lens - start).sum())
    else:
        s["starts"] = None
        s["r_off"], s["rows"] = off(lens), int(lens.sum())
    return s


def _fill(gen, pages, P, G, H, D, code, dt):
    """A cache as earlier writes left it."""
    kc = torch.empty((pages, P, H, D), dtype=CODE[code], device="cuda")
    ks = torch.empty((pages, H, P // G), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 25) // (P * H * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = _rows(gen, n * P, H, D, dt).float().view(n, P // G, G, H, D)
        sc = _scale(x.abs().amax(dim=(2, 4)), code)  # [n, groups, H]
        kc[a:a + n] = _codes(x, sc[:, :, None, :, None], code).view(n, P, H, D)
        ks[a:a + n] = sc.transpose(1, 2)
    return kc, ks


# ----------------------------------------------------------------------------- plain forms
def _scale(amax, code):
    """int8: the largest magnitude over 127; e4m3: the least power of two that brings it to 448 or less."""
    if code == "int8":
        return torch.clamp(amax / 127.0, min=FLOOR)
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    k = e - 9 + (m > 0.875).to(e.dtype)
    return torch.ldexp(torch.ones_like(amax), torch.clamp(torch.where(amax > 0, k, k - 1000), min=-100))


def _codes(x, scale, code):
    """x / scale rounded to the nearest code, ties to even (int8: in 64 bits, for quotients next to a border)."""
    if code == "int8":
        return torch.round(x.double() / scale.double()).to(torch.int8)
    return (x / scale).to(torch.float8_e4m3fn)


def _slots(s, off, starts, rows):
    """Page, row and sequence of packed rows: row i of a sequence is its token starts + i."""
    c = s["case"]
    i = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(off[1:], i, right=True)
    pos = i - off[seq] + starts[seq]
    page = s["table"][seq, pos // c["page"]].long()
    return page, pos % c["page"], seq


def _plain_rope(s):
    c = s["case"]
    a = s["pos"].double()[:, None] * s["freq"][None, :]
    cos, sin = (torch.cos(a) * s["m"]).float()[:, None, :], (torch.sin(a) * s["m"]).float()[:, None, :]
    if c["back"]:
        sin = -sin
    out = []
    for x in (s["q"], s["k"]):
        t, r = x.float(), c["rot"]
        if c["layout"] == "half":
            x1, x2 = t[..., :r // 2], t[..., r // 2:r]
            y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, t[..., r:]], -1)
        else:
            x1, x2 = t[..., :r:2], t[..., 1:r:2]
            y = torch.cat([torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2), t[..., r:]], -1)
        out.append(y.to(x.dtype))
    return tuple(out)


def _plain_write_one(s, x, cache, scales, page, row, seq):
    c = s["case"]
    G, P, H = c["g"], c["page"], c["hkv"]
    per = P // G
    x = x.float()
    gid = page * per + row // G
    amax = torch.full((scales.shape[0] * per, H), -1.0, device="cuda")
    amax = amax.scatter_reduce(0, gid[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    old = scales.transpose(1, 2).reshape(-1, H)
    # the group that a sequence's first new token falls into may hold tokens of earlier calls
    n = (s["q_off"][1:] - s["q_off"][:-1]).long()
    first = s["lens"].long() - n
    held = torch.where(n > 0, first % G, torch.zeros_like(n))
    fp = torch.clamp(first, max=s["table"].shape[1] * P - 1)
    fgid = s["table"][torch.arange(len(n), device="cuda"), fp // P].long().clamp(min=0) * per + fp % P // G
    keeps = torch.zeros(old.shape[0], device="cuda").index_put((fgid,), (held > 0).float(), accumulate=True) > 0
    new = _scale(amax.clamp(min=0.0), c["code"])
    new = torch.where(keeps[:, None], torch.maximum(old, new), new)
    new = torch.where(amax >= 0, new, old)
    j = torch.arange(G, device="cuda")
    at = (fgid[:, None] * G + j[None, :])
    flat = cache.view(torch.int8).view(-1, H, c["d"])
    codes = flat[at].view(cache.dtype)
    ratio_from, ratio_to = old[fgid][:, None, :, None], new[fgid][:, None, :, None]
    if c["code"] == "int8":
        again = torch.round(codes.double() * ratio_from.double() / ratio_to.double()).to(torch.int8)
    else:
        again = (codes.float() * (ratio_from / ratio_to)).to(torch.float8_e4m3fn)
    again = torch.where((j[None, :] < held[:, None])[:, :, None, None], again.view(torch.int8), flat[at])
    flat[at] = again
    flat[page * P + row] = _codes(x, new[gid][:, :, None], c["code"]).view(torch.int8)
    scales.copy_(new.view(-1, per, H).transpose(1, 2))


def _plain_gather(s, cache, scales, page, row):
    g = s["case"]["g"]
    return cache[page, row].float() * scales[page, :, row // g][:, :, None]


def _plain_read(s, starts):
    page, row, _ = _slots(s, s["r_off"], starts, s["rows"])
    dt = DT[s["case"]["dtype"]]
    return tuple(_plain_gather(s, a, b, page, row).to(dt) for a, b in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))


def _plain_write(s):
    n = s["k"].shape[0]
    page, row, seq = _slots(s, s["q_off"], s["lens"] - (s["q_off"][1:] - s["q_off"][:-1]), n)
    _plain_write_one(s, s["k"], s["kc"], s["ks"], page, row, seq)
    _plain_write_one(s, s["v"], s["vc"], s["vs"], page, row, seq)
    return (*_plain_read(s, s["starts"]), s["ks"], s["vs"])


def _plain_attn(s):
    c = s["case"]
    S, H, D, P, group = c["seqs"], c["hkv"], c["d"], c["page"], c["hq"] // c["hkv"]
    L, Q = s["max_l"], s["max_q"]
    j = torch.arange(L, device="cuda")
    page = s["table"][:, j // P].long().clamp(min=0)  # [S, L]; what lies past a sequence's end is masked below
    k = _plain_gather(s, s["kc"], s["ks"], page.flatten(), (j % P).repeat(S)).view(S, L, H, D)
    v = _plain_gather(s, s["vc"], s["vs"], page.flatten(), (j % P).repeat(S)).view(S, L, H, D)
    n = (s["q_off"][1:] - s["q_off"][:-1]).long()
    i = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["q_off"][1:], i, right=True)
    at = i - s["q_off"][seq]
    q = torch.zeros((S, Q, c["hq"], D), device="cuda")
    q[seq, at] = s["q"].float()
    q = q.view(S, Q, H, group, D).permute(0, 2, 1, 3, 4).reshape(S, H, Q * group, D)
    t = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    last = s["lens"].long()[:, None] - 1
    if c["causal"]:
        last = last - n[:, None] + 1 + torch.arange(Q, device="cuda")[None, :]
        last = torch.minimum(last, s["lens"].long()[:, None] - 1)
    else:
        last = last.expand(S, Q)
    hidden = j[None, None, :] > last[:, :, None]  # [S, Q, L]
    t = t.view(S, H, Q, group, L).masked_fill_(hidden[:, None, :, None, :], float("-inf"))
    top = t.amax(-1, keepdim=True)
    t = t.sub_(top).exp_()
    total = t.sum(-1, keepdim=True)
    o = torch.matmul(t.view(S, H, Q * group, L), v.permute(0, 2, 1, 3)).view(S, H, Q, group, D) / total
    lse = (top + torch.log(total)).squeeze(-1)
    o = o.permute(0, 2, 1, 3, 4).reshape(S, Q, c["hq"], D)[seq, at].to(s["q"].dtype)
    return o, lse.permute(0, 2, 1, 3).reshape(S, Q, c["hq"])[seq, at]


# ----------------------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    if own:
        from exact_scaled_dot_flash_gb300 import attn
        if c["op"] == "rope":
            f = attn.rope_bwd if c["back"] else attn.rope
            return f(s["q"], s["k"], s["pos"], s["freq"], layout=c["layout"], mscale=s["m"])
        cache = (s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"])
        if c["op"] == "write":
            attn.kv8_write(s["k"], s["v"], *cache, s["q_off"])
            k, v = attn.kv8_read(*cache, s["r_off"], s["rows"], starts=s["starts"], dtype=s["k"].dtype)
            return k, v, s["ks"], s["vs"]
        if c["op"] == "read":
            return attn.kv8_read(*cache, s["r_off"], s["rows"], dtype=DT[c["dtype"]])
        return attn.paged_kv8_fwd(s["q"], *cache, s["q_off"], causal=c["causal"], max_queries=s["max_q"],
                                  return_lse=True)
    if c["op"] == "rope":
        return _plain_rope(s)
    if c["op"] == "write":
        return _plain_write(s)
    if c["op"] == "read":
        return _plain_read(s, torch.zeros_like(s["lens"]))
    return _plain_attn(s)


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * n * ES[c["dtype"]] + 4 * c["tokens"], "flops": 3 * n}
    lens, new = _lengths(c)
    H, D, G, es = c["hkv"], c["d"], c["g"], ES[c["dtype"]]
    if c["op"] == "attn":
        rows = float(new.sum()) * c["hq"]
        back = (new * (new - 1) / 2.0) if c["causal"] else 0.0 * new
        pairs = float((new * lens - back).sum()) * c["hq"]
        codes = float(lens.sum()) * H * 2 * (D + 4.0 / G)
        return {"bytes": codes + rows * (2 * D * es + 4), "flops": 4 * pairs * D}
    if c["op"] == "read":
        n = float(lens.sum()) * H * 2
        return {"bytes": n * (D * (1 + es) + 4.0 / G), "flops": n * D}
    n = float(new.sum()) * H * 2  # new tokens: read, written as codes; the touched groups: read back
    t = float((lens - (lens - new) // G * G).sum()) * H * 2
    return {"bytes": n * D * (es + 1) + t * (D * (1 + es) + 8.0 / G), "flops": 3 * n * D + t * D}


# ----------------------------------------------------------------------------- in 64 bits
def _e4m3_values():
    """The 127 magnitudes 0 .. 448 of the format: 4 bits of exponent, 3 of mantissa, bias 7."""
    return np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127])


def _near(x, code):
    """Values of the nearest codes (ties to the even code) of float64 x."""
    if code == "int8":
        return torch.round(x)
    v = torch.from_numpy(_e4m3_values()).to(x.device)
    a = x.abs().contiguous()
    hi = torch.searchsorted(v, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = v[hi] - a, a - v[lo]
    i = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
    return torch.copysign(v[i], x)


def _exact_write_one(x, values, scales, table, lens, new, c):
    """values: float64 code values [pages, P, H, D], scales float32 [pages, H, groups]; both are updated."""
    G, P, at = c["g"], c["page"], 0
    for s, (L, n) in enumerate(zip(lens, new)):
        pos = L - n
        while pos < L:
            g0 = pos // G * G
            end = min(L, g0 + G)
            page, r, held = int(table[s, g0 // P]), g0 % P, pos - g0
            part = x[at:at + end - pos].double()  # [m, H, D]
            amax = part.abs().amax(dim=(0, 2)).cpu().numpy()
            if c["code"] == "int8":
                sc = (amax / 127.0).astype(np.float32).astype(np.float64)
            else:
                sc = np.array([2.0 ** -100 if a == 0 else 2.0 ** math.ceil(math.log2(a / 448.0)) for a in amax])
            sc = torch.from_numpy(np.maximum(sc, FLOOR)).to(x.device)
            if held:
                old = scales[page, :, r // G].double()
                sc = torch.maximum(sc, old)
                values[page, r:r + held] = _near(values[page, r:r + held] * old[:, None] / sc[:, None], c["code"])
            values[page, r + held:r + end - g0] = _near(part / sc[:, None], c["code"])
            scales[page, :, r // G] = sc.float()
            at += end - pos
            pos = end


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rope":
        out = []
        half = c["rot"] // 2
        ang = torch.outer(s["pos"].double(), s["freq"])
        turn = torch.polar(torch.full_like(ang, s["m"]), -ang if c["back"] else ang)[:, None, :]  # complex128
        for x in (s["q"], s["k"]):
            y = x.double()
            head = y[..., :c["rot"]]
            pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (half, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.transpose(-1, -2) if c["layout"] == "half" else z
            out.append(torch.cat([z.reshape(head.shape), y[..., c["rot"]:]], -1))
        return tuple(out)
    lens, new = _lengths(c)
    if c["op"] == "write" and int(new.sum()) // c["g"] + 2 * c["seqs"] > 20000:
        return None  # over 20 seconds, group by group
    table = s["table"].cpu().numpy()
    P, G = c["page"], c["g"]

    def tokens(codes, scales, q, a, b):
        """float64 [b - a, H, D]: tokens a .. b-1 of sequence q."""
        j = torch.arange(a, b, device="cuda")
        pg = s["table"][q].long()[j // P]
        return codes[pg, j % P].double() * scales[pg, :, j % P // G].double()[:, :, None]

    if c["op"] == "attn":
        outs, lses, at = [], [], 0
        H, group, D = c["hkv"], c["hq"] // c["hkv"], c["d"]
        for i, (L, n) in enumerate(zip(lens.tolist(), new.tolist())):
            k, v = tokens(s["kc"], s["ks"], i, 0, L), tokens(s["vc"], s["vs"], i, 0, L)
            q = s["q"][at:at + n].double().view(n, H, group, D)
            at += n
            seen = torch.arange(L, device="cuda")[None, :] <= (torch.arange(n, device="cuda")[:, None] + L - n
                                                              if c["causal"] else L)
            o = torch.empty((n, H, group, D), dtype=torch.float64, device="cuda")
            z = torch.empty((n, H, group), dtype=torch.float64, device="cuda")
            for h in range(H):
                t = torch.einsum("ngd,ld->ngl", q[:, h], k[:, h]) / math.sqrt(D)
                t = torch.where(seen[:, None, :], t, torch.full_like(t, float("-inf")))
                z[:, h] = torch.logsumexp(t, -1)
                o[:, h] = torch.einsum("ngl,ld->ngd", torch.exp(t - z[:, h][..., None]), v[:, h])
            outs.append(o.view(n, c["hq"], D))
            lses.append(z.view(n, c["hq"]))
        return torch.cat(outs), torch.cat(lses)
    kv, ks, vv, vs = s["kc"].double(), s["ks"].clone(), s["vc"].double(), s["vs"].clone()
    first = [0] * c["seqs"]
    if c["op"] == "write":
        _exact_write_one(s["k"], kv, ks, table, lens.tolist(), new.tolist(), c)
        _exact_write_one(s["v"], vv, vs, table, lens.tolist(), new.tolist(), c)
        first = s["starts"].tolist()
    rows = tuple(torch.cat([tokens(a, b, i, first[i], L) for i, L in enumerate(lens.tolist())])
                 for a, b in ((kv, ks), (vv, vs)))
    return rows + (ks.double(), vs.double()) if c["op"] == "write" else rows
