"""Measured cases of a batch that shares a prompt: the pages of a cache, attention that reads a
shared prefix once, and rotary positions with several axes. Their plain forms, the calls a program
makes of this package, and their values in 64 bits.

``pages`` manages the pages of a paged cache: a table [sequences, blocks] of page numbers (-1: none),
the lengths, and the number of table entries that name each page. ``prefix`` is attention of packed
queries over a paged cache where groups of sequences begin with the same tokens. ``rope`` turns
queries and keys by positions with an axis for each pair of elements (time, height, width).
"""
import math

import numpy as np
import torch

own = False  # False: the plain forms below; True: the package's kernels

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}


# ----------------------------------------------------------------------------- cases
def _pages(name, op, seqs, width, page, hkv, d, layers, lo, hi, meta):
    """seqs: rows in use; width: requests that fork (each has seqs / width rows)."""
    return {"name": name, "op": op, "seqs": seqs, "width": width, "page": page, "hkv": hkv, "d": d, "layers": layers,
            "lo": lo, "hi": hi, "meta": meta}


def _prefix(name, dtype, groups, mem_lo, mem_hi, hq, hkv, d, page, pre_lo, pre_hi, suf_lo, suf_hi, q_lo, q_hi, meta,
            causal=True):
    return {"name": name, "op": "prefix", "dtype": dtype, "groups": groups, "mem_lo": mem_lo, "mem_hi": mem_hi,
            "hq": hq, "hkv": hkv, "d": d, "page": page, "pre_lo": pre_lo, "pre_hi": pre_hi, "suf_lo": suf_lo,
            "suf_hi": suf_hi, "q_lo": q_lo, "q_hi": q_hi, "meta": meta, "causal": causal}


def _rope(name, tokens, hq, hk, d, rot, layout, dtype, axes, cycle, back=False):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rot, "layout": layout,
            "dtype": dtype, "axes": axes, "cycle": cycle, "back": back}


def listed():
    return [
        # a request is answered four times over: its row is forked, each answer gets room for a token
        _pages("pages_sample", "sample", 4, 1, 16, 2, 64, 1, 201, 201, 30),
        # a step of beam search: 16 requests of 4 beams, 8 layers, beams follow their parents
        _pages("pages_beams", "beams", 64, 16, 16, 8, 128, 8, 500, 3000, 31),
        # 64 of 512 sequences are done and as many prompts come in
        _pages("pages_admit", "admit", 512, 64, 16, 8, 128, 1, 100, 4000, 32),
        # the older half of a pool's sequences has left: the younger half moves down
        _pages("pages_compact", "compact", 64, 32, 64, 8, 128, 2, 1024, 4096, 33),
        # four answers to one chat just begun: latency
        _prefix("prefix_first_f16", "f16", 1, 4, 4, 8, 2, 64, 16, 201, 201, 1, 40, 1, 1, 40),
        # a step of 64 sequences behind one system prompt (the repository's decode heads)
        _prefix("prefix_step_bf16", "bf16", 1, 64, 64, 32, 8, 128, 64, 8192, 8192, 100, 2000, 1, 1, 41),
        # several rooms of a few sequences, groups of 7 heads
        _prefix("prefix_rooms_f16", "f16", 8, 2, 12, 28, 4, 128, 32, 1000, 8000, 1, 1500, 1, 1, 42),
        # 96 questions to one long document, an odd length
        _prefix("prefix_document_bf16", "bf16", 1, 96, 96, 32, 8, 128, 128, 60001, 60001, 20, 500, 1, 1, 43),
        # 24 questions of 16 to 128 tokens come in behind a shared prompt
        _prefix("prefix_questions_bf16", "bf16", 1, 24, 24, 32, 8, 128, 64, 4096, 4096, 16, 128, 16, 128, 44),
        # a check in full precision, small heads, 3 drafted tokens
        _prefix("prefix_f32", "f32", 3, 1, 9, 6, 2, 32, 8, 37, 700, 3, 90, 3, 3, 45),
        # the gradient of one image of 32 x 32 patches and its text, two axes
        _rope("rope_image_grad_f32", 1061, 16, 16, 64, 64, "half", "f32", 2, False, True),
        # a video prompt: frames x height x width, three axes in turn over the pairs
        _rope("rope_video_bf16", 9416, 32, 8, 128, 128, "half", "bf16", 3, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("pages", "prefix", "prefix", "rope"))
    if op == "rope":
        d = rng.choice((64, 128))
        c = _rope("", _log(rng, 1, 9000), rng.choice((8, 14, 32)), rng.choice((1, 2, 8)), d,
                  rng.choice((d, d // 2, d // 4 * 3)), rng.choice(("half", "interleaved")),
                  rng.choice(("f32", "f16", "bf16")), rng.choice((2, 3, 4)), rng.choice((False, True)),
                  rng.choice((False, True)))
    elif op == "pages":
        mode = rng.choice(("sample", "beams", "admit", "compact"))
        width = _log(rng, 1, 16)
        seqs = width * rng.choice((2, 3, 4)) if mode in ("sample", "beams") else 2 * width
        hi = _log(rng, 20, 2000)
        c = _pages("", mode, seqs, width, rng.choice((16, 32, 64)), rng.choice((1, 2, 8)), rng.choice((64, 128)),
                   rng.choice((1, 2)), max(1, int(hi * rng.uniform(0.2, 1.0))), hi, rng.randrange(1 << 20))
    else:
        groups = _log(rng, 1, 6)
        q = rng.choice((1, 1, 1, 2, 5, 40))
        mem = _log(rng, 1, (40 if q < 40 else 12) // groups)
        hkv = rng.choice((1, 2, 4, 8))
        d = rng.choice((64, 128))
        pre = _log(rng, 16, (16000 if q < 40 else 4000) // groups)
        suf = _log(rng, 8, 1500 if q < 40 else 300)
        c = _prefix("", rng.choice(("bf16", "f16")), groups, max(1, int(mem * rng.uniform(0.3, 1.0))), mem,
                    hkv * rng.choice((1, 3, 4, 7, 8)), hkv, d, rng.choice((16, 32, 64, 128)),
                    max(1, int(pre * rng.uniform(0.2, 1.0))), pre, max(1, int(suf * rng.uniform(0.1, 1.0))), suf,
                    max(1, int(q * rng.uniform(0.4, 1.0))), q, rng.randrange(1 << 20), rng.random() < 0.8)
    return {k: v for k, v in c.items() if k != "name"}


# ----------------------------------------------------------------------------- inputs
def _normal(gen, shape, dt):
    x = torch.empty(shape, dtype=dt, device="cuda")
    for part in x.flatten().split(1 << 27):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=torch.float32))
    return x


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _offsets(n):
    return np.concatenate([[0], np.cumsum(n)])


def _page_lengths(c):
    """Lengths of the rows in use; both halves alike for `compact`."""
    r = np.random.RandomState(c["meta"])
    if c["op"] in ("sample", "beams"):
        return np.repeat(r.randint(c["lo"], c["hi"] + 1, c["width"]), c["seqs"] // c["width"])
    if c["op"] == "compact":
        half = r.randint(c["lo"], c["hi"] + 1, c["seqs"] // 2)
        return np.concatenate([half, half])
    return r.randint(c["lo"], c["hi"] + 1, c["seqs"])


def _prepare_pages(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    P, n = c["page"], c["seqs"]
    r = np.random.RandomState(seed % (1 << 31))
    lens = _page_lengths(c)
    rows = {"sample": n + c["width"], "beams": 2 * n, "admit": n, "compact": n}[c["op"]]
    blocks = -(-(c["hi"] + 1) // P)
    need = -(-lens // P)
    table, full = np.full((rows, blocks), -1), np.zeros(rows, np.int64)
    if c["op"] == "sample":  # the requests; their answers' rows are empty
        lens, need, first = lens[::n // c["width"]], need[::n // c["width"]], n
        pages = int(need.sum()) + 2 * n + 5
    else:
        first = 0
        pages = int(need.sum()) + (n if c["op"] == "beams" else 0) + int(need.sum()) // 8 + 5
    if c["op"] == "compact":  # one half at the bottom of the pool, the other above it
        order = np.concatenate([r.permutation(int(need.sum()) // 2), int(need.sum()) // 2 + r.permutation(int(need.sum()) // 2)])
    else:
        order = r.permutation(pages)
    at = 0
    for i, b in enumerate(need):
        table[first + i, :b] = order[at:at + b]
        full[first + i] = lens[i]
        at += b
    refs = np.bincount(table[table >= 0], minlength=pages)
    s = {"case": c, "table": _i32(table), "lens": _i32(full), "refs": _i32(refs)}
    s["caches"] = [_normal(gen, (pages, P, c["hkv"], c["d"]), torch.bfloat16) for _ in range(2 * c["layers"])]
    one = lambda idx: _i32(np.isin(np.arange(rows), idx))  # noqa: E731  one new token for some rows
    if c["op"] == "sample":
        kids = np.arange(n)
        s.update(parents=_i32(n + kids // (n // c["width"])), kids=_i32(kids), new=one(kids))
    elif c["op"] == "beams":
        per = n // c["width"]
        parent = np.arange(n) // per * per + r.randint(0, per, n)
        s["sides"] = [(_i32(parent), _i32(np.arange(n)), _i32(n + np.arange(n)), one(n + np.arange(n))),
                      (_i32(n + parent), _i32(n + np.arange(n)), _i32(np.arange(n)), one(np.arange(n)))]
    elif c["op"] == "admit":
        out = r.permutation(n)[:c["width"]]
        new = np.zeros(rows)
        new[out] = lens[out]
        s.update(done=_i32(out), new=_i32(new))
    else:
        half = n // 2
        s["sides"] = []
        for rows_out in (np.arange(half), half + np.arange(half)):
            new = np.zeros(rows)
            new[rows_out] = lens[rows_out]
            s["sides"].append((_i32(rows_out), _i32(new)))
    return s


def _lengths(c):
    """Per group: sequences and prefix; per sequence: its own tokens and the new ones among them."""
    r = np.random.RandomState(c["meta"])
    members = r.randint(c["mem_lo"], c["mem_hi"] + 1, c["groups"])
    prefix = r.randint(c["pre_lo"], c["pre_hi"] + 1, c["groups"])
    new = r.randint(c["q_lo"], c["q_hi"] + 1, int(members.sum()))
    suffix = np.maximum(new, r.randint(c["suf_lo"], c["suf_hi"] + 1, len(new)))
    return members, prefix, suffix, new


def _prepare_prefix(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, P, H, D = DT[c["dtype"]], c["page"], c["hkv"], c["d"]
    members, prefix, suffix, new = _lengths(c)
    group = np.repeat(np.arange(c["groups"]), members)
    lens = prefix[group] + suffix
    shared = prefix // P  # full pages
    pages = int(shared.sum() + (-(-lens // P) - shared[group]).sum()) + 3
    perm = np.random.RandomState(seed % (1 << 31)).permutation(pages)
    table = np.full((len(lens), int((-(-lens // P)).max())), -1)
    at, first, copies = 0, _offsets(members), []
    for g in range(c["groups"]):
        common = perm[at:at + shared[g]]
        at += shared[g]
        for i in range(first[g], first[g + 1]):
            own_pages = -(-lens[i] // P) - shared[g]
            table[i, :shared[g]] = common
            table[i, shared[g]:shared[g] + own_pages] = perm[at:at + own_pages]
            at += own_pages
            if prefix[g] % P and i > first[g]:  # the shared tokens in the page where the rows part
                copies.append((table[first[g], shared[g]], table[i, shared[g]], prefix[g] % P))
    kc, vc = (_normal(gen, (pages, P, H, D), dt) for _ in range(2))
    if copies:
        src, dst, upto = (torch.from_numpy(np.array(a, dtype=np.int64)).cuda() for a in zip(*copies))
        keep = (torch.arange(P, device="cuda")[None, :] < upto[:, None])[:, :, None, None]
        for x in (kc, vc):
            x[dst] = torch.where(keep, x[src], x[dst])
    q = _normal(gen, (int(new.sum()), c["hq"], D), torch.float32)
    return {"case": c, "q": (2.0 * q).to(dt), "kc": kc, "vc": vc, "table": _i32(table), "lens": _i32(lens),
            "q_off": _i32(_offsets(new)), "g_off": _i32(first), "pre": _i32(prefix), "max_q": int(new.max()),
            "max_gq": int(np.add.reduceat(new, first[:-1]).max()), "max_pre": int(prefix.max()),
            "max_suf": int(suffix.max()), "group": torch.from_numpy(group).cuda()}


def _sections(c):
    """Axis of each pair: runs of pairs, or in turn."""
    n, a = c["rot"] // 2, c["axes"]
    return np.arange(n) % a if c["cycle"] else np.minimum(np.arange(n) * a // n, a - 1)


def _prepare_rope(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, a = c["tokens"], c["axes"]
    x = _normal(gen, (n, c["hq"] + 2 * c["hk"], c["d"]), DT[c["dtype"]])  # q, k and v of one projection
    start = int(torch.randint(0, 4000, (1,), generator=gen, device="cuda"))
    side = max(1, int(round(n ** (1.0 / a))))
    i = np.arange(n)  # a grid (time, height, width, ...); what is left over is text behind it
    grid = np.stack([i // side ** (a - 1 - k) % (side if k else n) for k in range(a)])
    text = np.broadcast_to(grid.max() + 1 + i - side ** a, grid.shape)
    pos = start + np.where(i < side ** a, grid, text)
    w = 10000.0 ** (-np.arange(0, c["rot"], 2) / c["rot"])
    return {"case": c, "q": x[:, :c["hq"]], "k": x[:, c["hq"]:c["hq"] + c["hk"]], "pos": _i32(pos),
            "freq": torch.from_numpy(w).cuda(), "axes": _i32(_sections(c))}


def prepare(case, seed):
    return {"prefix": _prepare_prefix, "rope": _prepare_rope}.get(case["op"], _prepare_pages)(case, seed)


# ----------------------------------------------------------------------------- plain forms
def _count(entries, n):
    """How often each of n pages is named (-1 names none)."""
    e = entries.flatten().long()
    return torch.zeros(n + 1, dtype=torch.int32, device="cuda").index_add_(
        0, torch.where(e < 0, n, e), torch.ones_like(e, dtype=torch.int32))[:n]


def _plain_fork(s, parents, kids):
    P, n = s["case"]["page"], s["refs"].shape[0]
    p, k = parents.long(), kids.long()
    blocks = torch.arange(s["table"].shape[1], device="cuda")
    rows = torch.where(blocks * P < s["lens"][p][:, None], s["table"][p], -1)
    s["refs"] += _count(rows, n) - _count(s["table"][k], n)
    s["table"][k] = rows
    s["lens"][k] = s["lens"][p]


def _plain_free(s, rows):
    r = rows.long()
    s["refs"] -= _count(s["table"][r], s["refs"].shape[0])
    s["table"][r] = -1
    s["lens"][r] = 0


def _plain_reserve(s, new):
    table, refs, P = s["table"], s["refs"], s["case"]["page"]
    n = refs.shape[0]
    b = torch.arange(table.shape[1], device="cuda")[None, :]
    L = s["lens"][:, None]
    end = torch.clamp(L + new[:, None], max=table.shape[1] * P)
    write = (new[:, None] > 0) & (b >= L // P) & (b * P < end)  # blocks that get tokens
    page = torch.where(table < 0, n, table).long()
    held = torch.cat([refs, refs.new_zeros(1)])[page]
    shared = write & (table >= 0) & (held > 1)
    writers = torch.cat([_count(torch.where(shared, table, -1), n), refs.new_zeros(1)])[page]
    order = torch.arange(table.numel(), device="cuda").view_as(table)
    last = torch.full((n + 1,), -1, device="cuda").scatter_reduce(
        0, page.flatten(), torch.where(shared, order, -1).flatten(), "amax")[page]
    need = write & ((table < 0) | (shared & ~((writers == held) & (last == order))))  # the last one of all keeps it
    total, free = need.sum(), (refs == 0).sum()
    need = need & (total <= free)
    fresh = torch.argsort((refs > 0).int(), stable=True).int()  # free pages first, the lowest first
    rank = torch.cumsum(need.flatten().long(), 0).view_as(table) - 1
    into = torch.where(need, fresh[rank.clamp(0, n - 1)], table)
    copy = need & shared & (b * P < L)
    src, dst = table[copy].long(), into[copy].long()
    for x in s["caches"]:
        x[dst] = x[src]
    refs += _count(torch.where(need, into, -1), n) - _count(torch.where(need, table, -1), n)
    table.copy_(into)
    return torch.stack([need.sum(), (total - free).clamp(min=0)]).int()


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    n = refs.shape[0]
    used, i = refs > 0, torch.arange(n, device="cuda")
    count = used.sum()
    dst, src = torch.nonzero(~used & (i < count)).flatten(), torch.nonzero(used & (i >= count)).flatten()
    for x in s["caches"]:
        x[dst] = x[src]
    to = torch.where(used, i, -1)
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    refs[dst] = refs[src]
    refs[src] = 0
    return to.int(), count.int().view(1)


def _gather(x, table, j, P):
    """float32 [rows, tokens, heads, D]: tokens j of the rows of a table; what is past a row's end is masked later."""
    page = torch.gather(table.long(), 1, (j // P).clamp(max=table.shape[1] - 1)).clamp(min=0)
    return x[page, j % P].float()


def _partial(q, k, v, lim, j):
    """(m, l, O) of rows that see the keys j < lim. q [B, Q, H, G, D], k and v [B, T, H, D], lim [B, Q], j [B, T]."""
    t = torch.einsum("bqhgd,bthd->bhgqt", q, k) * (1.0 / math.sqrt(q.shape[-1]))
    t = t.masked_fill_((j[:, None, :] >= lim[:, :, None])[:, None, None], float("-inf"))
    m = t.amax(-1)
    t = t.sub_(torch.where(m == float("-inf"), 0.0, m)[..., None]).exp_()
    o = torch.einsum("bhgqt,bthd->bqhgd", t, v)
    return m.permute(0, 3, 1, 2), t.sum(-1).permute(0, 3, 1, 2), o


def _plain_prefix(s):
    c = s["case"]
    P, H, D, G = c["page"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    n, S = s["q"].shape[0], s["lens"].shape[0]
    q = s["q"].float().view(n, H, G, D)
    i = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["q_off"][1:], i.int(), right=True)
    in_seq = i - s["q_off"][seq]
    lens, new = s["lens"].long(), (s["q_off"][1:] - s["q_off"][:-1]).long()
    sees = lens[seq] - new[seq] + in_seq + 1 if c["causal"] else lens[seq]
    # the prefix: the queries of a group at once
    grp = s["group"][seq]
    in_grp = i - s["q_off"][s["g_off"][grp].long()]
    pre = s["pre"].long()
    qg = torch.zeros((c["groups"], s["max_gq"], H, G, D), device="cuda")
    qg[grp, in_grp] = q
    lim = torch.zeros((c["groups"], s["max_gq"]), dtype=torch.long, device="cuda")
    lim[grp, in_grp] = torch.minimum(sees, pre[grp])
    j = torch.arange(s["max_pre"], device="cuda").expand(c["groups"], -1)
    rows = s["table"][s["g_off"][:-1].long()]
    a = [x[grp, in_grp] for x in _partial(qg, _gather(s["kc"], rows, j, P), _gather(s["vc"], rows, j, P), lim, j)]
    # the sequences' own keys
    qs = torch.zeros((S, s["max_q"], H, G, D), device="cuda")
    qs[seq, in_seq] = q
    lim = torch.zeros((S, s["max_q"]), dtype=torch.long, device="cuda")
    lim[seq, in_seq] = sees
    j = pre[s["group"]][:, None] + torch.arange(s["max_suf"], device="cuda")
    b = [x[seq, in_seq] for x in _partial(qs, _gather(s["kc"], s["table"], j, P), _gather(s["vc"], s["table"], j, P), lim, j)]
    top = torch.maximum(a[0], b[0])
    fa, fb = torch.exp(a[0] - top), torch.exp(b[0] - top)
    total = fa * a[1] + fb * b[1]
    o = (fa[..., None] * a[2] + fb[..., None] * b[2]) / total[..., None]
    return o.reshape(n, c["hq"], D).to(s["q"].dtype), (top + torch.log(total)).reshape(n, c["hq"])


def _plain_rope(s):
    c = s["case"]
    a = s["pos"][s["axes"].long()].double().T * s["freq"][None, :]
    cos, sin = torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]
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


# ----------------------------------------------------------------------------- one pass
def _run_pages(s, fork, free, reserve, compact):
    op, back = s["case"]["op"], []
    if op == "sample":  # the answers before are done; the requests are answered again
        free(s["kids"])
        fork(s["parents"], s["kids"])
        back = [reserve(s["new"])]
    elif op == "beams":  # the beams' rows and those of their parents change places
        parents, old, kids, new = s["sides"][0]
        s["sides"] = s["sides"][::-1]
        fork(parents, kids)
        free(old)
        back = [reserve(new)]
    elif op == "admit":
        free(s["done"])
        back = [reserve(s["new"])]
    else:  # the older half leaves, the pool is compacted, and as many come in above
        rows, new = s["sides"][0]
        s["sides"] = s["sides"][::-1]
        free(rows)
        back = [*compact(), reserve(new)]
    if op in ("admit", "compact"):
        s["lens"] += s["new"] if op == "admit" else new
    return [s["table"], s["lens"], s["refs"], *back, *s["caches"]]


def run(state):
    s, c = state, state["case"]
    if own:
        from exact_scaled_dot_flash_gb300 import attn
        if c["op"] == "prefix":
            return attn.paged_prefix_fwd(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["q_off"], s["g_off"], s["pre"],
                                         causal=c["causal"], max_queries=s["max_q"], max_group_queries=s["max_gq"],
                                         return_lse=True)
        if c["op"] == "rope":
            f = attn.rope_bwd if c["back"] else attn.rope
            return f(s["q"], s["k"], s["pos"], s["freq"], layout=c["layout"], axes=s["axes"])
        t, lens, refs, x = s["table"], s["lens"], s["refs"], s["caches"]
        return _run_pages(s, lambda p, k: attn.pages_fork(t, lens, refs, p, k, page_size=c["page"]),
                          lambda r: attn.pages_free(t, lens, refs, r),
                          lambda n: attn.pages_reserve(t, lens, refs, n, x, page_size=c["page"]),
                          lambda: attn.pages_compact(t, refs, x))
    if c["op"] == "prefix":
        return _plain_prefix(s)
    if c["op"] == "rope":
        return _plain_rope(s)
    return _run_pages(s, lambda p, k: _plain_fork(s, p, k), lambda r: _plain_free(s, r),
                      lambda n: _plain_reserve(s, n), lambda: _plain_compact(s))


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * n * ES[c["dtype"]] + 4 * c["axes"] * c["tokens"], "flops": 3 * n}
    if c["op"] == "prefix":
        members, prefix, suffix, new = _lengths(c)
        group = np.repeat(np.arange(c["groups"]), members)
        keys = new * (prefix[group] + suffix) - (new * (new - 1) / 2.0 if c["causal"] else 0.0)
        es, rows = ES[c["dtype"]], float(new.sum()) * c["hq"]
        cache = float(prefix.sum() + suffix.sum()) * c["hkv"] * c["d"] * 2 * es
        return {"bytes": cache + rows * (2 * c["d"] * es + 4), "flops": 4.0 * float(keys.sum()) * c["hq"] * c["d"]}
    lens = _page_lengths(c)
    need = -(-lens // c["page"])
    page = 2 * c["layers"] * c["page"] * c["hkv"] * c["d"] * 2.0  # bytes of a page in all buffers
    per = c["seqs"] // c["width"]
    if c["op"] in ("sample", "beams"):  # rows read, written, given back; pages that hold part of a page are copied
        # of `per` beams that choose a parent at random, so many find its page still named by another one
        again = per * (1.0 - 1.0 / per) ** per if c["op"] == "beams" else per
        moved = float((lens % c["page"] > 0).sum()) / per * again
        return {"bytes": float(need.sum()) * 4 * 6 + moved * 2 * page, "flops": 0}
    if c["op"] == "admit":
        return {"bytes": float(need.mean()) * c["width"] * 4 * 6 + float(need.sum()) * 4, "flops": 0}
    half = float(need.sum()) / 2
    return {"bytes": half * 2 * page + half * 4 * 12, "flops": 0}


# ----------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "rope":
        s = prepare(c, seed)
        out, half = [], c["rot"] // 2
        ang = torch.stack([s["pos"][a].double() * w for a, w in zip(_sections(c).tolist(), s["freq"])], 1)
        turn = torch.polar(torch.ones_like(ang), -ang if c["back"] else ang)[:, None, :]  # complex128
        for x in (s["q"], s["k"]):
            y = x.double()
            head = y[..., :c["rot"]]
            pairs = head.unflatten(-1, (2, half)).transpose(-1, -2) if c["layout"] == "half" else head.unflatten(-1, (half, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.transpose(-1, -2) if c["layout"] == "half" else z
            out.append(torch.cat([z.reshape(head.shape), y[..., c["rot"]:]], -1))
        return tuple(out)
    if c["op"] != "prefix":
        return None  # whole numbers and copies
    s = prepare(c, seed)
    H, D, P, G = c["hkv"], c["d"], c["page"], c["hq"] // c["hkv"]
    members, prefix, suffix, new = _lengths(c)
    lens = prefix[np.repeat(np.arange(c["groups"]), members)] + suffix
    outs, lses, at = [], [], 0
    for i, (L, n) in enumerate(zip(lens.tolist(), new.tolist())):  # every sequence by its own row alone
        j = torch.arange(L, device="cuda")
        k, v = (x[s["table"][i].long()[j // P], j % P].double() for x in (s["kc"], s["vc"]))
        q = s["q"][at:at + n].double().view(n, H, G, D)
        at += n
        seen = j[None, :] <= (torch.arange(n, device="cuda")[:, None] + L - n if c["causal"] else L)
        t = torch.einsum("nhgd,lhd->hngl", q, k) / math.sqrt(D)
        t = torch.where(seen[None, :, None, :], t, torch.full_like(t, float("-inf")))
        z = torch.logsumexp(t, -1)
        o = torch.einsum("hngl,lhd->nhgd", torch.exp(t - z[..., None]), v)
        outs.append(o.reshape(n, c["hq"], D))
        lses.append(z.permute(1, 0, 2).reshape(n, c["hq"]))
    return torch.cat(outs), torch.cat(lses)
