"""Measured cases of the paged bf16 KV cache: a step's masked attention for a
batch whose sequences share long prefixes, each prefix attended to once for
all of its sequences, and appending tokens to the cache with the position
rotation of queries and keys applied on the way.

``run`` computes each operator in a plain form of elementary torch operations
(``own`` false) or calls the library's ``la_kv16_*`` entry points through
``KV16Cache`` (``own`` true) on the same inputs.  ``exact`` states the same
results from the definitions in 64 bits.

Pages.  k_pages and v_pages are bf16 [n_pages][kv heads][page][D]; slot = page
index * page + offset in the page.

Attention.  Sequences first[p] .. first[p + 1] - 1 share prefix p: their keys
are the prefix's prefix_lens[p] tokens, then their own lens[b] tokens, then the
step's rows that the combined 2D-window + verification mask lets a row see.

Rotation.  Pair i of the first rot channels of a query or key at position t
turns by t * theta^(-2 i / rot); pair i is channels (i, i + rot / 2), or
(2 i, 2 i + 1) where neighbours form the pairs.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the tiny model's greedy step of two chats behind one short system prompt: pure latency
        dict(name="attend-tiny-greedy", op="attend", batch=2, heads=4, kv_heads=4, dim=64, W=0, N=2, G=0, lo=1, hi=5,
             prefixes="33x2", page=16),
        # one layer of a 7B service: 128 single tokens behind one prompt of 1000 tokens
        dict(name="attend-7b-greedy-128", op="attend", batch=128, heads=32, kv_heads=32, dim=128, W=0, N=2, G=0, lo=31,
             hi=256, prefixes="1000x128", page=64),
        # 32 single tokens of the 34B grouped-query model over one long document
        dict(name="attend-34b-greedy-document", op="attend", batch=32, heads=64, kv_heads=8, dim=128, W=0, N=2, G=0, lo=0,
             hi=700, prefixes="32767x32", page=128),
        # 8 lookahead steps (W=7 N=5 G=7, 57 rows) of the 34B model behind a prompt of 8191 tokens
        dict(name="attend-34b-lookahead-8", op="attend", batch=8, heads=64, kv_heads=8, dim=128, W=7, N=5, G=7, lo=100,
             hi=1300, prefixes="8191x8", page=64),
        # 4 lookahead steps (W=15 N=5 G=15, 121 rows) of the 7B model behind its 512-token prompt
        dict(name="attend-7b-lookahead-4", op="attend", batch=4, heads=32, kv_heads=32, dim=128, W=15, N=5, G=15, lo=17,
             hi=300, prefixes="511x4", page=16),
        # six questions' prompts (blocks of 100 rows) written behind the 13B model's 1024-token prompt
        dict(name="attend-13b-questions", op="attend", batch=6, heads=40, kv_heads=40, dim=128, W=0, N=100, G=1, lo=0,
             hi=200, prefixes="1024x6", page=32),
        # a mixed service: three prompts with 20, 5 and 15 of the 48 sequences, 8 without any
        dict(name="attend-34b-greedy-mixed", op="attend", batch=48, heads=64, kv_heads=8, dim=128, W=0, N=2, G=0, lo=5,
             hi=2047, prefixes="4000x20 777x5 1501x15", page=32),
        # a lookahead step's rows of 4 sequences (57 each): queries and keys rotated for the attention, nothing written
        # but the current token, whose key and value are final
        dict(name="append-7b-step", op="append", heads=32, kv_heads=32, dim=128, rot=128, pairs="half", dtype="bf16",
             n=4 * 57, stored=57, q=True, k_out=True, far=2303, theta=1e4, page=64),
        # 16 prompts of the 34B model, 18 K tokens in all, written behind what is there
        dict(name="append-34b-prompts", op="append", heads=64, kv_heads=8, dim=128, rot=128, pairs="half", dtype="bf16",
             n=18441, stored=1, q=True, k_out=True, far=4096, theta=1e4, page=64),
        # 128 single tokens at far positions, half of the channels rotated in neighbouring pairs
        dict(name="append-greedy-far", op="append", heads=32, kv_heads=8, dim=128, rot=64, pairs="next", dtype="bf16",
             n=128, stored=1, q=True, k_out=False, far=1048575, theta=1e6, page=128),
        # the fp32 debug model's prompts, keys and values alone
        dict(name="append-tiny-fp32", op="append", heads=4, kv_heads=4, dim=64, rot=64, pairs="half", dtype="fp32",
             n=1951, stored=1, q=False, k_out=False, far=800, theta=1e4, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append"])
    page = rng.choice([16, 32, 64, 128])
    dim = rng.choice([64, 128, 128])
    kv_heads = _log(rng, 1, 40)
    group = rng.choice([1, 1, 2, 3, 4, 7, 8])
    if op == "attend":
        # greedy rows, a lookahead step's rows, or a block of prompt rows (a chain of N rows)
        W, N, G = rng.choice([(0, 2, 0), (0, 2, 0), (rng.randint(1, 15), rng.randint(2, 5), rng.randint(0, 15)),
                              (0, rng.randint(2, 128), 1)])
        batch, hi = _log(rng, 1, 128), _log(rng, 2, 4096)
        cuts = sorted(rng.randint(0, batch) for _ in range(rng.choice([1, 1, 2, 4])))
        prefixes = [(_log(rng, 1, 32767), b - a) for a, b in zip([0] + cuts, cuts + [batch]) if b > a]
        if rng.random() < 0.5 and len(prefixes) > 1:
            prefixes.pop()                          # the last sequences have none
        c = dict(op=op, batch=batch, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, W=W, N=N, G=G,
                 lo=int(hi * rng.random()), hi=hi, prefixes=_text(prefixes), page=page)
        while work(c)["bytes"] > 2.5e8 or work(c)["flops"] > 1.2e11:
            if c["kv_heads"] > 1:
                c["kv_heads"] = c["kv_heads"] * 3 // 4
                c["heads"] = c["kv_heads"] * group
            else:
                c["lo"], c["hi"] = c["lo"] * 3 // 4, max(1, c["hi"] * 3 // 4)
                c["prefixes"] = _text([(max(1, n * 3 // 4), k) for n, k in _shared(c)])
        return c
    rot = rng.choice([dim, dim, dim // 2, 48])
    n = _log(rng, 1, max(1, min(20000, 18441 * 80 * 128 // ((group + 2) * kv_heads * dim))))
    return dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, rot=rot, pairs=rng.choice(["half", "half", "next"]),
                dtype=rng.choice(["bf16", "bf16", "fp32"]), n=n, stored=rng.choice([1, 1, 5]), q=rng.random() < 0.7,
                k_out=rng.random() < 0.5, far=_log(rng, 1, 1048575), theta=rng.choice([1e4, 5e5, 1e6]), page=page)


def _spread(n, lo, hi):
    """n whole numbers from lo to hi in even steps (a ragged batch's lengths)."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _shared(c):
    """The prefixes of a case: (tokens, sequences) of each, from "tokens x sequences" texts."""
    return [tuple(int(x) for x in t.split("x")) for t in c["prefixes"].split()]


def _text(prefixes):
    return " ".join(f"{n}x{k}" for n, k in prefixes)


def _pages(n, page):
    return -(-n // page)


def _rows(c):
    return 1 + (c["W"] + c["G"]) * (c["N"] - 1)


def work(case):
    c = case
    if c["op"] == "attend":
        T, H, Hkv, D = _rows(c), c["heads"], c["kv_heads"], c["dim"]
        lens = _spread(c["batch"], c["lo"], c["hi"])
        seen = sum(len(_visible(c["W"], c["N"], c["G"], r)) for r in range(T))
        tokens = sum(lens) + sum(n for n, _ in _shared(c))
        rows = c["batch"] * T * (2 * H + 2 * Hkv) * D * 2
        index = 4 * (c["batch"] + sum(_pages(n, c["page"]) for n in lens) + 1
                     + sum(2 + _pages(n, c["page"]) for n, _ in _shared(c)))
        keys = sum(lens) + sum(n * k for n, k in _shared(c))
        return {"bytes": tokens * Hkv * D * 4 + rows + index, "flops": 4 * D * H * (keys * T + c["batch"] * seen)}
    n, E, H, Hkv, D = c["n"], 2 if c["dtype"] == "bf16" else 4, c["heads"], c["kv_heads"], c["dim"]
    kept = _pages(n, c["stored"])
    vec = n * Hkv * (E + (2 if c["k_out"] else 0)) + kept * Hkv * (E + 4)   # K in (and out), V in, both to the cache
    if not c["k_out"]:
        vec = kept * Hkv * (2 * E + 4)
    vec += n * H * (E + 2) if c["q"] else 0
    turned = (n * H if c["q"] else 0) + (n if c["k_out"] else kept) * Hkv
    return {"bytes": vec * D + 8 * n, "flops": 3 * turned * c["rot"]}


# ----------------------------------------------------------- what is in hand

def _vectors(n, heads, dim, gen, dtype=torch.bfloat16):
    """Keys or values as a trained model has them: roughly normal, a few
    channels several times larger, every token at its own level."""
    x = torch.randn((n, heads, dim), generator=gen, device="cuda")
    big = torch.rand((1, heads, dim), generator=gen, device="cuda") < 0.03
    x = x * torch.where(big, 4.0, 1.0) * torch.exp(0.25 * torch.randn((n, heads, 1), generator=gen, device="cuda"))
    return x.to(dtype)


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = np.random.default_rng(seed)
    i32 = lambda a: torch.tensor(np.asarray(a, dtype=np.int32), device=dev)  # noqa: E731
    H, Hkv, D, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    st = {"case": dict(c)}
    if c["op"] == "append":
        n, dtype = c["n"], torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        # one projection's rows: queries, keys and values side by side
        st["qkv"] = _vectors(n, H + 2 * Hkv, D, gen, dtype).reshape(n, -1)
        kept = np.arange(0, n, c["stored"])
        n_pages = _pages(len(kept), page) + 3
        order = host.permutation(n_pages)
        at = 1 + np.arange(len(kept))                   # the first page was begun before
        slots = np.full(n, -1)
        slots[kept] = order[at // page] * page + at % page
        start = host.integers(0, max(1, c["far"] - n + 1)) if n <= c["far"] else 0
        pos = np.minimum(start + np.arange(n) // c["stored"] + np.arange(n) % c["stored"], c["far"])
        st |= dict(slots=i32(slots), pos=i32(pos), kept=i32(kept).long(), at=i32(slots[kept]).long(),
                   k_pages=torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=dev),
                   v_pages=torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=dev))
        if c["q"]:
            st["q_out"] = torch.zeros((n, H * D), dtype=torch.bfloat16, device=dev)
        if c["k_out"]:
            st["k_out"] = torch.zeros((n, Hkv * D), dtype=torch.bfloat16, device=dev)
        if own:
            from lossless_lookahead_decoding_gb300 import KV16Cache, Rope
            st["cache"] = KV16Cache(st["k_pages"], st["v_pages"], max_pages=1)
            st["rope"] = Rope(c["rot"], theta=c["theta"], neighbours=c["pairs"] == "next")
        return st
    B, T = c["batch"], _rows(c)
    lens = host.permutation(_spread(B, c["lo"], c["hi"]))
    plens = [n for n, _ in _shared(c)]
    first = np.concatenate([[0], np.cumsum([k for _, k in _shared(c)])])
    need = [_pages(int(n), page) for n in list(lens) + plens]
    n_pages = sum(need) + 3
    order, at, rows = host.permutation(n_pages), 0, []
    for k in need:
        rows.append(order[at: at + k])
        at += k
    # what no token was written to holds bytes of any kind: all ones are NaN
    pages = [torch.full((n_pages, Hkv, page, D), -1, dtype=torch.int16, device=dev).view(torch.bfloat16) for _ in range(2)]
    for n, row in zip(list(lens) + plens, rows):
        for x in pages:
            blk = torch.full((len(row) * page, Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev)
            blk[: int(n)] = _vectors(int(n), Hkv, D, gen)
            x[i32(row).long()] = blk.reshape(len(row), page, Hkv, D).transpose(1, 2)
    mp, pmp = max(1, max(need[:B])), max([1] + need[B:])
    table, ptable = np.full((B, mp), -1), np.full((len(plens), pmp), -1)
    for b in range(B):
        table[b, : need[b]] = rows[b]
    for p in range(len(plens)):
        ptable[p, : need[B + p]] = rows[B + p]
    # q, k and v as a fused projection writes them: one row after the other
    qkv = _vectors(B * T, H + 2 * Hkv, D, gen).reshape(B * T, -1)
    st |= dict(k_pages=pages[0], v_pages=pages[1], lens=i32(lens), table=i32(table), plens=i32(plens), ptable=i32(ptable),
               first=i32(first), qkv=qkv, out=torch.zeros((B * T, H * D), dtype=torch.bfloat16, device=dev))
    if own:
        from lossless_lookahead_decoding_gb300 import KV16Cache
        st["cache"] = KV16Cache(pages[0], pages[1], max_pages=mp)
        st["ws"] = torch.empty(st["cache"].attention_bytes(B, H, c["W"], c["N"], c["G"], prefixes=len(plens),
                                                           prefix_pages=pmp), dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------ the operators

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _attend_own, "append": _append_own}[op](state)
    return {"attend": _attend, "append": _append}[op](state)


def _split(st):
    c, qkv = st["case"], st["qkv"]
    a, b = c["heads"] * c["dim"], (c["heads"] + c["kv_heads"]) * c["dim"]
    return qkv[:, :a], qkv[:, a:b], qkv[:, b:]


def _attend_own(st):
    c = st["case"]
    q, k, v = _split(st)
    st["cache"].attention(q, k, v, st["lens"], st["table"], c["W"], c["N"], c["G"], out=st["out"], workspace=st["ws"],
                          prefix_lens=st["plens"], prefix_table=st["ptable"], prefix_first=st["first"])
    return st["out"]


def _append_own(st):
    q, k, v = _split(st)
    st["cache"].append(k, v, st["slots"], positions=st["pos"], rope=st["rope"], k_out=st.get("k_out"),
                       q=q if st["case"]["q"] else None, q_out=st.get("q_out"))
    return {x: st[x] for x in ("k_pages", "v_pages", "k_out", "q_out") if x in st}


def _turn(x, pos, c):
    """x [n, heads, D] turned to positions pos: angles in 64 bits, products in 32."""
    rot = c["rot"]
    f = c["theta"] ** (-2 * torch.arange(rot // 2, device=x.device, dtype=torch.float64) / rot)
    angle = pos.double()[:, None] * f
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.float().clone()
    part = y[..., :rot]
    a, b = (part[..., : rot // 2], part[..., rot // 2:]) if c["pairs"] == "half" else (part[..., 0::2], part[..., 1::2])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    if c["pairs"] == "half":
        part[...] = torch.cat([lo, hi], -1)
    else:
        part[...] = torch.stack([lo, hi], -1).flatten(-2)
    return y.to(torch.bfloat16)


def _append(st):
    c, D, page = st["case"], st["case"]["dim"], st["case"]["page"]
    q, k, v = (x.unflatten(-1, (-1, D)) for x in _split(st))
    out = {x: st[x] for x in ("k_pages", "v_pages")}
    where = st["at"] // page, slice(None), st["at"] % page
    if c["k_out"]:
        k = _turn(k, st["pos"], c)
        out["k_out"], kept = k.reshape(c["n"], -1), k[st["kept"]]
    else:
        kept = _turn(k[st["kept"]], st["pos"][st["kept"]], c)
    st["k_pages"][where] = kept
    st["v_pages"][where] = v[st["kept"]].to(torch.bfloat16)
    if c["q"]:
        out["q_out"] = _turn(q, st["pos"], c).reshape(c["n"], -1)
    return out


def _mask(W, N, G, T, dev):
    """Which step rows (columns) each step row sees: the combined 2D-window + verification mask."""
    r, n, w = torch.arange(T, device=dev), W * (N - 1), max(W, 1)
    i, j = r[:, None], r[None]
    li, ci, lj, cj = (i - 1) // w, (i - 1) % w, (j - 1) // w, (j - 1) % w
    both = (i >= 1) & (i <= n) & (j >= 1) & (j <= n)
    see = both & (((lj == 0) & (cj <= ci)) | ((cj == ci) & (lj <= li)))
    k = N - 1
    tail = (i > n) & (j > n) & ((i - 1 - n) // k == (j - 1 - n) // k) & (j <= i)
    return see | tail | (j == 0)


def _weigh(a, v):
    """A part's softmax numerators' products with V, their sums and the rows' largest scores."""
    top = a.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(a - top)
    return torch.matmul(p, v), p.sum(-1, keepdim=True), top


def _attend(st):
    c, lens, table, qkv = st["case"], st["lens"], st["table"], st["qkv"]
    T, H, Hkv, D = _rows(c), c["heads"], c["kv_heads"], c["dim"]
    B, mp, page, R = lens.shape[0], table.shape[1], c["page"], _rows(c) * (c["heads"] // c["kv_heads"])
    x = qkv.float().reshape(B, T, H + 2 * Hkv, D)
    q = x[:, :, :H].reshape(B, T, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, R, D)
    keep = torch.arange(mp * page, device=lens.device)[None] < lens[:, None]
    whole = []
    for part, pages in enumerate((st["k_pages"], st["v_pages"])):
        y = pages[table.clamp(min=0).long()].permute(0, 2, 1, 3, 4).reshape(B, Hkv, mp * page, D).float()
        y = torch.where(keep[:, None, :, None], y, 0.0)
        own_rows = x[:, :, H + part * Hkv: H + (part + 1) * Hkv].transpose(1, 2)
        whole.append(torch.cat([y, own_rows], 2))
    see = _mask(c["W"], c["N"], c["G"], T, lens.device).repeat(H // Hkv, 1)
    see = torch.cat([keep[:, None, None].expand(B, 1, R, mp * page), see[None, None].expand(B, 1, *see.shape)], -1)
    a = torch.matmul(q, whole[0].transpose(-1, -2)) / math.sqrt(D)
    o, l, m = _weigh(torch.where(see, a, float("-inf")), whole[1])
    at = 0
    for p, (n, count) in enumerate(_shared(c)):
        used = st["ptable"][p, : _pages(n, page)].long()
        kv = [pages[used].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].float() for pages in (st["k_pages"], st["v_pages"])]
        mine = slice(at, at + count)
        rows = q[mine].transpose(0, 1).reshape(Hkv, count * R, D)
        parts = _weigh(torch.matmul(rows, kv[0].transpose(-1, -2)) / math.sqrt(D), kv[1])
        po, pl, pm = (y.reshape(Hkv, count, R, -1).transpose(0, 1) for y in parts)
        top = torch.maximum(m[mine], pm)
        f, g = torch.exp(m[mine] - top), torch.exp(pm - top)
        o[mine], l[mine] = o[mine] * f + po * g, l[mine] * f + pl * g
        at += count
    o = o / l
    return o.reshape(B, Hkv, H // Hkv, T, D).permute(0, 3, 1, 2, 4).reshape(B * T, H * D).to(torch.bfloat16)


# ------------------------------------------------- the definitions, in 64 bits

def _visible(W, N, G, r):
    """The step rows that step row r sees, listed from the branches' meaning."""
    if r == 0:
        return [0]
    if r <= W * (N - 1):
        level, col = divmod(r - 1, W)
        return [0] + [1 + a for a in range(col + 1)] + [1 + m * W + col for m in range(1, level + 1)]
    g, i = divmod(r - 1 - W * (N - 1), N - 1)
    return [0] + [1 + W * (N - 1) + g * (N - 1) + a for a in range(i + 1)]


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attend(st)


def _exact_append(st):
    c, D, page = st["case"], st["case"]["dim"], st["case"]["page"]
    rows = st["qkv"].double().cpu().numpy().reshape(c["n"], -1, D)
    pos, slots = st["pos"].cpu().numpy().astype(np.float64), st["slots"].cpu().numpy()
    H, Hkv, half = c["heads"], c["kv_heads"], c["rot"] // 2

    def turn(x):
        # pair i as a complex number, times e^(i angle)
        y, i = x.copy(), np.arange(half)
        lo, hi = (i, i + half) if c["pairs"] == "half" else (2 * i, 2 * i + 1)
        z = (x[..., lo] + 1j * x[..., hi]) * np.exp(1j * np.outer(pos, np.power(c["theta"], -i / half)))[:, None]
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    k = turn(rows[:, H: H + Hkv])
    out = {}
    for name, x in (("k_pages", k), ("v_pages", rows[:, H + Hkv:])):
        out[name] = np.zeros(tuple(st[name].shape))
        for i in np.nonzero(slots >= 0)[0]:
            out[name][slots[i] // page, :, slots[i] % page] = x[i]
    if c["k_out"]:
        out["k_out"] = k.reshape(c["n"], -1)
    if c["q"]:
        out["q_out"] = turn(rows[:, :H]).reshape(c["n"], -1)
    return out


def _exact_attend(st):
    c = st["case"]
    T, H, Hkv, D, page = _rows(c), c["heads"], c["kv_heads"], c["dim"], c["page"]
    lens, plens = st["lens"].tolist(), st["plens"].tolist()
    home = [p for p, (_, k) in enumerate(_shared(c)) for _ in range(k)]
    hidden = torch.full((T, T), float("-inf"), dtype=torch.float64)
    for r in range(T):
        hidden[r, _visible(c["W"], c["N"], c["G"], r)] = 0
    hidden = hidden.cuda()
    rows = st["qkv"].double().reshape(len(lens), T, H + 2 * Hkv, D)
    out = torch.empty((len(lens), T, H, D), dtype=torch.float64, device="cuda")

    def tokens(pages, row, n):
        return pages[row[: _pages(n, page)].long()].transpose(1, 2).reshape(-1, Hkv, D)[:n].double()

    for b, n in enumerate(lens):
        kv = []
        for part, pages in enumerate((st["k_pages"], st["v_pages"])):
            have = [tokens(pages, st["ptable"][home[b]], plens[home[b]])] if b < len(home) else []
            have += [tokens(pages, st["table"][b], n), rows[b, :, H + part * Hkv: H + (part + 1) * Hkv]]
            kv.append(torch.cat(have))
        for g in range(Hkv):
            mine = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
            a = rows[b, :, mine].transpose(0, 1) @ kv[0][:, g].T / math.sqrt(D)     # [heads of the group, T, keys]
            a[..., -T:] += hidden
            out[b, :, mine] = (torch.softmax(a, -1) @ kv[1][:, g]).transpose(0, 1)
    return out.reshape(len(lens) * T, H * D)
