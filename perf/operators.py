"""Serving operators of the 8-bit paged K/V cache: their cases, their plain forms and the library's calls.

Four operators that a serving step runs one after another:

* ``page_map``: block tables and slot maps from the requests' lengths;
* ``store``: new K and V rows quantised into the pages the slot map names;
* ``decode``: one query token per sequence over the 8-bit paged cache;
* ``prefill``: a ragged batch of query rows over the same cache, causal.

The cache holds e4m3 codes and, for every block of ``sb`` positions of a page and head, one byte e: a position's row is
code * 2^(e - 127).  ``run`` computes each operator from elementary torch operations in 32 bits, or, with ``own`` set, by
the call a user of the package makes.
"""
import math

import torch

own = False

E_MIN = -120  # smallest exponent the writer gives a block
POOL_KEYS = ("k_pages", "v_pages", "k_scales", "v_scales")

# query heads, K heads, V heads, d_k, d_v
DIFFQKV = dict(n_q=16, n_k=4, n_v=16, d_k=64, d_v=128)
GQA = dict(n_q=16, n_k=16, n_v=16, d_k=128, d_v=128)
SIGMA = dict(n_q=32, n_k=4, n_v=16, d_k=64, d_v=64)
OTHERS = (dict(n_q=8, n_k=8, n_v=8, d_k=64, d_v=64), dict(n_q=16, n_k=8, n_v=2, d_k=128, d_v=64),
          dict(n_q=24, n_k=12, n_v=8, d_k=64, d_v=128), dict(n_q=16, n_k=1, n_v=1, d_k=64, d_v=64))


def listed():
    return [
        # the table update of a decode step: one new token for each request
        dict(name="map_decode_b64", op="page_map", batch=64, lo=1, hi=32768, new_lo=1, new_hi=1, page=16, capacity=64),
        # a mixed step: many decoding requests among chunks of prompts, a padded token buffer
        dict(name="map_mixed_b256", op="page_map", batch=256, lo=0, hi=8192, new_lo=0, new_hi=127, page=16,
             capacity=32768),
        # admitting a large batch of prompts at once
        dict(name="map_prompts_b1024", op="page_map", batch=1024, lo=0, hi=2000, new_lo=1, new_hi=1023, page=32,
             capacity=1 << 20),
        # the cache write of a decode step: one row per sequence, most of them into a block that holds rows already
        dict(name="store_decode_t16", op="store", lens="decode", batch=16, lo=1, hi=511, new=1, page=16, sb=16, **DIFFQKV),
        # ragged chunks that begin in the middle of a page, at the GQA control's shape
        dict(name="store_ragged_t3704", op="store", lens="ragged", batch=8, lo=0, hi=700, new=463, page=64, sb=32, **GQA),
        # a prompt batch of 2 x 8192 rows
        dict(name="store_prompts_t16384", op="store", lens="full", batch=2, lo=0, hi=0, new=8192, page=16, sb=16,
             **DIFFQKV),
        # the smallest decode: one sequence of 512 positions
        dict(name="decode_b1_t512", op="decode", batch=1, lo=512, hi=512, page=16, sb=16, **DIFFQKV),
        # 16 sequences at 32k
        dict(name="decode_b16_t32768", op="decode", batch=16, lo=32768, hi=32768, page=16, sb=16, **DIFFQKV),
        # ragged long contexts
        dict(name="decode_ragged_b8", op="decode", batch=8, lo=16384, hi=131072, page=64, sb=64, **DIFFQKV),
        # a verified chunk of a few rows over a cached context, odd sizes
        dict(name="prefill_rows17_t1003", op="prefill", batch=4, lo=900, hi=1003, new=17, page=16, sb=16, **DIFFQKV),
        # ragged chunked prefill over cached prefixes, the paper's own head shape
        dict(name="prefill_chunks_b4", op="prefill", batch=4, lo=4000, hi=16001, new=640, page=32, sb=32, **SIGMA),
        # two prompts of 8192 from the start
        dict(name="prefill_b2_s8192", op="prefill", batch=2, lo=0, hi=0, new=8192, page=16, sb=16, **DIFFQKV),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    page = rng.choice((8, 16, 24, 32, 64, 128))
    sb = rng.choice([s for s in (1, 4, 8, 16, 32, 64, 128) if page % s == 0])
    shape = rng.choice((DIFFQKV, DIFFQKV, GQA, SIGMA) + OTHERS)
    op = rng.choice(("page_map", "store", "decode", "decode", "prefill"))
    if op == "page_map":
        batch = _log(rng, 1, 2048)
        new_hi = _log(rng, 1, min(2000, (1 << 20) // batch))
        return dict(op=op, batch=batch, lo=0, hi=_log(rng, 1, 16384), new_lo=rng.randint(0, 1), new_hi=new_hi, page=page,
                    capacity=batch * new_hi + rng.randint(0, 999))
    if op == "store":
        batch = _log(rng, 1, 64)
        return dict(op=op, lens=rng.choice(("decode", "ragged", "full")), batch=batch, lo=0, hi=_log(rng, 1, 600),
                    new=_log(rng, 1, 8192 // batch), page=page, sb=sb, **shape)
    row = shape["n_k"] * shape["d_k"] + shape["n_v"] * shape["d_v"]
    if op == "decode":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, min(131072, (524288 * 2304) // (row * batch)))
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, page=page, sb=sb, **shape)
    batch = _log(rng, 1, 8)
    new = _log(rng, 1, 2048 // batch)
    hi = _log(rng, 1, 16384 // batch)
    return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, new=new, page=page, sb=sb, **shape)


# ------------------------------------------------------------------ inputs


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _lengths(c, gen):
    """(cached positions, new rows) of every request."""
    cached = _ints(gen, c["lo"], c["hi"], c["batch"])
    if c["op"] == "page_map":
        return cached, _ints(gen, c["new_lo"], c["new_hi"], c["batch"])
    if c["op"] == "decode":
        return cached, torch.zeros(c["batch"], dtype=torch.long)
    if c["op"] == "store" and c["lens"] == "decode":
        return cached, torch.ones(c["batch"], dtype=torch.long)
    if c["op"] == "store" and c["lens"] == "full" or c["op"] == "prefill" and c["lo"] == c["hi"]:
        return cached, torch.full((c["batch"],), c["new"])
    # ragged: pairs of mean + d and mean - d rows, so that a case has one number of rows
    d = _ints(gen, 0, c["new"] - 1, c["batch"] // 2)
    odd = torch.full((c["batch"] % 2,), c["new"])
    return cached, torch.cat([c["new"] + d, c["new"] - d, odd])[torch.randperm(c["batch"], generator=gen)]


def _rows(shape, gen, channels):
    """bf16 rows [..., heads, d]: unit normal, each channel with a gain of its own (a few channels of K and V rows
    are several times the others), each position with a size of its own."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    size = torch.randn(shape[:-2], generator=gen, device="cuda").mul_(0.4).exp_()
    return x.mul_(channels).mul_(size[..., None, None]).to(torch.bfloat16)


def _channels(heads, d, gen):
    g = torch.randn((heads, d), generator=gen, device="cuda").mul_(0.3).exp_()
    return torch.where(torch.rand((heads, d), generator=gen, device="cuda") < 0.03, g * 4, g)


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, at least E_MIN (amax = m * 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(min=E_MIN)


def _pool(pages, page, sb, heads, d, gen):
    """A filled pool: codes [pages, page, heads, d] e4m3 and scale bytes [pages, page / sb, heads]."""
    codes = torch.empty((pages, page, heads, d), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((pages, page // sb, heads), dtype=torch.uint8, device="cuda")
    ch = _channels(heads, d, gen)
    step = max(1, (1 << 27) // (page * heads * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = _rows((n, page // sb, sb, heads, d), gen, ch).float()
        e = _exponent(x.abs().amax(dim=(2, 4)))
        codes[i:i + n] = torch.ldexp(x, -e[:, :, None, :, None]).reshape(n, page, heads, d).to(torch.float8_e4m3fn)
        scales[i:i + n] = (e + 127).to(torch.uint8)
    return codes, scales


def _i32(t):
    return t.to(torch.int32).cuda()


def prepare(case, seed):
    c = dict(case)
    host = torch.Generator().manual_seed(int(seed))
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    cached, new = _lengths(c, host)
    total = cached + new
    B, P = c["batch"], c["page"]
    held = -(-total // P)
    have = -(-cached // P)
    even = c["op"] == "store" and c["lens"] != "ragged" or c["lo"] == c["hi"]
    max_blocks = max(1, -(-int(c["hi"] + c.get("new_hi", (1 if even else 2) * c.get("new", 0))) // P))
    if c["op"] == "page_map":
        pages = int(held.sum()) + 64
        perm = torch.randperm(pages, generator=host)
        first = torch.cumsum(have, 0) - have
        at = torch.arange(max_blocks)[None, :]
        table = torch.where(at < have[:, None], perm[(first[:, None] + at).clamp(max=pages - 1)], torch.tensor(-1))
        cap = c["capacity"]
        s = dict(c, seq_lens=_i32(cached), new_lens=_i32(new), block_table=_i32(table), free_pages=_i32(perm[int(have.sum()):]),
                 num_pages=pages)
        s.update(query_start=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                 slot_map=torch.empty(cap, dtype=torch.int32, device="cuda"),
                 positions=torch.empty(cap, dtype=torch.int32, device="cuda"),
                 total_lens=torch.empty(B, dtype=torch.int32, device="cuda"),
                 pages_used=torch.empty(1, dtype=torch.int32, device="cuda"))
        return s
    pages = B * max_blocks + 3
    perm = torch.randperm(pages, generator=host)
    first = torch.cumsum(held, 0) - held
    at = torch.arange(max_blocks)[None, :]
    table = torch.where(at < held[:, None], perm[(first[:, None] + at).clamp(max=pages - 1)], torch.tensor(-1))
    s = dict(c, block_table=_i32(table))
    s["k_pages"], s["k_scales"] = _pool(pages, P, c["sb"], c["n_k"], c["d_k"], gen)
    s["v_pages"], s["v_scales"] = _pool(pages, P, c["sb"], c["n_v"], c["d_v"], gen)
    T = int(new.sum())
    if c["op"] == "store":
        req = torch.repeat_interleave(torch.arange(B), new)
        pos = torch.arange(T) - (torch.cumsum(new, 0) - new)[req] + cached[req]
        s["slot_map"] = _i32(table[req, pos // P] * P + pos % P)
        s["k_new"] = _rows((T, c["n_k"], c["d_k"]), gen, _channels(c["n_k"], c["d_k"], gen))
        s["v_new"] = _rows((T, c["n_v"], c["d_v"]), gen, _channels(c["n_v"], c["d_v"], gen))
        return s
    s["seq_lens"] = _i32(total)
    s["scale"] = c["d_k"] ** -0.5
    rows = B if c["op"] == "decode" else T
    s["q"] = torch.randn((rows, c["n_q"], c["d_k"]), generator=gen, device="cuda").to(torch.bfloat16)
    s["out"] = torch.empty((rows, c["n_q"], c["d_v"]), dtype=torch.bfloat16, device="cuda")
    if c["op"] == "decode":
        s["longest"] = int(total.max())
    else:
        s["query_start"] = _i32(torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(new, 0)]))
        s["most_rows"] = int(new.max())
    # scratch that a user's program keeps between its calls
    s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _page_map(s):
    B, P, cap = s["batch"], s["page"], s["capacity"]
    cached, new = s["seq_lens"].long(), s["new_lens"].long()
    total = cached + new
    have, need = (cached + P - 1) // P, (total + P - 1) // P
    take = need - have
    off = torch.cumsum(take, 0) - take
    qs = torch.cumsum(new, 0)
    at = torch.arange(s["block_table"].shape[1], device="cuda")[None, :]
    fresh = (at >= have[:, None]) & (at < need[:, None])
    given = s["free_pages"][(off[:, None] + at - have[:, None]).clamp(0, s["free_pages"].numel() - 1)]
    table = torch.where(fresh, given, s["block_table"])
    t = torch.arange(cap, device="cuda")
    req = torch.searchsorted(qs, t, right=True)
    live = req < B
    req = req.clamp(max=B - 1)
    pos = t - (qs - new)[req] + cached[req]
    page = table[req, (pos // P).clamp(0, table.shape[1] - 1)]
    none = torch.full_like(t, -1)
    start = torch.cat([torch.zeros_like(qs[:1]), qs])
    return dict(block_table=table, query_start=start.int(), slot_map=torch.where(live, page * P + pos % P, none).int(),
                positions=torch.where(live, pos, none).int(), total_lens=total.int(), pages_used=take.sum()[None].int())


def _store_side(pages, scales, x, slots):
    """Quantises rows x [T, heads, d] into codes `pages` [pages, P, heads, d] and `scales` [pages, P / sb, heads]."""
    n, P, heads, d = pages.shape
    sb = P // scales.shape[1]
    codes = pages.view(n * P // sb, sb, heads, d)
    table = scales.view(-1, heads)
    blk, row = slots // sb, slots % sb
    x = x.float()
    amax = torch.zeros(table.shape, device="cuda").scatter_reduce_(
        0, blk[:, None].expand(-1, heads), x.abs().amax(2), "amax")
    low = torch.full((table.shape[0],), sb, device="cuda", dtype=torch.long).scatter_reduce_(0, blk, row, "amin")
    need = _exponent(amax[blk])
    old = table[blk].int() - 127
    e = torch.where(low[blk][:, None] == 0, need, torch.maximum(old, need))
    # rows of the touched blocks that were there before, at the new scale
    held = codes.view(torch.uint8)[blk].view(torch.float8_e4m3fn)
    moved = torch.ldexp(held.float(), (old - e)[:, None, :, None]).to(torch.float8_e4m3fn)
    keep = torch.arange(sb, device="cuda")[None, :] >= low[blk][:, None]
    codes.view(torch.uint8)[blk] = torch.where(keep[:, :, None, None], held.view(torch.uint8), moved.view(torch.uint8))
    codes.view(torch.uint8)[blk, row] = torch.ldexp(x, -e[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    table[blk] = (e + 127).to(torch.uint8)


def _store(s):
    slots = s["slot_map"].long()
    _store_side(s["k_pages"], s["k_scales"], s["k_new"], slots)
    _store_side(s["v_pages"], s["v_scales"], s["v_new"], slots)


def _gathered(pages, scales, table):
    """The values the cache stands for, [B, max_blocks * P, heads, d] in 32 bits."""
    idx = table.long().clamp(min=0)
    B, mb = idx.shape
    n, P, heads, d = pages.shape
    sb = P // scales.shape[1]
    x = pages.view(torch.uint8)[idx].view(torch.float8_e4m3fn).float().view(B, mb * P // sb, sb, heads, d)
    e = scales[idx].view(B, mb * P // sb, 1, heads, 1).int() - 127
    return torch.ldexp(x, e).view(B, mb * P, heads, d)


def _attend(s, q, last):
    """q [B, S, n_q, d_k] over the gathered cache; row (b, r) sees positions 0 .. last[b, r]."""
    B, S, n_q, _ = q.shape
    n_k, n_v = s["n_k"], s["n_v"]
    k = _gathered(s["k_pages"], s["k_scales"], s["block_table"])
    T = k.shape[1]
    qh = q.float().permute(0, 2, 1, 3).reshape(B, n_k, n_q // n_k * S, -1)
    w = (qh @ k.permute(0, 2, 3, 1)).view(B, n_q, S, T) * s["scale"]
    del k
    w.masked_fill_(torch.arange(T, device="cuda") > last[:, None, :, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    w.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = w.sum(-1, keepdim=True)
    v = _gathered(s["v_pages"], s["v_scales"], s["block_table"])
    o = w.view(B, n_v, n_q // n_v * S, T) @ v.permute(0, 2, 1, 3)
    o = o.view(B, n_q, S, -1) / torch.where(l > 0, l, torch.ones_like(l))
    return o.permute(0, 2, 1, 3).to(torch.bfloat16)


def _decode(s):
    return _attend(s, s["q"][:, None], s["seq_lens"].long()[:, None] - 1)[:, 0]


def _prefill(s):
    start = s["query_start"].long()
    n = start[1:] - start[:-1]
    r = torch.arange(s["most_rows"], device="cuda")[None, :]
    rows = (start[:-1, None] + r).clamp(max=s["q"].shape[0] - 1)
    last = s["seq_lens"].long()[:, None] - n[:, None] + r
    o = _attend(s, s["q"][rows], last)
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(start[1:], t, right=True)
    return o[b, t - start[b]]


def run(state):
    s = state
    if own:
        import asymmetric_head_kv_b200 as ak

        if s["op"] == "page_map":
            ak.page_map(s["seq_lens"], s["new_lens"], s["block_table"], s["free_pages"], s["page"], s["num_pages"],
                        s["query_start"], s["slot_map"], s["positions"], s["total_lens"], s["pages_used"])
            return {k: s[k] for k in ("block_table", "query_start", "slot_map", "positions", "total_lens", "pages_used")}
        if s["op"] == "store":
            ak.kv8_store(s["k_new"], s["v_new"], s["slot_map"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
            return {k: s[k] for k in POOL_KEYS}
        if s["op"] == "decode":
            return ak.decode_paged_kv8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["block_table"],
                                       s["seq_lens"], scale=s["scale"], max_seq_len=s["longest"], out=s["out"],
                                       workspace=s["workspace"])
        return ak.prefill_paged_kv8(s["q"], s["query_start"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                                    s["block_table"], s["seq_lens"], scale=s["scale"], out=s["out"],
                                    workspace=s["workspace"])
    if s["op"] == "page_map":
        return _page_map(s)
    if s["op"] == "store":
        _store(s)
        return {k: s[k] for k in POOL_KEYS}
    return _decode(s) if s["op"] == "decode" else _prefill(s)


# ------------------------------------------------------------------ work and definition


def _mean(lo, hi):
    return (lo + hi) / 2


def work(case):
    c = case
    B = c["batch"]
    cached = _mean(c["lo"], c["hi"])
    if c["op"] == "page_map":
        new = _mean(c["new_lo"], c["new_hi"])
        # lengths, starts and totals; slots and positions; pages taken (list read, table written), a page read a request
        return {"bytes": B * 16 + c["capacity"] * 8 + B * (new / c["page"]) * 8 + B * 4, "flops": 0}
    row = c["n_k"] * c["d_k"] + c["n_v"] * c["d_v"]
    heads = c["n_k"] + c["n_v"]
    new = c.get("new", 0)
    if c["op"] == "store" and c["lens"] == "decode":
        new = 1
    if c["op"] == "store":
        return {"bytes": B * new * (row * 3 + 4 + heads / c["sb"]), "flops": 0}
    kv = B * (cached + new) * (row + heads / c["sb"] + 4 / c["page"])
    rows = B if c["op"] == "decode" else B * new
    pairs = B * cached if c["op"] == "decode" else B * (new * cached + new * (new + 1) / 2)
    io = rows * c["n_q"] * (c["d_k"] + c["d_v"]) * 2
    return {"bytes": kv + io, "flops": 2 * pairs * c["n_q"] * (c["d_k"] + c["d_v"])}


def _code64(y):
    """The e4m3 value nearest to y (64 bits), ties to even: steps of 2^(max(floor(log2 |y|), -6) - 3)."""
    _, x = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (x - 1).clamp(min=-6) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_store(pages, scales, x, slots):
    P, sb = pages.shape[1], pages.shape[1] // scales.shape[1]
    codes, e_of = pages.double(), scales.long() - 127
    x = x.double()
    runs = {}
    for t, slot in enumerate(slots.tolist()):
        runs.setdefault(slot // sb, []).append((slot % sb, t))
    for blk, members in runs.items():
        page, part = blk * sb // P, blk * sb % P // sb
        rows = torch.tensor([r for r, _ in members], device="cuda") + part * sb
        vals = x[torch.tensor([t for _, t in members], device="cuda")]
        a = vals.abs().amax(dim=(0, 2))
        e = torch.ceil(torch.log2(a / 448)).long()
        e = torch.where(torch.ldexp(torch.full_like(a, 448.0), e - 1) >= a, e - 1, e)
        e = torch.where(torch.ldexp(torch.full_like(a, 448.0), e) < a, e + 1, e).clamp(min=E_MIN)
        first = int(rows.min())
        if first > part * sb:
            old = e_of[page, part]
            e = torch.maximum(e, old)
            codes[page, part * sb:first] = _code64(torch.ldexp(codes[page, part * sb:first], (old - e)[None, :, None]))
        codes[page, rows] = _code64(torch.ldexp(vals, -e[None, :, None]))
        e_of[page, part] = e
    return codes, e_of + 127


def _exact_rows(s, b, n, q, first):
    """Attention of rows q [R, n_q, d_k] at positions first .. first + R - 1 over the first n cached positions."""
    P = s["page"]
    pos = torch.arange(n, device="cuda")
    page = s["block_table"][b].long()[pos // P]
    side = []
    for name in ("k", "v"):
        codes, sc = s[name + "_pages"], s[name + "_scales"]
        e = sc[page, pos % P // s["sb"]].double() - 127
        side.append(codes.view(torch.uint8)[page, pos % P].view(torch.float8_e4m3fn).double() * torch.exp2(e)[:, :, None])
    k, v = side
    out = []
    for h in range(s["n_q"]):
        w = q[:, h].double() @ k[:, h // (s["n_q"] // s["n_k"])].T * s["scale"]
        w = w.masked_fill(pos[None, :] > (first + torch.arange(q.shape[0], device="cuda"))[:, None], -math.inf)
        out.append(torch.softmax(w, dim=1) @ v[:, h // (s["n_q"] // s["n_v"])])
    return torch.stack(out, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "page_map":
        return None
    if s["op"] == "store":
        if s["k_new"].shape[0] > 20000:
            return None
        k, ke = _exact_store(s["k_pages"], s["k_scales"], s["k_new"], s["slot_map"])
        v, ve = _exact_store(s["v_pages"], s["v_scales"], s["v_new"], s["slot_map"])
        return dict(k_pages=k, v_pages=v, k_scales=ke, v_scales=ve)
    lens = s["seq_lens"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    if s["op"] == "decode":
        for b, n in enumerate(lens):
            if n:
                out[b] = _exact_rows(s, b, n, s["q"][b:b + 1], n - 1)[0]
        return out
    start = s["query_start"].tolist()
    for b, n in enumerate(lens):
        for r0 in range(start[b], start[b + 1], 2048):
            r1 = min(start[b + 1], r0 + 2048)
            out[r0:r1] = _exact_rows(s, b, n, s["q"][r0:r1], n - (start[b + 1] - r0))
    return out
