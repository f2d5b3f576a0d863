"""Cases of the page operators of the rotated low-bit KV cache: sparse decode attention (key bounds of
each page, page scores of a query, page selection, attention over the selected pages) and page
management (remapping sequences onto pages, compacting kept tokens into fresh pages).

``run`` computes one operator: in plain form as elementary torch operations on the packed bytes, or with
``own`` set through the library's entry points.  Shapes follow the benchmark's workloads: 8 kv heads of
128 with 128-token pages (16 sequences of 32K tokens, 8 of 128K) and the ragged paged batch of 64
sequences, 4 kv heads of 256, 16-token pages.
"""
import math

import torch

own = False

SCALE_BYTES = {"f32": 4, "f16": 2, "e4m3": 1, "e4m3zp": 2}
OPS = ("bounds", "scores", "select", "attn", "remap", "compact")
DEV = "cuda"


# ---------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, batch=16, hkv=8, group=4, d=128, block=64, bits=3, scale="f16", page=128,
             lo=1024, hi=32768, budget=32, sinks=1, recent=2, append=False, keep=0, beam=0)
    c.update(kw)
    return c


def listed():
    return [
        # after a prompt phase: the key bounds of every page of 16 sequences of 32K tokens
        _case("bounds-prompt", "bounds", lo=32768),
        # a decode step of the ragged batch: only the page that holds each sequence's newest token
        _case("bounds-append", "bounds", batch=64, hkv=4, d=256, page=16, hi=8192, append=True),
        # page scores of one decode step: 16 sequences of 32K tokens (256 pages each)
        _case("scores-32k", "scores", lo=32768),
        # ragged batch with small pages: up to 4,096 pages a sequence, no two alike
        _case("scores-ragged", "scores", batch=64, hkv=4, d=256, page=16, hi=65536),
        # 32 of 256 pages for each of 128 rows
        _case("select-32k", "select", lo=32768),
        # 256 of up to 4,096 pages for each of 256 rows, ragged
        _case("select-ragged", "select", batch=64, hkv=4, page=16, hi=65536, budget=256, sinks=2, recent=4),
        # one decode step over 4,096 selected tokens of each (sequence, kv head)
        _case("attn-32k", "attn", lo=32768),
        # 8 query heads per kv head, E4M3 scales, 128K tokens, an eighth of them selected
        _case("attn-128k-g8", "attn", batch=8, group=8, scale="e4m3", lo=131072, hi=131072, budget=128),
        # the ragged batch, small pages: 2,048 tokens of each (sequence, kv head) in 128 pages
        _case("attn-ragged", "attn", batch=64, hkv=4, d=256, page=16, hi=16384, budget=128),
        # every decode step: each sequence grows by one token, few need a page
        _case("remap-grow", "remap", hi=8192),
        # a beam step: 64 sequences in beams of 8, each continued from a random one of its beam
        _case("remap-beam", "remap", batch=64, beam=8, hi=4096),
        # eviction: 4,096 kept tokens of each (sequence, kv head) gathered into fresh pages
        _case("compact-4k", "compact", batch=16, lo=16384, hi=16384, keep=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(OPS)
    d, block = rng.choice(((64, 32), (64, 64), (128, 32), (128, 64), (128, 64), (256, 64), (256, 32)))
    scale = rng.choice(("f32", "f16", "f16", "e4m3", "e4m3zp"))
    page = rng.choice((16, 16, 32, 48, 64, 128))
    c = dict(op=op, batch=_log(rng, 1, 64), hkv=rng.choice((1, 2, 4, 8)), group=rng.choice((1, 2, 3, 4, 5, 8, 16)), d=d,
             block=block, bits=3 if scale == "e4m3zp" else rng.choice((2, 3, 3, 4)), scale=scale, page=page, lo=1,
             hi=_log(rng, 64, 65536), budget=1, sinks=0, recent=1, append=False, keep=0, beam=0)
    # no drawn case holds more elements than the listed 32K batch
    while 2 * c["batch"] * c["hkv"] * c["d"] * c["hi"] > 1 << 30:
        c["hi"] = max(64, c["hi"] // 2)
    if op == "select":   # rows of which a choice is made, next to short ones that are taken whole
        c["hi"] = max(c["hi"], 24 * page)
    pages = -(-c["hi"] // page)
    if op == "bounds":
        c["append"] = rng.random() < 0.3
    if op in ("select", "attn"):
        c["sinks"], c["recent"] = rng.randint(0, 2), rng.randint(1, 4)
        most = pages // 3 if op == "select" else max(1, min(pages, 8192 // page))
        c["budget"] = max(c["sinks"] + c["recent"] + (op == "select"), _log(rng, 1, most))
    if op == "remap":
        c["beam"] = rng.choice((0, 2, 3, 8))
    if op == "compact":
        c["batch"] = min(c["batch"], 32)
        c["keep"] = _log(rng, 1, max(1, min(c["hi"], 8192)))
    return c


# ---------------------------------------------------------------- inputs
def _geometry(c):
    nb, sb, cb = c["d"] // c["block"], SCALE_BYTES[c["scale"]], c["bits"] * c["d"] // 8
    header = c["page"] * nb * sb
    return nb, sb, cb, header, header + c["page"] * cb


def _fill(c, pages, g):
    """Packed records [pages, hkv, 2, record bytes] of quantised vectors: normal entries around a centre of
    their page, one magnitude per page.  At most 2**24 vectors' worth of distinct elements; the pages
    beyond repeat them in random order."""
    nb, sb, cb, header, record = _geometry(c)
    d, P = c["d"], c["page"]
    distinct = max(1, min(pages, (1 << 26) // (c["hkv"] * 2 * P * d)))
    shape = (distinct, c["hkv"], 2, P)
    x = torch.randn(*shape, d, generator=g, device=DEV)
    x += 0.5 * torch.randn(distinct, c["hkv"], 2, 1, d, generator=g, device=DEV)
    x *= torch.exp(0.4 * torch.randn(distinct, c["hkv"], 2, 1, 1, generator=g, device=DEV))
    x = x.view(*shape, nb, c["block"])
    if c["scale"] == "e4m3zp":
        lo, hi = x.amin(-1), x.amax(-1)
        s = ((hi - lo + 1e-6) / 7).to(torch.float8_e4m3fn)
        z = lo.to(torch.float8_e4m3fn)
        head = torch.stack([s, z], -1).view(torch.uint8)
        s, z = s.float()[..., None], z.float()[..., None]
        codes = torch.where(s > 0, (x - z) / s, 0.0).round().clamp(0, 7).to(torch.int32)
    else:
        top = (1 << (c["bits"] - 1)) - 1
        s = (x.abs().amax(-1) + 1e-6) / top
        s = s.to({"f32": torch.float32, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[c["scale"]])
        head = s.view(torch.uint8)
        s = s.float()[..., None]
        codes = torch.where(s > 0, x / s, 0.0).round().clamp(-top, top).to(torch.int32) & ((1 << c["bits"]) - 1)
    del x
    shifts = c["bits"] * torch.arange(8, dtype=torch.int64, device=DEV)
    words = (codes.view(*shape, d // 8, 8).to(torch.int64) << shifts).sum(-1)
    body = ((words[..., None] >> (8 * torch.arange(c["bits"], device=DEV))) & 255).to(torch.uint8)
    rec = torch.cat([head.reshape(*shape[:3], header), body.reshape(*shape[:3], record - header)], -1)
    if distinct == pages:
        return rec
    return rec[torch.randint(0, distinct, (pages,), generator=g, device=DEV)]


def _rotation(c, g):
    """Signs and unit quaternions of a rotation, and the dense matrix U = B H D made of them."""
    d = c["d"]
    signs = (torch.randint(0, 2, (d,), generator=g, device=DEV) * 2 - 1).double()
    quats = torch.randn(d // 4, 4, generator=g, device=DEV, dtype=torch.float64)
    quats = (quats / quats.norm(dim=1, keepdim=True)).float()
    return signs, quats, _matrix(signs, quats)


def _matrix(signs, quats):
    d = signs.numel()
    i = torch.arange(d, device=DEV)
    bits = (i[:, None] & i[None, :])[..., None] >> torch.arange(8, device=DEV)
    h = (1.0 - 2.0 * ((bits & 1).sum(-1) % 2).double()) / math.sqrt(d)
    q = quats.double()
    q = q / q.norm(dim=1, keepdim=True)
    a, b, e, f = q.unbind(1)
    left = torch.stack([a, -b, -e, -f, b, a, -f, e, e, f, a, -b, f, -e, b, a], 1).view(-1, 4, 4)
    return torch.block_diag(*left) @ h @ torch.diag(signs)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    P, B, hkv, d = c["page"], c["batch"], c["hkv"], c["d"]
    record = _geometry(c)[4]
    rows = 2 * B if c["op"] == "compact" else B
    maxp = -(-c["hi"] // P) + 1
    # lengths spread evenly over the range, in random order: every seed needs the same number of pages
    spread = (torch.randperm(B, generator=g, device=DEV) + 0.5) / B
    lens = (c["lo"] + ((c["hi"] - c["lo"]) * spread).round()).to(torch.int32).repeat(rows // B)
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device=DEV), maxp=maxp, rows=rows)
    if c["op"] == "compact":   # the last B rows are the destinations, with pages for the kept tokens
        lens[:B] = torch.clamp(lens[:B], min=min(c["keep"], c["hi"]))
        lens[B:] = min(c["keep"], c["hi"])
        s["keep"] = torch.stack([
            torch.rand(hkv, c["hi"], generator=g, device=DEV).masked_fill_(
                torch.arange(c["hi"], device=DEV) >= n, 2.0).argsort(-1)[:, : c["keep"]].sort(-1).values
            for n in lens[:B].tolist()]).to(torch.int32).contiguous()
        s["n_keep"] = torch.minimum(lens[B:], lens[:B]).contiguous()
        s["src_seq"] = torch.arange(B, dtype=torch.int32, device=DEV)
        s["dst_seq"] = s["src_seq"] + B
    need = (lens + P - 1) // P
    spare = B * 2 if c["op"] == "remap" else 0
    num_pages = int(need.sum()) + spare
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    used = torch.arange(maxp, device=DEV)[None, :] < need[:, None]
    table = torch.full((rows, maxp), -1, dtype=torch.int32, device=DEV)
    table[used] = order[: num_pages - spare]
    s.update(lens=lens, table=table, num_pages=num_pages)
    if c["op"] in ("bounds", "attn"):
        s["pool"] = torch.empty(num_pages + 1, hkv, 2, record, dtype=torch.uint8, device=DEV)
        s["pool"][:num_pages] = _fill(c, num_pages, g)
    elif c["op"] in ("remap", "compact"):
        # pages are moved, not read: any bytes do
        s["pool"] = torch.randint(0, 256, (num_pages + 1, hkv, 2, record), generator=g, device=DEV, dtype=torch.uint8)
    else:
        s["pool"] = torch.zeros(1, dtype=torch.uint8, device=DEV).expand(16).contiguous()
    if c["op"] in ("scores", "attn"):
        s["signs"], s["quats"], u = _rotation(c, g)
        s["U"] = u.float()
        s["q"] = torch.randn(B, hkv * c["group"], d, generator=g, device=DEV).half()
    if c["op"] == "bounds":
        s["bounds"] = torch.zeros(num_pages + 1, hkv, 2, d, dtype=torch.float16, device=DEV)
        s["first"] = lens - 1 if c["append"] else torch.zeros_like(lens)
    if c["op"] == "scores":
        # a page's bounds: a centre per page with a spread, in a magnitude of its own
        mid = 0.5 * torch.randn(num_pages, hkv, 1, d, generator=g, device=DEV)
        half = 1.5 + torch.rand(num_pages, hkv, 1, d, generator=g, device=DEV)
        size = torch.exp(0.4 * torch.randn(num_pages, hkv, 1, 1, generator=g, device=DEV))
        s["bounds"] = (torch.cat([mid - half, mid + half], 2) * size).half()
        s["scores"] = torch.empty(B, hkv, maxp, device=DEV)
    if c["op"] == "select":
        s["scores"] = 60.0 * torch.exp(0.4 * torch.randn(B, hkv, maxp, generator=g, device=DEV))
        past = torch.arange(maxp, device=DEV)[None, None, :] >= need[:, None, None]
        s["scores"].masked_fill_(past, -math.inf)
        s["pages"] = torch.empty(B, hkv, c["budget"], dtype=torch.int32, device=DEV)
        s["counts"] = torch.empty(B, hkv, dtype=torch.int32, device=DEV)
    if c["op"] == "attn":
        # the newest page and a random choice of the others, ascending
        key = torch.rand(B, hkv, maxp, generator=g, device=DEV)
        at = torch.arange(maxp, device=DEV)
        key = torch.where(at >= need[:, None, None], 3.0, torch.where(at == need[:, None, None] - 1, -1.0, key))
        take = key.argsort(-1)[..., : c["budget"]]
        if take.shape[-1] < c["budget"]:
            take = torch.cat([take, take.new_full((B, hkv, c["budget"] - take.shape[-1]), maxp)], -1)
        take = torch.where(take < need[:, None, None], take, maxp).sort(-1).values
        s["pages"] = torch.where(take < maxp, take, -1).to(torch.int32)
        s["counts"] = (s["pages"] >= 0).sum(-1).to(torch.int32)
        s["out"] = torch.empty(B, hkv * c["group"], d, dtype=torch.float16, device=DEV)
    if c["op"] == "remap":
        at = torch.arange(B, device=DEV)
        if c["beam"]:
            pick = (at // c["beam"]) * c["beam"] + torch.randint(0, c["beam"], (B,), generator=g, device=DEV)
            s["src"] = pick.clamp_(max=B - 1).to(torch.int32)
        else:
            s["src"] = at.to(torch.int32)
        s["new_lens"] = torch.clamp(lens[s["src"].long()] + 1, max=maxp * P).to(torch.int32)
        s["table_out"] = torch.empty_like(table)
        s["lens_out"] = torch.empty_like(lens)
    return s


# ---------------------------------------------------------------- the library's calls
def _library(s):
    """The description, cache, rotation and workspace that a program makes once and keeps."""
    import hadamard_rotated_bit_kvq3_gb300 as K
    c = s["case"]
    desc = K.CacheDesc(c["d"], c["hkv"], c["block"], c["bits"], K.SCALE_TYPES[c["scale"]], 1e-6, c["page"],
                       s["rows"], s["maxp"], 0, s["num_pages"])
    cache = K.Cache(s["pool"].data_ptr(), s["table"].data_ptr(), s["lens"].data_ptr())
    rot = ws = None
    if "U" in s:
        rot = K.kvq3_rotation_create_from_params(c["d"], s["signs"].cpu().numpy(), s["quats"].cpu().numpy())
    if c["op"] == "remap":
        ws = torch.empty(K.kvq3_remap_workspace_size(desc), dtype=torch.uint8, device=DEV)
    # what a pass returns: the pages that the cache knows, without the spare one behind them
    whole = s["bounds"][: s["num_pages"]] if c["op"] == "bounds" else s["pool"][: s["num_pages"]]
    return K, desc, cache, rot, ws, whole


def _run_own(s):
    if "library" not in s:
        s["library"] = _library(s)
    K, desc, cache, rot, ws, whole = s["library"]
    c, op = s["case"], s["case"]["op"]
    if op == "bounds":
        K.kvq3_key_bounds(desc, cache, s["first"], s["bounds"], s["status"])
        return whole
    if op == "scores":
        K.kvq3_page_scores(rot, desc, cache, s["bounds"], s["q"], s["scores"], s["status"])
        return s["scores"]
    if op == "select":
        K.kvq3_page_select(desc, cache, s["scores"], c["budget"], c["sinks"], c["recent"], s["pages"], s["counts"],
                           s["status"])
        return s["pages"], s["counts"]
    if op == "attn":
        K.kvq3_decode_attn_pages(rot, desc, cache, s["q"], s["pages"], s["counts"], s["out"], 0.0, s["status"])
        return s["out"]
    if op == "remap":
        K.kvq3_remap(desc, cache, s["src"], s["new_lens"], s["table_out"], s["lens_out"], ws, s["status"])
        return s["table_out"], s["lens_out"], whole
    K.kvq3_compact(desc, cache, s["src_seq"], s["dst_seq"], s["keep"], s["n_keep"], s["status"])
    return whole


# ---------------------------------------------------------------- the plain forms
def _values(c, rec):
    """Records [..., record bytes] -> rotated-domain vectors [..., P, d] in 32 bits."""
    nb, sb, cb, header, record = _geometry(c)
    lead, P, bits = rec.shape[:-1], c["page"], c["bits"]
    head = rec[..., :header].contiguous()
    body = rec[..., header:].reshape(*lead, P, c["d"] // 8, bits).to(torch.int32)
    word = (body << (8 * torch.arange(bits, device=DEV, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    field = (word[..., None] >> (bits * torch.arange(8, device=DEV, dtype=torch.int32))) & ((1 << bits) - 1)
    field = field.reshape(*lead, P, nb, c["block"])
    if c["scale"] == "e4m3zp":
        sz = head.view(torch.float8_e4m3fn).float().reshape(*lead, P, nb, 2)
        x = field * sz[..., :1] + sz[..., 1:]
    else:
        kind = {"f32": torch.float32, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[c["scale"]]
        scale = head.view(kind).float().reshape(*lead, P, nb, 1)
        half = 1 << (bits - 1)
        x = ((field ^ half) - half) * scale
    return x.reshape(*lead, P, c["d"])


def _run_bounds(s):
    c, P = s["case"], s["case"]["page"]
    width = 1 if c["append"] else s["maxp"]
    lens, first = s["lens"].long(), s["first"].long()
    lp = first[:, None] // P + torch.arange(width, device=DEV)
    valid = lp * P < lens[:, None]
    page = torch.where(valid, s["table"].long().gather(1, lp.clamp(max=s["maxp"] - 1)), s["num_pages"]).reshape(-1)
    x = _values(c, s["pool"][page, :, 0])                                  # [B * width, hkv, P, d]
    held = (lp.reshape(-1, 1) * P + torch.arange(P, device=DEV) < lens.repeat_interleave(width)[:, None])[:, None, :, None]
    lo = torch.where(held, x, math.inf).amin(2)
    hi = torch.where(held, x, -math.inf).amax(2)
    s["bounds"][page] = torch.stack([lo, hi], 2).half()
    return s["bounds"][: s["num_pages"]]


def _run_scores(s):
    c = s["case"]
    B, hkv, G, d = c["batch"], c["hkv"], c["group"], c["d"]
    page = s["table"].long().clamp(min=0)
    b = s["bounds"][page].float()                                          # [B, maxp, hkv, 2, d]
    q = (s["q"].float() @ s["U"].T).view(B, 1, hkv, G, d)
    best = torch.maximum(q * b[:, :, :, :1], q * b[:, :, :, 1:]).sum(-1).amax(-1)
    there = torch.arange(s["maxp"], device=DEV)[None, :] * c["page"] < s["lens"].long()[:, None]
    return torch.where(there[..., None], best, -math.inf).permute(0, 2, 1).contiguous()


def _run_select(s):
    c = s["case"]
    n = ((s["lens"].long() + c["page"] - 1) // c["page"])[:, None, None]
    at = torch.arange(s["maxp"], device=DEV)
    # forced pages first, then by score, then what does not exist; ties to the lower page
    forced = (at < c["sinks"]) | (at >= n - c["recent"])
    key = torch.where(forced, math.inf, s["scores"])
    rank = torch.where(at >= n, 2, torch.where(forced, 0, 1)).expand_as(key)
    order = key.sort(stable=True, dim=-1, descending=True).indices
    order = order.gather(-1, rank.gather(-1, order).sort(stable=True, dim=-1).indices)[..., : c["budget"]]
    chosen = torch.where(order < n, order, s["maxp"]).sort(-1).values
    chosen = torch.nn.functional.pad(chosen, (0, c["budget"] - chosen.shape[-1]), value=s["maxp"])
    pages = torch.where(chosen < s["maxp"], chosen, -1).to(torch.int32)
    return pages, (pages >= 0).sum(-1).to(torch.int32)


def _run_attn(s):
    c = s["case"]
    B, hkv, G, d, P = c["batch"], c["hkv"], c["group"], c["d"], c["page"]
    lp = s["pages"].long()                                                 # [B, hkv, row]
    page = s["table"].long()[torch.arange(B, device=DEV)[:, None, None], lp.clamp(min=0)].clamp(min=0)
    x = _values(c, s["pool"][page, torch.arange(hkv, device=DEV)[None, :, None]])   # [B, hkv, row, 2, P, d]
    pos = lp[..., None] * P + torch.arange(P, device=DEV)
    held = ((lp[..., None] >= 0) & (pos < s["lens"].long()[:, None, None, None])).reshape(B, hkv, 1, -1)
    k, v = x[:, :, :, 0].reshape(B, hkv, -1, d), x[:, :, :, 1].reshape(B, hkv, -1, d)
    q = (s["q"].float() @ s["U"].T).view(B, hkv, G, d)
    logit = torch.where(held, (q @ k.transpose(-1, -2)) / math.sqrt(d), -math.inf)
    w = torch.exp(logit - logit.amax(-1, keepdim=True))
    y = (w @ v) / w.sum(-1, keepdim=True)
    return (y @ s["U"]).reshape(B, hkv * G, d).half()


def _run_remap(s):
    c, P, B, N = s["case"], s["case"]["page"], s["case"]["batch"], s["num_pages"]
    nb, sb, cb, header, record = _geometry(c)
    src, at = s["src"].long(), torch.arange(s["maxp"], device=DEV)
    old = s["table"].long()[src]
    held = torch.minimum(s["lens"].long()[src], s["new_lens"].long())      # tokens that stay
    full, tail = held // P, held % P
    shared = at < full[:, None]
    # a whole page may be shared; a part-filled one has one owner, the lowest row, unless it is shared whole
    whole = torch.zeros(N + 1, dtype=torch.bool, device=DEV)
    whole[torch.where(shared, old, N)] = True
    tail_page = torch.where(tail > 0, old.gather(1, full.clamp(max=s["maxp"] - 1)[:, None])[:, 0], N)
    owner = torch.full((N + 1,), B, dtype=torch.int64, device=DEV)
    owner.scatter_reduce_(0, tail_page, torch.arange(B, device=DEV), "amin")
    keeps = (tail > 0) & ~whole[tail_page] & (owner[tail_page] == torch.arange(B, device=DEV))
    taken = whole[:N].clone()
    taken[torch.where(keeps, tail_page, 0)] |= keeps
    # the other entries take the lowest free pages, row by row
    wanted = (at * P < s["new_lens"].long()[:, None]) & (at >= (full + keeps)[:, None])
    rank = wanted.reshape(-1).cumsum(0).view_as(wanted) - 1
    free = taken.to(torch.int8).sort(stable=True).indices
    fresh = free[rank.clamp(min=0, max=N - 1)]
    table = torch.where(shared | (keeps[:, None] & (at == full[:, None])), old, torch.where(wanted, fresh, -1))
    copies = (tail > 0) & ~keeps
    into = torch.where(copies, table.gather(1, full.clamp(max=s["maxp"] - 1)[:, None])[:, 0], N)
    slot = torch.arange(P, device=DEV) < tail[:, None]
    used = torch.cat([slot.repeat_interleave(nb * sb, 1), slot.repeat_interleave(cb, 1)], 1)[:, None, None, :]
    s["pool"][into] = torch.where(used, s["pool"][tail_page], s["pool"][into])
    return table.to(torch.int32), held.to(torch.int32), s["pool"][:N]


def _run_compact(s):
    c, P, N = s["case"], s["case"]["page"], s["num_pages"]
    nb, sb, cb, header, record = _geometry(c)
    head = s["pool"][..., :header].unflatten(-1, (P, nb * sb))             # views: [page, hkv, 2, slot, bytes]
    body = s["pool"][..., header:].unflatten(-1, (P, cb))
    keep = s["keep"].long()                                                # [n, hkv, kept]
    i = torch.arange(keep.shape[-1], device=DEV)
    valid = i < s["n_keep"].long()[:, None, None]
    old, new = s["table"].long()[s["src_seq"].long()], s["table"].long()[s["dst_seq"].long()]
    src = old[:, None, :].expand(-1, keep.shape[1], -1).gather(2, keep // P)
    dst = torch.where(valid, new[:, None, :].gather(2, (i // P).expand(keep.shape[0], 1, -1)), N)
    h = torch.arange(c["hkv"], device=DEV)[None, :, None].expand_as(keep)
    to = (i % P).expand_as(keep)
    src = torch.where(valid, src, N)
    dst = dst.expand_as(keep)
    for part in (head, body):
        part[dst, h, :, to] = part[src, h, :, keep % P]
    return s["pool"][:N]


PLAIN = dict(bounds=_run_bounds, scores=_run_scores, select=_run_select, attn=_run_attn, remap=_run_remap,
             compact=_run_compact)


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    c = case
    nb, sb, cb, header, record = _geometry(c)
    B, hkv, G, d, P = c["batch"], c["hkv"], c["group"], c["d"], c["page"]
    token = nb * sb + cb                                   # packed bytes of one key or value vector
    mean = (c["lo"] + c["hi"]) / 2
    pages = B * (mean / P + 0.5)                           # pages of the batch, the last ones part filled
    if c["op"] == "bounds":
        tokens, touched = (B * P / 2, B) if c["append"] else (B * mean, pages)
        return {"bytes": tokens * hkv * token + touched * hkv * 4 * d + 4 * touched, "flops": 2.0 * tokens * hkv * d}
    if c["op"] == "scores":
        return {"bytes": pages * hkv * (4 * d + 4) + 4 * pages + 2 * B * hkv * G * d, "flops": 4.0 * pages * hkv * G * d}
    if c["op"] == "select":
        return {"bytes": 4.0 * pages * hkv + 4 * B * hkv * (c["budget"] + 1), "flops": pages * hkv}
    if c["op"] == "attn":
        tokens = B * hkv * max(1.0, min(mean, (c["budget"] - 0.5) * P))
        return {"bytes": tokens * 2 * token + 4 * B * hkv * c["budget"] + 4 * B * hkv * G * d, "flops": 4.0 * tokens * G * d}
    if c["op"] == "remap":
        k = c["beam"]
        copies = B * (1 - (1 - (1 - 1 / k) ** k)) if k else 0
        return {"bytes": 2 * 4 * pages + copies * P / 2 * 2 * hkv * 2 * token + 16 * B, "flops": pages}
    tokens = B * hkv * min(c["keep"], c["hi"])
    return {"bytes": tokens * (4 * token + 4), "flops": tokens}


# ---------------------------------------------------------------- 64 bits, from the definitions
def _exact_vectors(c, rec):
    """One record batch [n, record bytes] -> [n, P, d] in 64 bits, bit by bit."""
    nb, sb, cb, header, record = _geometry(c)
    n, P, d, bits = rec.shape[0], c["page"], c["d"], c["bits"]
    stream = (rec[:, header:].reshape(n, P, cb, 1) >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1
    stream = stream.reshape(n, P, d, bits)
    code = torch.zeros(n, P, d, dtype=torch.float64, device=DEV)
    for k in range(bits):
        sign = -1.0 if k == bits - 1 and c["scale"] != "e4m3zp" else 1.0
        code += sign * float(1 << k) * stream[..., k].double()
    head = rec[:, :header].contiguous()
    if c["scale"] == "e4m3zp":
        sz = head.view(torch.float8_e4m3fn).double().reshape(n, P, nb, 2)
        return code * sz[..., 0].repeat_interleave(c["block"], -1) + sz[..., 1].repeat_interleave(c["block"], -1)
    kind = {"f32": torch.float32, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[c["scale"]]
    return code * head.view(kind).double().reshape(n, P, nb).repeat_interleave(c["block"], -1)


def exact(case, seed):
    """The floating outputs in 64 bits; whole-number outputs (selections, tables, moved bytes) have none."""
    c = dict(case)
    if c["op"] in ("select", "remap", "compact"):
        return None
    s = prepare(case, seed)
    P, B, hkv, G, d = c["page"], c["batch"], c["hkv"], c["group"], c["d"]
    lens = s["lens"].tolist()
    if c["op"] == "bounds":
        out = torch.zeros(s["num_pages"], hkv, 2, d, dtype=torch.float64, device=DEV)
        for b, n in enumerate(lens):
            for p0 in range((n - 1) // P if c["append"] else 0, -(-n // P), 64):
                p1 = min(-(-n // P), p0 + 64)
                ids = s["table"][b, p0:p1].long()
                for h in range(hkv):
                    x = _exact_vectors(c, s["pool"][ids, h, 0]).reshape(-1, d)
                    last = n - p0 * P
                    x = torch.cat([x[:last], x[min(last, len(x)) - 1].expand(max(0, len(x) - last), d)])
                    x = x.reshape(p1 - p0, P, d)
                    out[ids, h, 0], out[ids, h, 1] = x.min(1).values, x.max(1).values
        return out
    u = _matrix(s["signs"], s["quats"])
    q = torch.einsum("ij,bhj->bhi", u, s["q"].double()).reshape(B, hkv, G, d)
    if c["op"] == "scores":
        out = torch.full((B, hkv, s["maxp"]), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(lens):
            ids = s["table"][b, : -(-n // P)].long()
            lo, hi = s["bounds"][ids, :, 0].double(), s["bounds"][ids, :, 1].double()
            best = torch.einsum("hgd,phd->hpg", q[b].clamp(min=0), hi) + torch.einsum("hgd,phd->hpg", q[b].clamp(max=0), lo)
            out[b, :, : len(ids)] = best.max(-1).values
        return out
    out = torch.empty(B, hkv, G, d, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        for h in range(hkv):
            lp = s["pages"][b, h, : int(s["counts"][b, h])].long()
            rec = s["pool"][s["table"][b][lp].long(), h]
            held = (lp[:, None] * P + torch.arange(P, device=DEV) < n).reshape(-1)
            k = _exact_vectors(c, rec[:, 0]).reshape(-1, d)[held]
            v = _exact_vectors(c, rec[:, 1]).reshape(-1, d)[held]
            out[b, h] = torch.softmax(q[b, h] @ k.T / math.sqrt(d), -1) @ v
    return torch.einsum("bhgi,ij->bhgj", out, u).reshape(B, hkv * G, d)
