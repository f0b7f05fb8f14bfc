"""A decode step's 4-bit layers with group scales and its paged key-value cache: cases, inputs, plain forms and work.

Kinds of case (the mat-vec: gemv, swiglu; attention: attend; the cache's rows: append; its pages: fork, compact):
  gemv     y = W x + b, W in 4-bit codes with a binary16 scale (and a zero point) per group of weights
  swiglu   silu(gate) * up of two such matrices
  attend   attention of one new token per sequence over a paged cache (binary16, or 8 bits with a scale per row)
  append   new tokens' K and V written into their pages; "replace": a finished sequence's pages go back and a new one's are taken before
  fork     the last step's forks are freed, sequences forked anew: whole pages shared, the last page copied
  compact  live pages moved to the front of the pool
"""
import math

import torch

own = False

F32, F16, I8 = "f32", "f16", "i8row"
TYPES = {F32: torch.float32, F16: torch.float16}
LONGEST = 131071


def listed():
    return [
        # the O projection of a decode step, one token: latency
        dict(name="gemv 1x896x896", kind="gemv", batch=1, out=896, inf=896, group=128, zeros=False, bias=False),
        # the output head for eight sequences: nothing but weights
        dict(name="gemv 8x151936x896", kind="gemv", batch=8, out=151936, inf=896, group=128, zeros=True, bias=False),
        # gate and up of one token, small groups
        dict(name="swiglu 1x4864x896", kind="swiglu", batch=1, out=4864, inf=896, group=32, zeros=True),
        # gate and up of a wider layer for five sequences, odd rows
        dict(name="swiglu 5x11009x4096", kind="swiglu", batch=5, out=11009, inf=4096, group=64, zeros=True),
        # the first tokens of one answer: latency
        dict(name="attend 1x97 f16", kind="attend", form=F16, rows=1, longest=97, kv=2, g=7, d=64, page=16, io=F32),
        # one long document, its cache in binary16
        dict(name="attend 1x131071 f16", kind="attend", form=F16, rows=1, longest=LONGEST, kv=8, g=4, d=128, page=64, io=F16),
        # a batch of sequences of all lengths, cache in 8 bits, small pages
        dict(name="attend 48x8191 i8", kind="attend", form=I8, rows=48, longest=8191, kv=8, g=4, d=128, page=16, io=F16),
        # a decode step's new tokens
        dict(name="append 64x1 f16", kind="append", form=F16, seqs=64, new=1, replace=False, kv=2, d=64, page=16, io=F32),
        # two prompts in the slots of finished sequences, cache in 8 bits
        dict(name="append 2x1021 i8", kind="append", form=I8, seqs=2, new=1021, replace=True, kv=8, d=128, page=32, io=F16),
        # four samples of one prompt
        dict(name="fork 1 to 4", kind="fork", parents=1, each=4, length=1000, layers=24, kv=2, d=64, page=16),
        # a beam step of sixteen sequences with four beams, long pages
        dict(name="fork 16 to 64", kind="fork", parents=16, each=4, length=777, layers=24, kv=2, d=64, page=256),
        # a pool with a third of its pages given back
        dict(name="compact 2560 pages", kind="compact", pages=2560, live=1700, moves=500, layers=24, kv=2, d=64, page=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        kind = rng.choice(["gemv", "swiglu", "attend", "append", "fork", "compact"])
        heads = dict(kv=rng.choice([1, 2, 4, 8, 12]), d=rng.choice([32, 64, 96, 128, 192, 256]), page=rng.choice([8, 16, 32, 64, 128, 256]))
        if kind in ("gemv", "swiglu"):
            c = dict(kind=kind, batch=rng.randint(1, 8), out=_log(rng, 64, 151936 if kind == "gemv" else 14336),
                     inf=32 * _log(rng, 8, 256), group=rng.choice([32, 64, 128, 256]), zeros=rng.random() < 0.5)
            if kind == "gemv":
                c["bias"] = rng.random() < 0.5
        elif kind == "attend":
            c = dict(kind=kind, form=rng.choice([F16, I8]), rows=_log(rng, 1, 64), longest=_log(rng, 1, LONGEST),
                     g=rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), io=rng.choice([F32, F16]), **heads)
        elif kind == "append":
            c = dict(kind=kind, form=rng.choice([F16, I8]), seqs=_log(rng, 1, 64), new=_log(rng, 1, 2048), replace=rng.random() < 0.5,
                     io=rng.choice([F32, F16]), **heads)
        elif kind == "fork":
            c = dict(kind=kind, parents=_log(rng, 1, 16), each=rng.randint(1, 6), length=_log(rng, 1, 2048),
                     layers=rng.choice([1, 12, 24]), **heads)
        else:
            pages = _log(rng, 16, 4096)
            live = rng.randint(pages // 4, pages - 1)
            c = dict(kind=kind, pages=pages, live=live, moves=rng.randint(0, min(live, pages - live)), layers=rng.choice([1, 12, 24]),
                     **heads)
        w = work(c)["bytes"]
        if w <= most and _pool_bytes(c) <= 2 * most and (kind != "attend" or c["rows"] * c["longest"] * c["kv"] * c["d"] <= 1 << 29):
            return c


def _lengths(c):
    """Tokens of each sequence in the cache (the new one among them): spread from one token to the longest."""
    if c["kind"] == "attend":
        return [max(1, round(c["longest"] * (1.0 if r == 0 else (r * 0.6180339887) % 1.0))) for r in range(c["rows"])]
    if c["kind"] == "append":
        return [c["new"] + (0 if c["replace"] else (37 * s) % 300) for s in range(c["seqs"])]
    if c["kind"] == "fork":
        return [max(1, c["length"] - 5 * p) for p in range(c["parents"])]
    return []


def _pages_of(c, tokens):
    return -(-tokens // c["page"])


def _row_bytes(c):
    """One token's K (or V) of all heads of one layer."""
    return c["kv"] * (c["d"] + 4 if c.get("form") == I8 else 2 * c["d"])


def _pool_pages(c):
    if c["kind"] == "compact":
        return c["pages"]
    used = sum(_pages_of(c, n) for n in _lengths(c))
    return used + (c["parents"] * c["each"] + 3 if c["kind"] == "fork" else 3)


def _pool_bytes(c):
    if c["kind"] in ("gemv", "swiglu"):
        return 0
    return 2 * c.get("layers", 1) * _pool_pages(c) * c["page"] * _row_bytes(c)


def work(case):
    c = case
    if c["kind"] in ("gemv", "swiglu"):
        groups = -(-c["inf"] // c["group"])
        mats = 2 if c["kind"] == "swiglu" else 1
        matrix = c["out"] * (c["inf"] // 2 + groups * (3 if c["zeros"] else 2))
        return {"bytes": mats * matrix + 4 * c["batch"] * (c["inf"] + c["out"]) + (4 * c["out"] if c.get("bias") else 0),
                "flops": 2 * mats * c["batch"] * c["out"] * c["inf"]}
    size = 4 if c.get("io") == F32 else 2
    if c["kind"] == "attend":
        tokens, heads = sum(_lengths(c)), c["kv"] * c["g"]
        return {"bytes": 2 * tokens * _row_bytes(c) + 2 * c["rows"] * heads * c["d"] * size
                + 4 * sum(_pages_of(c, n) for n in _lengths(c)) + 4 * c["rows"], "flops": 4 * tokens * heads * c["d"]}
    if c["kind"] == "append":
        rows = c["seqs"] * c["new"]
        return {"bytes": 2 * rows * (c["kv"] * c["d"] * size + _row_bytes(c)) + 8 * rows, "flops": 2 * rows * c["kv"] * c["d"]}
    page = c["page"] * _row_bytes(c)
    if c["kind"] == "fork":
        whole = sum(c["each"] * (n // c["page"]) for n in _lengths(c))
        part = sum(c["each"] for n in _lengths(c) if n % c["page"])
        return {"bytes": 4 * c["layers"] * part * page + 12 * (whole + part) + 4 * _pool_pages(c), "flops": whole + part}
    return {"bytes": 4 * c["layers"] * c["moves"] * page + 8 * c["live"] + 8 * c["pages"], "flops": c["live"]}


def _packed(gen, c):
    """Codes of a trained matrix in groups: normal weights, the scale from the group's spread, the zero point near the middle."""
    groups = -(-c["inf"] // c["group"])
    m = dict(packed=torch.randint(0, 256, (c["out"], c["inf"] // 2), generator=gen, device="cuda", dtype=torch.uint8),
             scales=((torch.rand(c["out"], groups, generator=gen, device="cuda") + 0.5) * 0.006).half(), zeros=None)
    if c["zeros"]:
        m["zeros"] = torch.randint(5, 11, (c["out"], groups), generator=gen, device="cuda", dtype=torch.uint8)
    return m


def _i8_rows(values):
    """8-bit codes and scales of rows (here without the framework's quantizer)."""
    s = (values.abs().amax(-1).double() / 127).float()
    return (values.double() / s.double().unsqueeze(-1)).round().clamp(-127, 127).to(torch.int8), s


def _pool(gen, c, layers, pages):
    """K and V pages [layers][pages][kv][page][d], filled as a running program's are."""
    shape = (layers, pages, c["kv"], c["page"], c["d"])
    p = dict(k_scales=None, v_scales=None)
    for x in "kv":
        if c.get("form") == I8:
            p[x] = torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
            p[x + "_scales"] = (torch.rand(shape[:-1], generator=gen, device="cuda") + 0.5) * (3 / 127)
        else:
            p[x] = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    return p


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["kind"] in ("gemv", "swiglu"):
        s["x"] = torch.randn(c["batch"], c["inf"], generator=gen, device="cuda")
        loud = torch.randint(0, c["inf"], (max(1, c["inf"] // 128),), generator=gen, device="cuda")
        s["x"][:, loud] *= 8.0   # a few channels are much larger, as hidden states have them
        s["mats"] = [_packed(gen, c) for _ in range(2 if c["kind"] == "swiglu" else 1)]
        s["bias"] = torch.randn(c["out"], generator=gen, device="cuda") if c.get("bias") else None
        s["y"] = torch.empty(c["batch"], c["out"], device="cuda")
        return s
    lengths, pages, layers = _lengths(c), _pool_pages(c), c.get("layers", 1)
    s.update(_pool(gen, c, layers, pages))
    mixed = torch.randperm(pages, generator=gen, device="cuda").int()   # pages come in no order
    if c["kind"] == "compact":
        # live pages: `moves` of them past the first `live` places, held by 64-page sequences
        front = torch.randperm(c["live"], generator=gen, device="cuda")[:c["live"] - c["moves"]]
        back = c["live"] + torch.randperm(pages - c["live"], generator=gen, device="cuda")[:c["moves"]]
        used = torch.cat([front, back])[torch.randperm(c["live"], generator=gen, device="cuda")].int()
        lengths = [min(64, c["live"] - at) * c["page"] for at in range(0, c["live"], 64)]
        width = 64
    else:
        used = mixed[:sum(_pages_of(c, n) for n in lengths)]
        width = max(_pages_of(c, n) for n in lengths) + 1
    slots = len(lengths) * (1 + c["each"]) if c["kind"] == "fork" else len(lengths)
    s["table"] = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(lengths):
        m = _pages_of(c, n)
        s["table"][r, :m] = used[at:at + m]
        at += m
    s["lengths"] = torch.tensor(lengths + [0] * (slots - len(lengths)), dtype=torch.int32, device="cuda")
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["refs"][used.long()] = 1
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if c["kind"] == "attend":
        heads = c["kv"] * c["g"]
        # the fused QKV projection's output, whose query part is read; some tokens matter much more than others
        s["qkv"] = (3 * torch.randn(c["rows"], (heads + 2 * c["kv"]) * c["d"], generator=gen, device="cuda")).to(TYPES[c["io"]])
        s["y"] = torch.empty(c["rows"], heads, c["d"], dtype=TYPES[c["io"]], device="cuda")
    if c["kind"] == "append":
        rows = c["seqs"] * c["new"]
        s["kv_new"] = torch.randn(rows, 2 * c["kv"] * c["d"], generator=gen, device="cuda").to(TYPES[c["io"]])
        s["seq_ids"] = torch.arange(c["seqs"], device="cuda", dtype=torch.int32).repeat_interleave(c["new"])
        s["positions"] = torch.cat([torch.arange(n - c["new"], n, device="cuda", dtype=torch.int32) for n in lengths])
        s["slots"] = torch.arange(c["seqs"], device="cuda", dtype=torch.int32)
        s["counts"] = torch.full((c["seqs"],), c["new"], device="cuda", dtype=torch.int32)
        if c["form"] == I8:
            s["values"] = [torch.empty(s["k"].shape, device="cuda") for _ in range(2)]
    if c["kind"] == "fork":
        s["parents"] = torch.arange(c["parents"], device="cuda", dtype=torch.int32).repeat_interleave(c["each"])
        s["children"] = torch.arange(c["parents"], slots, device="cuda", dtype=torch.int32)
    if c["kind"] == "compact":
        s["before"] = [s["table"].clone(), s["refs"].clone()]   # as the program left them, to be compacted in every pass
    if own:
        _handles(s)
    return s


def _handles(s):
    import dequantize_mat_vec_amd as dmv
    c = s["case"]
    if c["kind"] in ("gemv", "swiglu"):
        return
    layers, pages = s["k"].shape[:2]
    s["cache"] = dmv.kv_cache(c.get("form", F16), layers, pages, c["page"], c["kv"], c["d"], s["k"], s["v"], s["k_scales"],
                              s["v_scales"])
    s["seqs"] = dmv.kv_table(s["table"], s["lengths"], s["refs"])
    need = 0
    if c["kind"] == "attend":
        need = dmv.pesti_attn_paged_workspace_bytes(s["cache"], c["rows"], c["kv"] * c["g"], c["longest"])
    elif c["kind"] in ("fork", "compact"):
        need = dmv.pesti_cache_workspace_bytes(s["cache"], s["seqs"])
    s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None


def _own(s):
    import dequantize_mat_vec_amd as dmv
    c = s["case"]
    if c["kind"] == "gemv":
        m = s["mats"][0]
        dmv.pesti_gemv_i4group(c["out"], c["inf"], c["group"], m["packed"], m["scales"], m["zeros"], s["x"], s["y"], s["bias"],
                               c["batch"])
        return s["y"]
    if c["kind"] == "swiglu":
        g, u = s["mats"]
        dmv.pesti_gemv_i4group_swiglu(c["out"], c["inf"], c["group"], g["packed"], g["scales"], g["zeros"], u["packed"],
                                      u["scales"], u["zeros"], s["x"], s["y"], c["batch"])
        return s["y"]
    if "cache" not in s:
        _handles(s)
    cache, seqs = s["cache"], s["seqs"]
    if c["kind"] == "attend":
        dmv.pesti_attn_paged(cache, seqs, 0, c["rows"], c["kv"] * c["g"], s["qkv"], s["y"], c["d"] ** -0.5,
                             q_stride=s["qkv"].shape[1], max_length=c["longest"], workspace=s["workspace"])
        return s["y"]
    if c["kind"] == "append":
        n = c["kv"] * c["d"]
        if c["replace"]:
            dmv.pesti_cache_free(cache, seqs, c["seqs"], s["slots"])
            dmv.pesti_cache_extend(cache, seqs, c["seqs"], s["slots"], s["counts"], s["status"])
        dmv.pesti_cache_append(cache, seqs, 0, c["seqs"] * c["new"], s["kv_new"], s["kv_new"][:, n:], stride=2 * n,
                               seq_ids=s["seq_ids"], positions=s["positions"])
        if c["form"] == I8:   # as the values that they stand for
            rows = s["k"].numel() // c["d"]
            dmv.pesti_dequant_i8row(rows, c["d"], s["k"], s["k_scales"], s["values"][0])
            dmv.pesti_dequant_i8row(rows, c["d"], s["v"], s["v_scales"], s["values"][1])
            return [*s["values"], s["table"], s["lengths"], s["refs"]]
    elif c["kind"] == "fork":
        n = c["parents"] * c["each"]
        dmv.pesti_cache_free(cache, seqs, n, s["children"])
        dmv.pesti_cache_fork(cache, seqs, n, s["parents"], s["children"], s["status"], s["workspace"])
    else:
        s["table"].copy_(s["before"][0])
        s["refs"].copy_(s["before"][1])
        dmv.pesti_cache_compact(cache, seqs, s["status"], s["workspace"])
        return [s["k"], s["v"], s["table"], s["lengths"], s["refs"], s["status"]]
    return [s["k"], s["v"], s["table"], s["lengths"], s["refs"]]


def _weights(m, c):
    codes = torch.stack([m["packed"] & 15, m["packed"] >> 4], -1).reshape(c["out"], c["inf"]).float()
    group = torch.arange(c["inf"], device=codes.device) // c["group"]
    zero = 8.0 if m["zeros"] is None else m["zeros"].float()[:, group]
    return (codes - zero) * m["scales"].float()[:, group]


def _free_plain(s, rows):
    """The pages of the sequences `rows` (distinct) go back."""
    table, lengths, refs, page = s["table"], s["lengths"], s["refs"], s["case"]["page"]
    place = torch.arange(table.shape[1], device="cuda")
    held = place < ((lengths[rows] + page - 1) // page).unsqueeze(1)
    refs.index_add_(0, table[rows].clamp(min=0).reshape(-1), -held.int().reshape(-1))
    table[rows] = -1
    lengths[rows] = 0


def _take_plain(s, wanted):
    """The k-th true place of `wanted` (any shape, in its order) gets the k-th lowest free page; pages by place."""
    order = torch.argsort((s["refs"] > 0).int(), stable=True)
    rank = (wanted.reshape(-1).cumsum(0) - 1).clamp(0, order.shape[0] - 1)
    pages = order[rank].reshape(wanted.shape)
    s["refs"].index_add_(0, pages.reshape(-1), wanted.reshape(-1).int())
    return pages.int()


def _plain(s):
    c = s["case"]
    if c["kind"] == "gemv":
        y = s["x"] @ _weights(s["mats"][0], c).t()
        return y if s["bias"] is None else y + s["bias"]
    if c["kind"] == "swiglu":
        g, u = (s["x"] @ _weights(m, c).t() for m in s["mats"])
        return g / (1 + torch.exp(-g)) * u
    page, kv, d = c["page"], c["kv"], c["d"]
    if c["kind"] == "attend":
        rows, g, longest = c["rows"], c["g"], c["longest"]
        n = -(-longest // page)
        at = s["table"][:, :n].clamp(min=0).long()

        def tokens(x):   # [rows * kv][n * page][d]
            t = s[x][0][at].float()
            if c["form"] == I8:
                t = t * s[x + "_scales"][0][at].unsqueeze(-1)
            return t.transpose(1, 2).reshape(rows * kv, n * page, d)

        q = s["qkv"][:, :kv * g * d].float().reshape(rows * kv, g, d) * d ** -0.5
        score = torch.bmm(tokens("k"), q.transpose(1, 2).contiguous()).transpose(1, 2)   # [rows * kv][g][tokens]
        seen = torch.arange(n * page, device="cuda") < s["lengths"].repeat_interleave(kv).unsqueeze(1)
        score = torch.where(seen.unsqueeze(1), score, torch.full_like(score, -math.inf))
        p = torch.exp(score - score.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        return torch.bmm(p, tokens("v")).reshape(rows, kv * g, d).to(s["y"].dtype)
    if c["kind"] == "append":
        if c["replace"]:
            rows = s["slots"].long()
            _free_plain(s, rows)
            place = torch.arange(s["table"].shape[1], device="cuda")
            wanted = place < ((s["counts"] + page - 1) // page).unsqueeze(1)
            pages = _take_plain(s, wanted)
            s["table"][rows] = torch.where(wanted, pages, s["table"][rows])
            s["lengths"][rows] = s["counts"]
        pos = s["positions"].long()
        at, slot = s["table"][s["seq_ids"].long(), pos // page].long(), pos % page
        new = s["kv_new"].reshape(-1, 2, kv, d).float()
        for i, x in enumerate("kv"):
            t = new[:, i]
            if c["form"] == I8:
                scale = (t.abs().amax(-1).double() / 127).float()
                ratio = t.double() / scale.double().unsqueeze(-1)   # in 64 bits: in 32 a quotient is rounded onto borders
                ratio = torch.where(scale.unsqueeze(-1) > 0, ratio, torch.zeros_like(ratio))
                s[x + "_scales"][0][at, :, slot] = scale
                t = torch.sign(ratio) * torch.floor(ratio.abs() + 0.5)
            s[x][0][at, :, slot] = t.to(s[x].dtype)
        if c["form"] == I8:
            for i, x in enumerate("kv"):
                torch.mul(s[x].float(), s[x + "_scales"].unsqueeze(-1), out=s["values"][i])
            return [*s["values"], s["table"], s["lengths"], s["refs"]]
    elif c["kind"] == "fork":
        parents, children = s["parents"].long(), s["children"].long()
        _free_plain(s, children)
        lengths = s["lengths"][parents]
        place = torch.arange(s["table"].shape[1], device="cuda")
        whole = place < (lengths // page).unsqueeze(1)
        rows = torch.where(whole, s["table"][parents], torch.full_like(s["table"][parents], -1))
        part = lengths % page > 0
        new = _take_plain(s, part)
        s["refs"].index_add_(0, rows.clamp(min=0).reshape(-1), whole.int().reshape(-1))
        last = (lengths // page).long()
        old = s["table"][parents, last]
        rows.scatter_(1, last.unsqueeze(1), torch.where(part, new, torch.full_like(new, -1)).unsqueeze(1))
        s["table"][children] = rows
        s["lengths"][children] = lengths
        first = s["table"][parents, 0]   # a shared page onto itself where nothing is to be copied
        src, dst = torch.where(part, old, first).long(), torch.where(part, new, first).long()
        for x in "kv":
            s[x][:, dst] = s[x][:, src]
    else:
        s["table"].copy_(s["before"][0])
        s["refs"].copy_(s["before"][1])
        live = s["refs"] > 0
        count, index = live.sum(), torch.arange(c["pages"], device="cuda")
        holes = torch.argsort((live | (index >= count)).int(), stable=True)[:c["moves"]]
        movers = torch.argsort((~live | (index < count)).int(), stable=True)[:c["moves"]]
        for x in "kv":
            s[x][:, holes] = s[x][:, movers]
        to = index.clone()
        to[movers] = holes
        s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()].int(), s["table"]))
        s["refs"][holes] = s["refs"][movers]
        s["refs"][movers] = 0
        s["status"].copy_(count.reshape(1))
        return [s["k"], s["v"], s["table"], s["lengths"], s["refs"], s["status"]]
    return [s["k"], s["v"], s["table"], s["lengths"], s["refs"]]


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] in ("gemv", "swiglu"):
        x = s["x"].double()

        def product(m):
            y = torch.empty(c["batch"], c["out"], dtype=torch.float64, device="cuda")
            step = max(1, (1 << 27) // c["inf"])
            for a in range(0, c["out"], step):
                w = torch.empty(m["packed"][a:a + step].shape[0], c["inf"], dtype=torch.float64, device="cuda")
                w[:, 0::2] = (m["packed"][a:a + step] % 16).double()
                w[:, 1::2] = torch.div(m["packed"][a:a + step], 16, rounding_mode="floor").double()
                for j in range(m["scales"].shape[1]):
                    cols = slice(j * c["group"], (j + 1) * c["group"])
                    w[:, cols] -= 8 if m["zeros"] is None else m["zeros"][a:a + step, j:j + 1].double()
                    w[:, cols] *= m["scales"][a:a + step, j:j + 1].double()
                y[:, a:a + step] = torch.mm(x, w.t())
            return y

        y = product(s["mats"][0])
        if c["kind"] == "swiglu":
            return y * torch.sigmoid(y) * product(s["mats"][1])
        return y if s["bias"] is None else y + s["bias"].double()
    page, kv, d = c["page"], c["kv"], c["d"]
    if c["kind"] == "attend":
        g, y = c["g"], torch.empty(c["rows"], c["kv"] * c["g"], d, dtype=torch.float64, device="cuda")
        for r, n in enumerate(_lengths(c)):
            at = s["table"][r, :_pages_of(c, n)].long()
            for h in range(kv):
                k, v = (s[x][0, at, h].reshape(-1, d)[:n].double() for x in "kv")
                if c["form"] == I8:
                    k = k * s["k_scales"][0, at, h].reshape(-1, 1)[:n].double()
                    v = v * s["v_scales"][0, at, h].reshape(-1, 1)[:n].double()
                q = s["qkv"][r, h * g * d:(h + 1) * g * d].double().reshape(g, d)
                y[r, h * g:(h + 1) * g] = torch.mm(torch.softmax(torch.mm(q, k.t()) * d ** -0.5, -1), v)
        return y
    table, refs = s["table"].cpu(), s["refs"].cpu()
    lengths = s["lengths"].tolist()

    def take():   # the lowest free page
        p = int((refs == 0).nonzero()[0])
        refs[p] = 1
        return p

    if c["kind"] == "append":
        if c["replace"]:
            refs[table[table >= 0].long()] = 0
            table.fill_(-1)
            for r in range(c["seqs"]):
                for j in range(_pages_of(c, c["new"])):
                    table[r, j] = take()
        k, v = s["k"].double(), s["v"].double()
        if c["form"] == I8:
            k, v = k * s["k_scales"].double().unsqueeze(-1), v * s["v_scales"].double().unsqueeze(-1)
        new, row = s["kv_new"].double().reshape(-1, 2, kv, d), 0
        if c["form"] == I8:
            scale = (new.abs().max(-1, keepdim=True).values / 127).float().double()   # the scale is a float32 number
            ratio = new / torch.where(scale > 0, scale, torch.ones_like(scale))
            code = ratio.trunc() + torch.sign(ratio) * ((ratio - ratio.trunc()).abs() >= 0.5)
            new = code.clamp(-127, 127) * scale
        for r, n in enumerate(lengths):
            m = torch.arange(n - c["new"], n)
            at, slot = table[r][m // page].long().cuda(), (m % page).cuda()
            k[0, at, :, slot], v[0, at, :, slot] = new[row:row + c["new"], 0], new[row:row + c["new"], 1]
            row += c["new"]
        return [k, v, table.cuda(), s["lengths"], refs.cuda()]
    if c["kind"] == "fork":
        child = c["parents"]
        for p in range(c["parents"]):
            for _ in range(c["each"]):
                n = lengths[p]
                table[child, :n // page] = table[p, :n // page]
                refs[table[p, :n // page].long()] += 1
                if n % page:
                    old, new = int(table[p, n // page]), take()
                    table[child, n // page] = new
                    for x in "kv":
                        s[x][:, new] = s[x][:, old]
                lengths[child] = n
                child += 1
        return [s["k"].double(), s["v"].double(), table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), refs.cuda()]
    count = int((refs > 0).sum())
    holes = (refs[:count] == 0).nonzero().reshape(-1)
    movers = count + (refs[count:] > 0).nonzero().reshape(-1)
    to = torch.arange(c["pages"])
    to[movers] = holes
    for x in "kv":
        for a, b in zip(holes.tolist(), movers.tolist()):
            s[x][:, a] = s[x][:, b]
    refs[holes], refs[movers] = refs[movers], 0
    table = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table)
    return [s["k"].double(), s["v"].double(), table.cuda(), s["lengths"], refs.cuda(),
            torch.tensor([count], dtype=torch.int32).cuda()]
