"""What the paged-cache operators are measured on.

Five operators that a serving loop runs around a paged key-value cache:

  extend   block tables, lengths and slot maps made on the GPU from request lengths
  append   new key and value rows written into an uncompressed paged cache, with the running
           channel minimum and maximum of every block's keys
  scores   an upper bound of every block's query-key products, from those minima and maxima
  select   the blocks that each (sequence, KV head) attends to, as a block table
  attend   attention of one new token per sequence over the uncompressed paged cache

`run` computes them in plain torch operations, or, where `own` is true, makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a ragged batch: every sequence grows by one token, a few by a block
        {"name": "extend decode 64", "op": "extend", "batch": 64, "heads": 8, "block": 16, "lo": 1024, "hi": 32767,
         "new_lo": 1, "new_hi": 1},
        # a whole ragged batch is admitted: the slot of every (token, head) of its prompts
        {"name": "extend prompts 64", "op": "extend", "batch": 64, "heads": 8, "block": 16, "lo": 0, "hi": 0,
         "new_lo": 1024, "new_hi": 32768},
        # the append of one decode step
        {"name": "append decode 64", "op": "append", "batch": 64, "heads": 8, "block": 16, "d": 128, "dtype": "bf16",
         "lo": 1024, "hi": 32767, "new_lo": 1, "new_hi": 1},
        # prefill of four long prompts, keys and values as halves of one projection's output
        {"name": "append prompts 4 x 128K", "op": "append", "batch": 4, "heads": 8, "block": 16, "d": 128, "dtype": "bf16",
         "lo": 0, "hi": 0, "new_lo": 131072, "new_hi": 131072},
        # the cheap score of a decode step over four long contexts
        {"name": "scores 4 x 128K", "op": "scores", "batch": 4, "heads": 8, "group": 4, "block": 16, "d": 128,
         "dtype": "bf16", "lo": 131072, "hi": 131072},
        # the same of a ragged batch kept in fp32
        {"name": "scores ragged 64 f32", "op": "scores", "batch": 64, "heads": 8, "group": 4, "block": 16, "d": 128,
         "dtype": "f32", "lo": 1024, "hi": 32768},
        # few rows of many blocks each
        {"name": "select 4 x 128K", "op": "select", "batch": 4, "heads": 8, "block": 16, "lo": 131072, "hi": 131072,
         "keep": 256, "first": 1, "last": 4},
        # many rows of ragged length, some shorter than what is kept
        {"name": "select ragged 64", "op": "select", "batch": 64, "heads": 8, "block": 16, "lo": 1024, "hi": 32768,
         "keep": 128, "first": 1, "last": 2},
        # one short conversation: latency
        {"name": "attend 1 x 1000", "op": "attend", "batch": 1, "heads": 8, "group": 4, "block": 16, "d": 128,
         "dtype": "bf16", "out": "f32", "lo": 1000, "hi": 1000},
        # the ragged paged batch that the benchmark's decode step runs on
        {"name": "attend ragged 64", "op": "attend", "batch": 64, "heads": 8, "group": 4, "block": 16, "d": 128,
         "dtype": "bf16", "out": "bf16", "lo": 1024, "hi": 32768},
        # an fp32 cache of small heads in large blocks, eight query heads to a KV head, odd lengths
        {"name": "attend 7 x 9999 f32", "op": "attend", "batch": 7, "heads": 4, "group": 8, "block": 64, "d": 64,
         "dtype": "f32", "out": "f32", "lo": 1, "hi": 9999},
        # attention over 256 selected blocks of four long contexts: one-head sequences of 4096 tokens
        {"name": "attend selected 32 x 4096", "op": "attend", "batch": 32, "heads": 1, "group": 4, "block": 16, "d": 128,
         "dtype": "bf16", "out": "f32", "lo": 4081, "hi": 4096},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["extend", "append", "scores", "select", "attend", "attend"])
    batch, heads = _log(rng, 1, 96), rng.choice([1, 2, 3, 4, 8, 8, 16])
    block = rng.choice([8, 16, 16, 24, 32, 64, 128])
    case = {"op": op, "batch": batch, "heads": heads, "block": block}
    if op in ("extend", "append"):
        if rng.random() < 0.5:  # decode steps, or a few tokens at once
            case |= {"lo": 1, "hi": _log(rng, 16, 32767), "new_lo": rng.choice([0, 1]), "new_hi": _log(rng, 1, 8)}
        else:
            case |= {"lo": 0, "hi": rng.choice([0, _log(rng, 1, 4000)]), "new_lo": 0,
                     "new_hi": _log(rng, 64, max(64, min(131072, (8 if op == "extend" else 3) * 1000000 // (batch * heads))))}
        if op == "append":
            case |= {"d": rng.choice([64, 80, 96, 128, 128, 192, 256]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
            case["new_hi"] = max(1, min(case["new_hi"], 128 * case["new_hi"] // case["d"]))
            case["hi"] = min(case["hi"], max(1, 3000000 // (batch * heads)))
            case["lo"] = min(case["lo"], case["hi"])
        return case
    most = max(16, min(131072, 6000000 // (batch * heads)))  # tokens of a sequence
    case |= {"lo": 1, "hi": _log(rng, 16, most)}
    if rng.random() < 0.3:
        case["lo"] = case["hi"]
    if op == "select":
        first, last = rng.choice([0, 1, 4]), rng.choice([1, 2, 8])
        return case | {"first": first, "last": last, "keep": first + last + _log(rng, 1, 500)}
    case |= {"group": rng.choice([1, 2, 4, 4, 5, 7, 8, 16]), "d": rng.choice([64, 80, 96, 128, 128, 192, 256]),
             "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "attend":
        case["hi"] = max(1, case["hi"] * (64 if case["dtype"] == "bf16" else 32) // max(64, case["d"]))
        case["lo"] = min(case["lo"], case["hi"])
        case["out"] = rng.choice(["f32", case["dtype"]])
    return case


# ------------------------------------------------------------------------------------ inputs
def _lengths(batch, lo, hi):
    """Lengths spread evenly over [lo, hi]: their sum, and so every buffer's size, goes by the case alone."""
    return torch.tensor([hi if batch == 1 else lo + (hi - lo) * i // (batch - 1) for i in range(batch)], device="cuda")


def _tables(g, counts, width, spare=0):
    """A block table [batch, width] whose rows hold `counts` blocks of one random order, and the blocks left over."""
    n = int(counts.sum())
    perm = torch.randperm(n + spare, generator=g, device="cuda").to(torch.int32)
    at = torch.cumsum(counts, 0) - counts
    j = torch.arange(width, device="cuda")
    table = torch.where(j < counts[:, None], perm[(at[:, None] + j).clamp(max=max(n + spare - 1, 0))], -1).to(torch.int32)
    return table.contiguous(), perm[n:].contiguous(), n + spare


def _channels(g, shape, heads, d, dtype):
    """Rows [..., heads, d] whose channels have scales of their own."""
    scale = torch.exp(0.5 * torch.randn(heads, d, generator=g, device="cuda"))
    x = torch.empty(*shape, heads, d, dtype=dtype, device="cuda")
    x.normal_(generator=g)
    return x.mul_(scale.to(dtype))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    b, h, bs, op = case["batch"], case["heads"], case["block"], case["op"]
    order = torch.randperm(b, generator=g, device="cuda")
    lens = _lengths(b, case["lo"], case["hi"])[order]
    s = {"case": case, "op": op, "heads": h, "block": bs}
    if op in ("extend", "append"):
        new = _lengths(b, case["new_lo"], case["new_hi"]).flip(0)[order]
        width = -(-(case["hi"] + case["new_hi"]) // bs)
        have, total = (lens + bs - 1) // bs, (lens + new + bs - 1) // bs
        spare = int((total - have).sum())
        # a serving loop gives the rows' buffers a fixed size: the last rows are padding
        n_rows = int(new.sum()) + (5 if op == "extend" else 0)
        s["n_rows"] = max(n_rows, 1)
        if op == "extend":
            # the free list has a few blocks more than this batch takes, behind some that are gone
            table, free, n_blocks = _tables(g, have, width, spare + 7 + 3)
            s |= {"free": free, "head": torch.full((1,), 3, dtype=torch.int32, device="cuda"),
                  "lens": lens.to(torch.int32), "new": new.to(torch.int32)}
            if own:
                from kv_cache_vector_06_b200 import tq
                e = lambda n, t: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
                s["outs"] = {"new_slots": e(s["n_rows"] * h, torch.int64), "seq_lens_out": e(b, torch.int32),
                             "granted": e(b, torch.int32), "free_head_out": e(1, torch.int32),
                             "row_offsets": e(b + 1, torch.int64)}
        else:
            table, _, n_blocks = _tables(g, total, width)
            d, dt = case["d"], DTYPES[case["dtype"]]
            # keys and values leave one projection side by side
            kv = _channels(g, (s["n_rows"], 2), h, d, dt)
            offsets = torch.zeros(b + 1, dtype=torch.int64, device="cuda")
            offsets[1:] = torch.cumsum(new, 0)
            s |= {"k": kv[:, 0], "v": kv[:, 1], "lens": (lens + new).to(torch.int32), "granted": new.to(torch.int32),
                  "offsets": offsets, "k_cache": torch.zeros(n_blocks, h, bs, d, dtype=dt, device="cuda"),
                  "v_cache": torch.zeros(n_blocks, h, bs, d, dtype=dt, device="cuda"),
                  "bounds": _channels(g, (n_blocks, h), 2, d, dt).sort(dim=2).values}
    else:
        width = -(-case["hi"] // bs)
        table, _, n_blocks = _tables(g, (lens + bs - 1) // bs, width)
        s["lens"] = lens.to(torch.int32)
        if op == "select":
            s["scores"] = torch.randn(b * h, width, generator=g, device="cuda") * 8
            if own:
                s["outs"] = {"table": torch.empty(b * h, case["keep"], dtype=torch.int32, device="cuda"),
                             "lens": torch.empty(b * h, dtype=torch.int32, device="cuda")}
        else:
            d, dt, group = case["d"], DTYPES[case["dtype"]], case["group"]
            s["q"] = torch.randn(b, h * group, d, generator=g, device="cuda").to(dt)
            if op == "scores":
                s["bounds"] = _channels(g, (n_blocks, h), 2, d, dt).sort(dim=2).values
                if own:
                    s["outs"] = {"out": torch.empty(b * h, width, device="cuda")}
            else:
                s["k_cache"] = _channels(g, (n_blocks, h), bs, d, dt)
                s["v_cache"] = _channels(g, (n_blocks, h), bs, d, dt)
                if own:
                    from kv_cache_vector_06_b200 import tq
                    s["outs"] = {"out": torch.empty(b, h * group, d, dtype=DTYPES[case["out"]], device="cuda")}
    s["table"], s["n_blocks"] = table, n_blocks
    if own:
        from kv_cache_vector_06_b200 import tq
        s["pages"] = tq.Pages(table, n_kv_heads=h, block_size=bs, n_blocks=n_blocks)
        if op == "attend":
            s["outs"]["ws"] = torch.empty(tq.attend_paged_workspace_size(s["pages"], case["hi"], h * case["group"], case["d"]),
                                          dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"extend": _extend, "append": _append, "scores": _scores, "select": _select, "attend": _attend}[s["op"]](s)


def _own(s):
    from kv_cache_vector_06_b200 import tq
    c, o, p = s["case"], s.get("outs"), s["pages"]
    if s["op"] == "extend":
        tq.page_extend(p, s["lens"], s["new"], s["free"], s["head"], **o)
        return [s["table"], o["seq_lens_out"], o["granted"], o["free_head_out"], o["row_offsets"], o["new_slots"]]
    if s["op"] == "append":
        tq.append_kv(p, s["lens"], s["granted"], s["offsets"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["bounds"])
        return [s["k_cache"], s["v_cache"], s["bounds"]]
    if s["op"] == "scores":
        return [tq.block_scores(p, s["lens"], s["q"], s["bounds"], **o)]
    if s["op"] == "select":
        return list(tq.select_blocks(p, s["lens"], s["scores"], c["keep"], n_first=c["first"], n_last=c["last"], **o))
    return [tq.attend_paged(p, s["lens"], c["hi"], s["q"], s["k_cache"], s["v_cache"], **o)]


def _row_slots(table, before, granted, offsets, n_rows, heads, bs, n_blocks):
    """Position and slot (or -1) of every (row, head), and the rows' sequences."""
    r = torch.arange(n_rows, device=table.device)
    b = torch.searchsorted(offsets[1:].contiguous(), r, right=True)
    inside = b < table.shape[0]
    b = b.clamp(max=table.shape[0] - 1)
    pos = before[b] + r - offsets[b]
    j = (pos // bs).clamp(0, table.shape[1] - 1)
    entry = table[b, j].long()
    ok = inside & (granted[b] > 0) & (entry >= 0) & (entry < n_blocks)
    slot = (entry[:, None] * heads + torch.arange(heads, device=table.device)) * bs + (pos % bs)[:, None]
    return b, pos, torch.where(ok[:, None], slot, -1)


def _extend(s):
    h, bs, table, n_rows = s["heads"], s["block"], s["table"], s["n_rows"]
    lens, new, width = s["lens"].long(), s["new"].long(), table.shape[1]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=table.device), torch.cumsum(new, 0)])
    have = (lens + bs - 1) // bs
    fits = (lens + new <= width * bs) & (offsets[1:] <= n_rows)
    need = torch.where(fits, (lens + new + bs - 1) // bs - have, 0)
    upto = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (upto <= s["free"].shape[0] - s["head"].long()))
    need = torch.where(ok, need, 0)
    granted = torch.where(ok, new, 0)
    j = torch.arange(width, device=table.device) - have[:, None]
    taken = (s["head"].long() + (upto - need)[:, None] + j).clamp(0, s["free"].shape[0] - 1)
    table = torch.where((j >= 0) & (j < need[:, None]), s["free"][taken], table)
    _, _, slots = _row_slots(table, lens, granted, offsets, n_rows, h, bs, s["n_blocks"])
    return [table, (lens + granted).to(torch.int32), granted.to(torch.int32), (s["head"] + need.sum()).to(torch.int32),
            offsets, slots.reshape(-1)]


def _append(s):
    h, bs, d, n_rows = s["heads"], s["block"], s["case"]["d"], s["n_rows"]
    before = s["lens"].long() - s["granted"].long()
    b, pos, slots = _row_slots(s["table"], before, s["granted"], s["offsets"], n_rows, h, bs, s["n_blocks"])
    ok = slots >= 0
    at, kf = slots[ok], s["k"][ok]
    s["k_cache"].view(-1, d)[at] = kf
    s["v_cache"].view(-1, d)[at] = s["v"][ok]
    # blocks that begin with a new row start from nothing
    block = at // bs
    fresh = block[(pos - pos % bs >= before[b])[:, None].expand(-1, h)[ok]]
    bounds = s["bounds"].view(-1, 2, d)
    lo, hi = bounds[:, 0].float(), bounds[:, 1].float()
    lo[fresh], hi[fresh] = math.inf, -math.inf
    to = block[:, None].expand(-1, d)
    lo.scatter_reduce_(0, to, kf.float(), "amin")
    hi.scatter_reduce_(0, to, kf.float(), "amax")
    bounds[:, 0], bounds[:, 1] = lo.to(bounds.dtype), hi.to(bounds.dtype)
    return [s["k_cache"], s["v_cache"], s["bounds"]]


def _scores(s):
    b, width = s["table"].shape
    h, d, bs = s["heads"], s["case"]["d"], s["block"]
    q = s["q"].float().view(b, h, -1, d)
    x = s["bounds"][s["table"].long().clamp(min=0)].permute(0, 2, 3, 4, 1)  # [b, h, 2, d, width]
    t = torch.matmul(q.clamp(min=0), x[:, :, 1].float()) + torch.matmul(q.clamp(max=0), x[:, :, 0].float())
    n = (s["lens"].long() + bs - 1) // bs
    inside = torch.arange(width, device=q.device) < n[:, None]
    return [torch.where(inside[:, None], t.amax(2), -math.inf).view(b * h, width)]


def _select(s):
    c, h, bs = s["case"], s["heads"], s["block"]
    b, width = s["table"].shape
    keep = c["keep"]
    n = ((s["lens"].long() + bs - 1) // bs)[:, None]
    j = torch.arange(width, device=n.device)
    forced = (j < c["first"]) | (j >= n - c["last"])
    rank = torch.where(j < n, torch.where(forced, math.inf, s["scores"].view(b, h, width).transpose(0, 1)), -math.inf)
    order = torch.sort(rank.transpose(0, 1), dim=2, descending=True, stable=True).indices[:, :, :keep]
    order = torch.sort(torch.where(order < n[:, :, None], order, width), dim=2).values
    held = n.clamp(max=keep)
    if order.shape[2] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[2]), value=width)
    entry = torch.gather(s["table"].long()[:, None].expand(b, h, width), 2, order.clamp(max=width - 1))
    entry = entry * h + torch.arange(h, device=n.device)[:, None]
    table = torch.where(order < width, entry, -1).to(torch.int32)
    tail = s["lens"].long()[:, None] - (n - 1) * bs  # tokens of the last block
    lens = torch.where(n > 0, (held - 1) * bs + tail, 0).expand(b, h)
    return [table.view(b * h, keep), lens.reshape(-1).to(torch.int32)]


def _attend(s):
    b, width = s["table"].shape
    c, h, bs, d = s["case"], s["heads"], s["block"], s["case"]["d"]
    q = s["q"].float().view(b, h, -1, d) / math.sqrt(d)
    at = s["table"].long().clamp(min=0)
    x = s["k_cache"][at].transpose(1, 2).reshape(b, h, width * bs, d)
    logits = torch.matmul(q, x.float().transpose(2, 3))
    inside = (torch.arange(width * bs, device=q.device) < s["lens"][:, None])[:, None, None]
    logits = torch.where(inside, logits, -math.inf)
    p = torch.exp(logits - logits.amax(3, keepdim=True))
    x = s["v_cache"][at].transpose(1, 2).reshape(b, h, width * bs, d)
    o = torch.matmul(p, x.float()) / p.sum(3, keepdim=True)
    return [o.view(b, -1, d).to(DTYPES[c["out"]])]


# ------------------------------------------------------------------------------------ the least work
def work(case):
    b, h, bs, op = case["batch"], case["heads"], case["block"], case["op"]
    mean = (case["lo"] + case["hi"]) / 2
    blocks = b * (mean / bs + (0.5 if case["hi"] > case["lo"] else 0))
    if op in ("extend", "append"):
        rows = b * (case["new_lo"] + case["new_hi"]) / 2
        if op == "extend":
            return {"bytes": 8 * rows * h + 8 * rows / bs + 28 * b, "flops": 0}
        e = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        # rows in and out, the bounds of the blocks they touch (read again where they were begun before)
        touched = b * (case["new_lo"] + case["new_hi"]) / 2 / bs + b
        return {"bytes": (4 * rows + 2 * touched + (2 * b if case["hi"] else 0)) * h * case["d"] * e, "flops": 2 * rows * h * case["d"]}
    if op == "select":
        return {"bytes": 4 * blocks * h + 8 * b * h * min(case["keep"], -(-mean // bs)), "flops": 0}
    e = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    d, group = case["d"], case["group"]
    if op == "scores":
        return {"bytes": blocks * h * (2 * d * e + 4) + b * h * group * d * e, "flops": 4 * blocks * h * group * d}
    return {"bytes": b * h * (2 * mean + 2 * group) * d * e, "flops": 4 * b * mean * h * group * d}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, h, bs = case["op"], case["heads"], case["block"]
    if op in ("extend", "select"):
        return None  # whole numbers
    d, lens, table = case["d"], s["lens"].tolist(), s["table"].long()
    if op == "append":
        if sum(lens) * h * d > 1.5e9:
            return None
        out = s["bounds"].double()
        grown, at = s["granted"].tolist(), s["offsets"].tolist()
        for b, (n, m) in enumerate(zip(lens, grown)):
            if m == 0:
                continue
            first, rows = (n - m) // bs, s["k"][at[b]:at[b] + m].double()
            lead, tail = (n - m) % bs, -n % bs
            pad = lambda fill: torch.cat([torch.full((lead, h, d), fill, device="cuda", dtype=torch.float64), rows,  # noqa: E731
                                          torch.full((tail, h, d), fill, device="cuda", dtype=torch.float64)]).view(-1, bs, h, d)
            lo, hi = pad(math.inf).amin(1), pad(-math.inf).amax(1)
            where = table[b, first:-(-n // bs)]
            if lead:
                lo[0], hi[0] = torch.minimum(lo[0], out[where[0], :, 0]), torch.maximum(hi[0], out[where[0], :, 1])
            out[where, :, 0], out[where, :, 1] = lo, hi
        return [None, None, out]
    q = s["q"].double()
    group = case["group"]
    if op == "scores":
        width = table.shape[1]
        out = torch.full((len(lens) * h, width), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            held = -(-n // bs)
            x = s["bounds"][table[b, :held]].double()
            for hq in range(h * group):
                y = q[b, hq] * x[:, hq // group]
                t = torch.maximum(y[:, 0], y[:, 1]).sum(1)
                row = out[b * h + hq // group]
                row[:held] = torch.maximum(row[:held], t)
        return [out]
    out = torch.zeros(len(lens), h * group, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v = (s[x][table[b, :-(-n // bs)]].transpose(1, 2).reshape(-1, h, d)[:n].double() for x in ("k_cache", "v_cache"))
        w = torch.softmax(torch.einsum("hgd,nhd->hgn", q[b].view(h, group, d), k) * d ** -0.5, dim=2)
        out[b] = torch.einsum("hgn,nhd->hgd", w, v).reshape(h * group, d)
    return [out]
