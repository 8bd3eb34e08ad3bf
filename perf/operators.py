"""The paged-cache operators as they are measured: block tables and slot maps,
the write of new rows, attention of one new token, key bounds per block, and
attention over the blocks that a score on those bounds selects.

Each operator has a plain form in elementary torch operations (``own`` false)
and the calls a program makes of the library (``own`` true). Shapes follow the
workload table of this repository (8 or 4 heads of 128, 2 or 3 of 64, pages of
16 tokens, 8192 to 32768 tokens, 16 requests) and the ranges around it.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------- the cases ---

def listed():
    return [
        # one decoding step's bookkeeping: every request grows by one token
        {"name": "tables_step", "op": "tables", "requests": 64, "block": 16, "longest": 8192, "grow": 1},
        # a batch admitted or restored at once: every page of every request is new
        {"name": "tables_admit", "op": "tables", "requests": 512, "block": 16, "longest": 8192, "grow": 0},
        # one decoding step's K and V rows of one layer, cut out of the fused projection
        {"name": "write_step", "op": "write", "tokens": 64, "heads": 8, "dim": 128, "block": 16, "type": "bf16", "source": "bf16"},
        # the rows of a prefill, from fp32 activations into bf16 pages
        {"name": "write_prefill", "op": "write", "tokens": 32768, "heads": 8, "dim": 128, "block": 16, "type": "bf16", "source": "f32"},
        # a single user, 8K tokens: latency
        {"name": "attend_one", "op": "attend", "requests": 1, "heads": 8, "group": 4, "dim": 128, "block": 16, "longest": 8192,
         "even": True, "type": "bf16"},
        # 16 paged requests of 8K tokens, 4 heads of 128 shared by 7 queries each
        {"name": "attend_batch", "op": "attend", "requests": 16, "heads": 4, "group": 7, "dim": 128, "block": 16, "longest": 8192,
         "even": True, "type": "bf16"},
        # lengths from one token to 16K in one batch, odd heads of 64 in fp32
        {"name": "attend_ragged_f32", "op": "attend", "requests": 48, "heads": 3, "group": 4, "dim": 64, "block": 16, "longest": 16384,
         "even": False, "type": "f32"},
        # the largest: eight requests of 64K tokens
        {"name": "attend_long", "op": "attend", "requests": 8, "heads": 8, "group": 8, "dim": 128, "block": 32, "longest": 65536,
         "even": True, "type": "bf16"},
        # one decoding step's bounds: the last page of each request
        {"name": "bounds_step", "op": "bounds", "requests": 64, "heads": 8, "dim": 128, "block": 16, "longest": 8192, "fresh": False,
         "type": "bf16"},
        # bounds of a restored cache: every page of 16 requests
        {"name": "bounds_restore", "op": "bounds", "requests": 16, "heads": 8, "dim": 128, "block": 16, "longest": 8192, "fresh": True,
         "type": "bf16"},
        # select and attend, one 32K request: latency
        {"name": "sparse_one", "op": "sparse", "requests": 1, "heads": 8, "group": 4, "dim": 128, "block": 16, "longest": 32768,
         "even": True, "budget": 64, "type": "bf16"},
        # select and attend, a ragged batch of up to 64K tokens
        {"name": "sparse_batch", "op": "sparse", "requests": 16, "heads": 8, "group": 4, "dim": 128, "block": 16, "longest": 65536,
         "even": False, "budget": 256, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "write", "attend", "attend", "bounds", "sparse"])
    if op == "tables":
        return {"op": op, "requests": _log(rng, 1, 512), "block": rng.choice([1, 8, 16, 24, 32, 64]),
                "longest": _log(rng, 16, 8192), "grow": rng.choice([0, 1, 5, 300])}
    heads, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 80, 96, 128, 192, 256])
    c = {"op": op, "heads": heads, "dim": dim, "block": rng.choice([8, 16, 16, 20, 32, 64]), "type": rng.choice(["bf16", "bf16", "f32"])}
    if op == "write":
        c.update(tokens=_log(rng, 1, 16384), source=rng.choice(["bf16", "f32"]))
        return c
    c["longest"] = _log(rng, 1, 65536)
    # at most 2^18 tokens of 1024 bf16 features in all
    most = max(1, (1 << 28) // (c["longest"] * heads * dim * (2 if c["type"] == "f32" else 1)))
    c["requests"] = _log(rng, 1, min(128, most))
    if op == "bounds":
        c["fresh"] = rng.choice([True, False])
        return c
    c.update(group=rng.choice([1, 2, 4, 5, 7, 8, 16, 24]), even=rng.choice([True, False]))
    if op == "sparse":
        c["budget"] = _log(rng, 4, max(4, min(512, 2 * -(-c["longest"] // c["block"]))))   # up to twice the pages there are
    return c


# ---------------------------------------------------------------- the inputs ---

def _spread(n, longest):
    """n lengths spread evenly over the logarithm, a single token and the longest among them."""
    inner = [max(1, min(longest, round(longest ** (i / (n - 1))))) for i in range(1, n - 1)]
    return [longest] + inner + [1] * (n > 1)


def _lengths(case, g):
    """int32 [requests]: all the longest, or the spread lengths in random order."""
    n, longest = case["requests"], case["longest"]
    if case.get("even", False):
        return torch.full((n,), longest, dtype=torch.int32, device=DEV)
    order = torch.randperm(n, generator=g, device=DEV)
    return torch.tensor(_spread(n, longest), dtype=torch.int32, device=DEV)[order].contiguous()


def _keys(shape, heads, dim, dtype, g):
    """Rows [..., heads * dim] like a key cache: a fixed offset per feature and four strong channels per head."""
    x = torch.empty(shape, dtype=dtype, device=DEV)
    x.normal_(generator=g)
    strong = torch.ones(heads, dim, device=DEV)
    strong[:, torch.randperm(dim, generator=g, device=DEV)[:4]] = 4.0
    offset = 0.5 * torch.randn(heads * dim, generator=g, device=DEV)
    x.mul_(strong.reshape(-1).to(dtype)).add_(offset.to(dtype))
    return x


def _table(lens, block, n_blocks, g):
    """int32 [requests, width]: distinct pages in random order, zeros behind each request's last page."""
    need = (lens.long() + block - 1) // block
    width = int(need.max())
    ids = torch.randperm(n_blocks, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(width, device=DEV)[None, :]
    first = (torch.cumsum(need, 0) - need)[:, None]
    return torch.where(at < need[:, None], ids[(first + at).clamp(max=n_blocks - 1)], 0).to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = case["op"], {"case": dict(case)}
    if op == "tables":
        n, b, longest, grow = case["requests"], case["block"], case["longest"], case["grow"]
        lens = _lengths(case, g)
        old = lens if grow else torch.zeros_like(lens)
        new = lens + grow if grow else lens
        width = (longest + grow + b - 1) // b
        held = (old.long() + b - 1) // b
        n_blocks = int(((new.long() + b - 1) // b).sum()) + 7
        ids = torch.randperm(n_blocks, generator=g, device=DEV).to(torch.int32)
        at = torch.arange(width, device=DEV)[None, :]
        first = (torch.cumsum(held, 0) - held)[:, None]
        s["table"] = torch.where(at < held[:, None], ids[(first + at).clamp(max=n_blocks - 1)], -1).to(torch.int32).contiguous()
        taken = int(held.sum())
        s["free"] = ids[taken:].contiguous()
        s["free_from"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s.update(old=old, new=new, n_blocks=n_blocks)
        # a padded batch: some slots behind the last token
        s["slots"] = torch.empty(int((new - old).sum()) + 13, dtype=torch.int32, device=DEV)
        s["starts"] = torch.empty(n + 1, dtype=torch.int32, device=DEV)
        s["taken"] = torch.empty(1, dtype=torch.int32, device=DEV)
        return s
    h, d, b = case["heads"], case["dim"], case["block"]
    f, dt = h * d, TYPES[case["type"]]
    if op == "write":
        t = case["tokens"]
        n_blocks = (t + b - 1) // b + 3
        s["k"] = torch.zeros(n_blocks, b, f, dtype=dt, device=DEV)
        s["v"] = torch.zeros_like(s["k"])
        fused = torch.empty(t, 4 * f, dtype=TYPES[case["source"]], device=DEV).normal_(generator=g)   # queries, keys, values
        s["k_rows"], s["v_rows"] = fused[:, 2 * f:3 * f], fused[:, 3 * f:]
        s["slots"] = torch.randperm(n_blocks * b, generator=g, device=DEV)[:t].to(torch.int32)
        s["slots"][t // 2 + 1::97] = -1   # padding rows
        return s
    lens = _lengths(case, g)
    n_blocks = int(((lens.long() + b - 1) // b).sum()) + 5
    s["lens"], s["table"] = lens, _table(lens, b, n_blocks, g)
    s["k"] = _keys((n_blocks, b, f), h, d, dt, g)
    if op == "bounds":
        s["from"] = torch.zeros_like(lens) if case["fresh"] else (lens - 1).clamp(min=0)
        s["bounds"] = torch.zeros(n_blocks, 2, f, dtype=dt, device=DEV)
        s["v"] = s["k"]
        return s
    s["v"] = torch.empty_like(s["k"]).normal_(generator=g)
    hq = h * case["group"]
    s["q"] = _keys((case["requests"], hq * d), hq, d, dt, g)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(case["requests"], hq, dtype=torch.float32, device=DEV)
    if op == "sparse":
        valid = torch.zeros(n_blocks, dtype=torch.int64, device=DEV)   # rows in use of each page
        at = torch.arange(s["table"].shape[1], device=DEV)[None, :]
        rows = (lens.long()[:, None] - at * b).clamp(0, b)
        used = rows > 0
        valid[s["table"].long()[used]] = rows[used]
        live = (torch.arange(b, device=DEV)[None, :] < valid[:, None])[:, :, None]
        s["bounds"] = torch.stack([s["k"].masked_fill(~live, math.inf).amin(1), s["k"].masked_fill(~live, -math.inf).amax(1)], 1).contiguous()
        s["chosen"] = torch.empty(case["requests"], h, case["budget"], dtype=torch.int32, device=DEV)
    return s


def _first_last(case):
    """Pages kept whatever their score: the first one and the last two, as far as the budget goes."""
    return 1, min(2, case["budget"] - 1)


# ------------------------------------------------------------ the plain forms ---

def _plain_tables(s):
    b = s["case"]["block"]
    old, new = s["old"].long(), s["new"].long()
    had, have = (old + b - 1) // b, (new + b - 1) // b
    need = have - had
    first = torch.cumsum(need, 0) - need
    served = (need == 0) | (s["free_from"] + first + need <= s["free"].numel())
    at = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    fill = served[:, None] & (at >= had[:, None]) & (at < have[:, None])
    pick = (s["free_from"] + first[:, None] + at - had[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fill, s["free"][pick], s["table"])
    grow = new - old
    ends = torch.cumsum(grow, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(s["slots"].numel(), device=DEV)
    i = torch.searchsorted(ends, t, right=True)
    live = i < old.numel()
    i = i.clamp(max=old.numel() - 1)
    p = old[i] + t - starts[i]
    page = table[i, (p // b).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(live & served[i], page * b + p % b, -1)
    return {"table": table, "slots": slots.int(), "starts": starts.int(), "taken": need[served].sum().int()}


def _plain_write(s):
    f = s["k"].shape[-1]
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    s["k"].view(-1, f)[at] = s["k_rows"][keep].to(s["k"].dtype)
    s["v"].view(-1, f)[at] = s["v_rows"][keep].to(s["v"].dtype)
    return {"k": s["k"], "v": s["v"]}


def _plain_bounds(s):
    b = s["case"]["block"]
    lens = s["lens"].long()
    at = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    todo = (at >= (s["from"].long() // b)[:, None]) & (at * b < lens[:, None])
    pages = s["table"].long()[todo]
    rows = (lens[:, None] - at * b).clamp(max=b)[todo]
    k = s["k"][pages].float()
    live = (torch.arange(b, device=DEV)[None, :] < rows[:, None])[:, :, None]
    lo = k.masked_fill(~live, math.inf).amin(1)
    hi = k.masked_fill(~live, -math.inf).amax(1)
    s["bounds"][pages] = torch.stack([lo, hi], 1).to(s["bounds"].dtype)
    return s["bounds"]


def _softmax_rows(q, k, v, live, scale):
    """q [n, h, g, d], k and v [n, h, t, d] in fp32, live [n, h or 1, t]; rows with nothing live give 0 and -inf."""
    w = torch.matmul(q, k.transpose(-1, -2).contiguous()) * scale
    w = w.masked_fill(~live[:, :, None, :], -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = torch.exp(w - top)
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w, v.masked_fill(~live[..., None], 0.0))
    return out / torch.where(total > 0, total, torch.ones_like(total)), (torch.log(total) + top).squeeze(-1)


def _plain_attend(s):
    c = s["case"]
    n, h, g, d, b = c["requests"], c["heads"], c["group"], c["dim"], c["block"]
    t = s["table"].shape[1] * b
    k = s["k"][s["table"].long()].view(n, t, h, d).transpose(1, 2).float()
    v = s["v"][s["table"].long()].view(n, t, h, d).transpose(1, 2).float()
    live = (torch.arange(t, device=DEV)[None, :] < s["lens"][:, None])[:, None, :]
    out, lse = _softmax_rows(s["q"].view(n, h, g, d).float(), k, v, live, d ** -0.5)
    return {"out": out.reshape(n, h * g * d).to(s["q"].dtype), "lse": lse.reshape(n, h * g)}


def _plain_sparse(s):
    c = s["case"]
    n, h, g, d, b, budget = c["requests"], c["heads"], c["group"], c["dim"], c["block"], c["budget"]
    first, last = _first_last(c)
    q, width = s["q"].view(n, h, g, d).double(), s["table"].shape[1]
    box = s["bounds"][s["table"].long()].view(n, width, 2, h, d).permute(2, 0, 3, 1, 4).double()   # [lo/hi, n, h, width, d]
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    score = ((box[1] * up[:, :, None]).sum(-1) + (box[0] * down[:, :, None]).sum(-1)).float() + 0.0
    # an integer that orders like the score, NaN above all numbers, kept pages above those
    bits = score.view(torch.int32).long()
    rank = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF) - 1)
    rank = torch.where(torch.isnan(score), 0x7FFFFFFE, rank)
    at = torch.arange(width, device=DEV)[None, :]
    pages = (s["lens"].long()[:, None] + b - 1) // b
    kept = (at < first) | (at >= pages - last)
    rank = torch.where(kept[:, None], 0x7FFFFFFF, rank)
    rank = torch.where((at < pages)[:, None], rank, -(1 << 33))
    order = torch.sort(rank, dim=-1, descending=True, stable=True)
    take = min(budget, width)
    there = order.values[..., :take] > -(1 << 33)
    chosen = torch.where(there, order.indices[..., :take], 1 << 30).sort(-1).values
    chosen = torch.where(chosen < (1 << 30), chosen, -1)
    chosen = torch.nn.functional.pad(chosen, (0, budget - take), value=-1)
    # attention over the chosen pages' tokens
    ids = torch.gather(s["table"].long()[:, None].expand(n, h, width), 2, chosen.clamp(min=0))
    head = torch.arange(h, device=DEV)[None, :, None, None]
    row = torch.arange(b, device=DEV)[None, None, None, :]
    k = s["k"].view(-1, b, h, d)[ids[..., None], row, head].reshape(n, h, budget * b, d).float()
    v = s["v"].view(-1, b, h, d)[ids[..., None], row, head].reshape(n, h, budget * b, d).float()
    live = ((chosen[..., None] >= 0) & (chosen[..., None] * b + row < s["lens"].long()[:, None, None, None])).reshape(n, h, budget * b)
    out, lse = _softmax_rows(q.float(), k, v, live, d ** -0.5)
    return {"chosen": chosen.int(), "out": out.reshape(n, h * g * d).to(s["q"].dtype), "lse": lse.reshape(n, h * g)}


# -------------------------------------------------------- the library's calls ---

def _own(s):
    import kv_cache_transform_amd as K
    c = s["case"]
    stream = torch.cuda.current_stream()
    if c["op"] == "tables":
        plan = K.make_page_plan(s["old"], s["new"], c["requests"], c["block"], s["free"], s["free"].numel(), s["n_blocks"],
                                s["table"], s["table"].shape[1], s["slots"], s["slots"].numel(),
                                free_from=s["free_from"], starts=s["starts"], taken=s["taken"])
        K.kvtc_page_tables(plan, stream)
        return {"table": s["table"], "slots": s["slots"], "starts": s["starts"], "taken": s["taken"][0]}
    dt = K.KVTC_BF16 if c["type"] == "bf16" else K.KVTC_F32
    pages = K.make_pages(s["k"], s["v"], s["k"].shape[0], c["block"], c["heads"], c["dim"], dt)
    if c["op"] == "write":
        rows = K.make_page_rows(s["k_rows"], s["v_rows"], c["tokens"], s["slots"], K.KVTC_BF16 if c["source"] == "bf16" else K.KVTC_F32,
                                k_stride=s["k_rows"].stride(0), v_stride=s["v_rows"].stride(0))
        K.kvtc_page_write(pages, rows, stream)
        return {"k": s["k"], "v": s["v"]}
    req = K.make_requests(s["table"], s["table"].shape[1], s["lens"], s["lens"].numel())
    if c["op"] == "bounds":
        K.kvtc_page_bounds(pages, req, s["from"], s["bounds"], stream=stream)
        return s["bounds"]
    queries = K.make_queries(s["q"], s["out"], c["heads"] * c["group"], c["dim"] ** -0.5, lse=s["lse"])
    chosen = None
    if c["op"] == "sparse":
        first, last = _first_last(c)
        chosen = K.make_selection(s["chosen"], c["budget"], first, last)
    if "ws" not in s:   # one workspace for both calls, kept as a program keeps it
        s["ws"] = torch.empty(K.kvtc_page_workspace_bytes(pages, req, queries, chosen), dtype=torch.uint8, device=DEV)
    if chosen is not None:
        K.kvtc_page_select(pages, req, queries, s["bounds"], chosen, s["ws"], stream=stream)
    K.kvtc_page_attend(pages, req, queries, chosen, s["ws"], stream=stream)
    if chosen is None:
        return {"out": s["out"], "lse": s["lse"]}
    return {"chosen": s["chosen"], "out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "write": _plain_write, "bounds": _plain_bounds, "attend": _plain_attend,
            "sparse": _plain_sparse}[state["case"]["op"]](state)


# ----------------------------------------------------------- the work of each ---

def work(case):
    op, b, n = case["op"], case["block"], case["requests"] if "requests" in case else 0
    lens = [] if op == "write" else [case["longest"]] * n if case.get("even", False) else _spread(n, case["longest"])
    if op == "tables":
        old = lens if case["grow"] else [0] * n
        new = [x + case["grow"] for x in lens]
        tokens = sum(new) - sum(old)
        ids = sum(-(-y // b) - -(-x // b) for x, y in zip(old, new))
        touched = sum(-(-y // b) - x // b for x, y in zip(old, new))
        return {"bytes": 8 * n + 4 * (n + 1) + 4 * (tokens + 13) + 4 * (ids + touched), "flops": 0}
    h, d, e = case["heads"], case["dim"], 2 if case["type"] == "bf16" else 4
    f = h * d
    if op == "write":
        return {"bytes": case["tokens"] * (2 * f * (e + (2 if case["source"] == "bf16" else 4)) + 4), "flops": 0}
    pages = sum(-(-x // b) for x in lens)
    if op == "bounds":
        rows = sum(lens) if case["fresh"] else sum((x - 1) % b + 1 for x in lens)
        pages = pages if case["fresh"] else n
        return {"bytes": rows * f * e + pages * (2 * f * e + 4) + 8 * n, "flops": 2 * rows * f}
    hq = h * case["group"]
    ends = 2 * n * hq * d * e + 4 * n * hq + 4 * n
    if op == "attend":
        return {"bytes": 2 * sum(lens) * f * e + 4 * pages + ends, "flops": 4 * hq * d * sum(lens)}
    some = sum(min(x, case["budget"] * b) for x in lens)
    return {"bytes": pages * (2 * f * e + 4) + 2 * some * f * e + 4 * n * h * case["budget"] + ends, "flops": 4 * pages * f + 4 * hq * d * some}


# --------------------------------------------------------------- in 64 bits ---

def exact(case, seed):
    if case["op"] == "tables":
        return None   # whole numbers
    s = prepare(case, seed)
    if case["op"] == "write":
        f = s["k"].shape[-1]
        res = {"k": s["k"].double().view(-1, f), "v": s["v"].double().view(-1, f)}
        for i, slot in enumerate(s["slots"].tolist() if case["tokens"] <= 4096 else []):
            if slot >= 0:
                res["k"][slot], res["v"][slot] = s["k_rows"][i].double(), s["v_rows"][i].double()
        return {x: r.view(s[x].shape) for x, r in res.items()} if case["tokens"] <= 4096 else None
    h, d, b = case["heads"], case["dim"], case["block"]
    lens = s["lens"].tolist()
    if case["op"] == "bounds":
        res = torch.zeros(s["k"].shape[0], 2, h * d, dtype=torch.float64, device=DEV)
        for i, n in enumerate(lens):
            a = int(s["from"][i]) // b
            ids = s["table"][i, a:(n + b - 1) // b].long()
            full = (n - a * b) // b
            if full:
                rows = s["k"][ids[:full]].double()
                res[ids[:full], 0], res[ids[:full], 1] = rows.min(1).values, rows.max(1).values
            if n % b:
                rows = s["k"][ids[full], :n % b].double()
                res[ids[full], 0], res[ids[full], 1] = rows.min(0).values, rows.max(0).values
        return res
    g = case["group"]
    out = torch.zeros(len(lens), h * g * d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(len(lens), h * g, dtype=torch.float64, device=DEV)
    chosen = []
    for i, n in enumerate(lens):
        ids = s["table"][i, :(n + b - 1) // b].long()
        q = s["q"][i].view(h, g, d).double()
        if case["op"] == "sparse":
            first, last = _first_last(case)
            lo, hi = s["bounds"][ids].double().view(-1, 2, h, d).unbind(1)
            take = []
            for j in range(h):
                bound = torch.where(q[j][:, None] >= 0, q[j][:, None] * hi[:, j], q[j][:, None] * lo[:, j]).sum((0, 2)).float()
                bound[:first], bound[max(0, len(ids) - last):] = math.inf, math.inf
                best = torch.sort(bound, descending=True, stable=True).indices[:case["budget"]]
                take.append(torch.sort(best).values)
            chosen.append(take)
        for j in range(h):
            at = torch.arange(n, device=DEV)
            if case["op"] == "sparse":
                at = (chosen[i][j][:, None] * b + torch.arange(b, device=DEV)).reshape(-1)
                at = at[at < n]
            k = s["k"][ids[at // b], at % b, j * d:(j + 1) * d].double()
            v = s["v"][ids[at // b], at % b, j * d:(j + 1) * d].double()
            w = (k @ q[j].t().contiguous()) / math.sqrt(d)
            z = torch.logsumexp(w, 0)
            lse[i, j * g:(j + 1) * g] = z
            p = torch.exp(w - z).t().contiguous()
            out[i, j * g * d:(j + 1) * g * d] = (p @ v).reshape(-1)
    if case["op"] == "attend":
        return {"out": out, "lse": lse}
    return {"chosen": None, "out": out, "lse": lse}
