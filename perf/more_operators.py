"""The cases on which the sparse path over the 8-bit paged cache and the operators of its page pool are measured.

Five operators. `select` scores the complete pages that each new token sees by their mean keys and lists the best of them,
for each token and KV head; `attend` is attention over such lists (each token has its own, and the newest tokens up to
itself); `reserve` takes free pages of the pool for the pages that a step will complete; `fork` makes requests copies of
others, sharing their pages (a request that becomes a copy of none is emptied, and pages that nobody names are free again);
`compact` moves the pages in use to the front of the pool. A case says how many requests there are, how many tokens each
has in the cache and how many are new; where these are ranges, `lengths` spreads them over the requests.
"""
import math
import random

import torch

own = False

D = 128          # head dim
PAGE = 64        # tokens of a page
F8 = torch.float8_e4m3fn
TOP = 448.0      # the largest e4m3 value


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def _case(name, op, batch, kv_heads, past, new=(1, 1), group=1, topk=0, drift=0.0, pool=0, fork=1, alive=1, moved=0, apart=0):
    """drift: how much of a token's preferences the next one keeps. pool: pages of the pool beyond those in use, in parts of
    1/16 of them. fork, alive, moved, apart: requests come in groups of `fork`, of which the first `alive` hold something
    and share all but their last `apart` pages, and `moved` become copies of others."""
    c = {"op": op, "batch": batch, "kv_heads": kv_heads, "group": group, "past_lo": past[0], "past_hi": past[1],
         "new_lo": new[0], "new_hi": new[1], "topk": topk, "drift": drift, "pool": pool, "fork": fork, "alive": alive,
         "moved": moved, "apart": apart}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the measured serving configuration: the next token of 32 requests of 32K
        _case("select 32K of 32 requests", "select", 32, 8, (32767, 32767), group=5, topk=32, drift=0.9),
        # one very long request's next token: few rows, many pages
        _case("select 1M of one request", "select", 1, 8, (1048575, 1048575), group=5, topk=128, drift=0.9),
        # one chunk of a long prompt: many rows over the same pages
        _case("select chunk 2048 onto 30000", "select", 1, 8, (30000, 30000), (2048, 2048), group=8, topk=32, drift=0.95),
        # five drafted tokens verified at once, each over its own pages
        _case("attend 5 drafts of 16 requests", "attend", 16, 8, (4000, 32768), (5, 5), group=8, topk=32, drift=0.9),
        # prompts and continuations of mixed lengths, odd groups, short lists
        _case("attend ragged prompts", "attend", 6, 2, (0, 9000), (1, 1500), group=7, topk=15, drift=0.95),
        # one chunk of a long prompt onto the 30,000 tokens before it
        _case("attend chunk 2048 onto 30000", "attend", 1, 8, (30000, 30000), (2048, 2048), group=8, topk=32, drift=0.95),
        # the decode step of a full serving batch: a page now and then, nothing but latency
        _case("reserve one token of 256 requests", "reserve", 256, 8, (8192, 32768), pool=4),
        # prompt chunks of many requests at once
        _case("reserve ragged chunks", "reserve", 24, 8, (0, 20000), (1, 2048), pool=16),
        # one prompt sampled eight times: the copies share its pages
        _case("fork a prompt into 8", "fork", 8, 8, (30050, 30050), fork=8, alive=1, moved=7, pool=4),
        # beam search: in each of 16 groups half of the 8 beams go on as copies of others
        _case("reorder 16 groups of 8 beams", "fork", 128, 8, (1000, 8000), fork=8, alive=8, moved=4, apart=3, pool=2),
        # a small pool, most of it free again
        _case("compact a small pool", "compact", 4, 4, (500, 4000), pool=24),
        # a gigabyte of pages, half of them free
        _case("compact a pool of 1 GB", "compact", 16, 8, (12000, 20000), pool=16),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm where that spans more than a factor of ten."""
    if hi > 10 * max(lo, 1):
        return min(hi, int(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1)))))
    return rng.randint(lo, hi)


def draw(rng):
    op = rng.choice(["select", "attend", "reserve", "fork", "compact"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    if op in ("select", "attend"):
        group = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
        kind = rng.choice(["one", "few", "many"])
        if kind == "one":
            batch, new = _spread(rng, 1, 256), (1, 1)
        elif kind == "few":
            n = rng.randint(2, 12)
            batch, new = _spread(rng, 1, 64), (rng.randint(1, n), n)
        else:
            n = _spread(rng, 13, 2048)
            batch, new = _spread(rng, 1, 16), (rng.randint(1, n), n)
            batch = max(1, min(batch, 4096 // n))
        topk = _spread(rng, 1, 128)
        hi = _spread(rng, 1, 400000)
        rows = batch * kv_heads * new[1]
        if op == "select":   # scores in all, and summaries in all
            hi = max(1024, min(hi, 64 * 8000000 // rows, 64 * 130000 // (batch * kv_heads)))
            topk = min(topk, hi // PAGE // 4 + 1)  # of pages that every row sees, so that there is something to select
        else:                # keys in all, what the lists gather, and pairs of queries and keys
            topk = max(1, min(topk, 520000 // rows))
            hi = max(1, min(hi, 6000000 // (batch * kv_heads) - new[1], 4300000000 // (rows * group)))
        lo = rng.choice([hi // 2, hi] if op == "select" else [0, hi // 2, hi])
        return _case("", op, batch, kv_heads, (lo, hi), new, group, topk, rng.choice([0.0, 0.9, 0.95, 0.98]))
    pages = _spread(rng, 200, 30000)     # in all, or thereabouts
    if op == "fork":
        fork = rng.choice([2, 3, 4, 8])
        batch = fork * _spread(rng, 1, 32)
        alive = rng.choice([1, fork])
        moved = fork - 1 if alive == 1 else rng.randint(1, fork - 1)
        hi = max(200, pages * PAGE // (batch // fork * kv_heads))
        return _case("", op, batch, kv_heads, (rng.choice([hi // 3, hi]), hi), fork=fork, alive=alive, moved=moved,
                     apart=rng.randint(0, 5) if alive > 1 else 0, pool=rng.randint(1, 32))
    batch = _spread(rng, 1, 256 if op == "reserve" else 32)
    hi = max(100, pages * PAGE // (batch * kv_heads))
    new = (1, 1)
    if op == "reserve" and rng.random() < 0.6:
        n = _spread(rng, 2, 4096)
        new = (rng.randint(1, n), n)
    return _case("", op, batch, kv_heads, (rng.choice([hi // 8, hi // 2]), hi), new, pool=rng.randint(16, 48))


def lengths(case):
    """(tokens in the cache before the call, new tokens) of each request: they follow from the case alone."""
    rng = random.Random("%(op)s %(batch)d %(past_lo)d %(past_hi)d %(new_lo)d %(new_hi)d" % case)
    out = []
    for b in range(case["batch"]):
        past, new = _spread(rng, case["past_lo"], case["past_hi"]), rng.randint(case["new_lo"], case["new_hi"])
        i = b % case["fork"]
        if i:  # a group's requests are as long as its first, or empty
            past = out[b - i][0] if i < case["alive"] else 0
        out.append((past, new))
    return out


def _pages_in_use(case):
    """(pages of a group's first requests, pages that the others have of their own), of one head."""
    first = own_ones = 0
    for b, (past, _) in enumerate(lengths(case)):
        if b % case["fork"] == 0:
            first += past // PAGE
        else:
            own_ones += min(case["apart"], past // PAGE)
    return first, own_ones


def work(case):
    op, H, G, k = case["op"], case["kv_heads"], case["group"], case["topk"]
    both = lengths(case)
    used = H * sum(_pages_in_use(case))
    pool = used + used * case["pool"] // 16
    moved_bytes = flops = 0
    if op == "select":
        for past, new in both:
            seen = (past + new) // PAGE
            moved_bytes += H * seen * D * 4 + H * G * new * D * 2 + H * new * k * 4
            flops += 2 * D * H * sum((past + i + 1) // PAGE for i in range(new)) + H * (G - 1) * D * new
    elif op == "attend":
        for past, new in both:
            n = past + new
            listed_tokens = sum(min(k, (past + i + 1) // PAGE) * PAGE + (past + i + 1) % PAGE for i in range(new))
            whole = min(n // PAGE, k * new + (n // PAGE - past // PAGE))  # the most pages that its lists can name
            if case["drift"] and new > 1:  # each token adds about this share of its list to what the others name
                whole = min(whole, int(k * (1 + (new - 1) * 0.5 * (1 - case["drift"]))) + n // PAGE - past // PAGE)
            moved_bytes += H * (2 * whole * (PAGE * D + 4) + 4 * (n % PAGE) * D) + 4 * H * G * new * D + 4 * H * new * min(k, n // PAGE)
            flops += 4 * D * H * G * listed_tokens
    elif op == "reserve":
        need = H * sum((p + n) // PAGE - p // PAGE for p, n in both)
        moved_bytes = 4 * pool + 8 * case["batch"] + 12 * need
    elif op == "fork":
        for a in range(0, case["batch"], case["fork"]):
            past = both[a][0]
            pages = past // PAGE
            differ = min(pages, case["apart"]) if case["alive"] > 1 else pages
            per = H * (pages * 12 + differ * 8 + 2 * differ * D * 4 + 2 * 2 * (past % PAGE) * D * 2)
            moved_bytes += case["moved"] * per
        moved_bytes += 12 * case["batch"]
    else:
        go = used * (pool - used) // max(1, pool)
        moved_bytes = 4 * pool + 4 * used + go * (2 * (2 * PAGE * D + 8) + 12)
    return {"bytes": moved_bytes, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _table(case, both, g, s, P):
    """The pool's state: a table, a count of the entries that name each page, and lengths, in one array of 32-bit numbers."""
    dev = torch.device("cuda")
    B, H = case["batch"], case["kv_heads"]
    past = torch.tensor([p for p, _ in both], device=dev)
    p = torch.arange(P, device=dev)
    b = torch.arange(B, device=dev)
    there = p < (past // PAGE)[:, None]
    first = b - b % case["fork"]
    shared = there & (first != b)[:, None] & (p < (past // PAGE - case["apart"])[:, None])
    mine = (there & ~shared)[:, None, :].expand(B, H, P)
    used = int(mine.sum())
    n_pages = max(1, used + used * case["pool"] // 16)
    place = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, H, P), -1, dtype=torch.int32, device=dev)
    table[mine] = place[:used]
    table = torch.where(shared[:, None, :], table[first], table)
    refs = torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)
    s["first"] = torch.cat([table.flatten(), refs, past.to(torch.int32)])
    s["now"] = s["first"].clone()
    s["table"] = s["now"][: table.numel()].view(B, H, P)
    s["refs"] = s["now"][table.numel(): table.numel() + n_pages]
    s["past"] = s["now"][table.numel() + n_pages:]
    return n_pages


def _lists(case, both, g, P):
    """The pages that a selection picks for each token and head: its likes drift from token to token."""
    dev = torch.device("cuda")
    B, H, k, a = case["batch"], case["kv_heads"], case["topk"], case["drift"]
    past = torch.tensor([p for p, _ in both], device=dev)
    page = torch.arange(P, device=dev)
    x = torch.randn((B, H, P), generator=g, device=dev)
    out = torch.empty((max(n for _, n in both), B, H, k), dtype=torch.int32, device=dev)
    noise = torch.empty_like(x)
    for i in range(out.shape[0]):
        if i:
            x = x.mul_(a).add_(noise.normal_(generator=g), alpha=math.sqrt(1.0 - a * a))
        y = x.masked_fill(page >= ((past + i + 1) // PAGE)[:, None, None], -math.inf)
        val, idx = y.topk(min(k, P), -1)
        idx = torch.where(val > -math.inf, idx, P).sort(-1).values
        out[i, :, :, : idx.shape[-1]] = torch.where(idx < P, idx, -1)
        out[i, :, :, idx.shape[-1]:] = -1
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, B, H, G, k = case["op"], case["batch"], case["kv_heads"], case["group"], case["topk"]
    both = lengths(case)
    past, new = [p for p, _ in both], [n for _, n in both]
    if op in ("fork", "compact"):
        new = [0] * B
    total, cu = sum(new), [0]
    for n in new:
        cu.append(cu[-1] + n)
    full = [(p + n) // PAGE for p, n in zip(past, new)]
    P = max(1, max(full))
    ints = dict(dtype=torch.int32, device=dev)
    s = {"op": op, "group": G, "topk": k, "pages_max": P, "new_max": max(new), "cu": torch.tensor(cu, **ints)}
    n_t = torch.tensor(new, device=dev)
    s["tok_b"] = torch.repeat_interleave(torch.arange(B, device=dev), n_t)
    s["tok_i"] = torch.arange(total, device=dev) - torch.tensor(cu[:-1], device=dev)[s["tok_b"]]

    if op == "select":
        s["past"] = torch.tensor(past, **ints)
        s["table"] = torch.zeros((B, H, P), **ints)
        n_pages = 1
        # Mean keys: channels that are larger than others, and a part that all of a head's pages have in common.
        loud = torch.exp(0.5 * torch.randn((1, H, 1, D), generator=g, device=dev))
        s["summaries"] = torch.randn((B, H, P, D), generator=g, device=dev)
        s["summaries"] += 0.5 * torch.randn((1, H, 1, D), generator=g, device=dev)
        s["summaries"] *= 0.5 * loud
        # Queries drift from token to token.
        q = torch.empty((s["new_max"], B, H * G, D), device=dev)
        x, noise = torch.randn((B, H * G, D), generator=g, device=dev), torch.empty((B, H * G, D), device=dev)
        for i in range(s["new_max"]):
            q[i] = x
            x = x.mul_(case["drift"]).add_(noise.normal_(generator=g), alpha=math.sqrt(1.0 - case["drift"] ** 2))
        s["q"] = q[s["tok_i"], s["tok_b"]].to(torch.bfloat16)
        s["sel"] = torch.empty((total, H, k), **ints)
    elif op == "attend":
        s["past"] = torch.tensor(past, **ints)
        n_pages = max(1, H * sum(full))
        place = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        held = (torch.arange(P, device=dev) < torch.tensor(full, device=dev)[:, None])[:, None, :].expand(B, H, P)
        s["table"] = torch.full((B, H, P), -1, **ints)
        s["table"][held] = place[: int(held.sum())]
        # Keys have channels that are larger than others; values do not.
        pages, scales = torch.empty((n_pages, 2, PAGE, D), dtype=torch.uint8, device=dev), torch.empty((n_pages, 2), device=dev)
        loud = torch.exp(0.7 * torch.randn((1, 1, 1, D), generator=g, device=dev))
        for a in range(0, n_pages, 16384):
            x = torch.randn((min(16384, n_pages - a), 2, PAGE, D), generator=g, device=dev)
            x[:, 0:1] *= loud
            x *= torch.exp(0.3 * torch.randn((x.shape[0], 2, 1, 1), generator=g, device=dev))
            sc = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / TOP)))
            pages[a:a + 16384] = (x / sc[:, :, None, None]).to(F8).view(torch.uint8)
            scales[a:a + 16384] = sc
        s["pages"], s["scales"] = pages, scales
        s["tails"] = torch.randn((B, H, 2, PAGE, D), generator=g, device=dev).to(torch.bfloat16)
        s["q"] = (1.3 * torch.randn((total, H * G, D), generator=g, device=dev)).to(torch.bfloat16)
        s["sel"] = _lists(case, both, g, P)[s["tok_i"], s["tok_b"]].contiguous()
        s["out"] = torch.empty((total, H * G, D), dtype=torch.bfloat16, device=dev)
    else:
        n_pages = _table(case, both, g, s, P)
        s["free"] = torch.zeros(1, **ints)
        if op == "compact":
            s["pages"] = torch.randint(0, 127, (n_pages, 2, PAGE, D), dtype=torch.uint8, generator=g, device=dev)
            s["scales"] = torch.exp2(torch.randint(-12, 3, (n_pages, 2), generator=g, device=dev).float())
        if op == "fork":
            s["summaries"] = torch.randn((B, H, P, D), generator=g, device=dev)
            s["tails"] = torch.randn((B, H, 2, PAGE, D), generator=g, device=dev).to(torch.bfloat16)
            rng = random.Random(seed)
            src = list(range(B))
            for a in range(0, B, case["fork"]):  # those that go on keep their places; the others become copies of them
                gone = rng.sample(range(a + (case["alive"] == 1), a + case["fork"]), case["moved"])
                stay = [b for b in range(a, a + case["alive"]) if b not in gone]
                for b in gone:
                    src[b] = rng.choice(stay)
            s["src"] = torch.tensor(src, **ints)
    if own:
        import sparse_attention_tiered_gb300 as spin

        def like(name, shape, dtype):  # what the operator does not look at
            return s[name] if name in s else torch.zeros(shape, dtype=dtype, device=dev)

        s["cache"] = spin.SpinKV8(B, H * G, H, P, pages=like("pages", (n_pages, 2, PAGE, D), torch.uint8),
                                  scales=like("scales", (n_pages, 2), torch.float32),
                                  tails=like("tails", (B, H, 2, PAGE, D), torch.bfloat16), table=s["table"],
                                  summaries=s.get("summaries", False), refs=s.get("refs", False))
        s["step"] = spin.SpinKV8Step(s["past"], s["cu"], total_new=total, max_new=max(1, s["new_max"]))
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if op in ("reserve", "fork", "compact"):
        s["now"].copy_(s["first"])  # every pass starts from the same pool
        if own:
            if op == "reserve":
                s["cache"].reserve(s["step"], free_pages=s["free"])
            elif op == "fork":
                s["cache"].fork(s["past"], s["src"])
            else:
                s["cache"].compact(free_pages=s["free"])
        else:
            {"reserve": plain_reserve, "fork": plain_fork, "compact": plain_compact}[op](s)
        out = {"table": s["table"], "refs": s["refs"]}
        if op == "fork":
            return dict(out, lengths=s["past"], tails=s["tails"], summaries=s["summaries"])
        out["free"] = s["free"]
        return out if op == "reserve" else dict(out, pages=s["pages"].view(F8), scales=s["scales"])
    if own:
        if op == "select":
            return s["cache"].select(s["step"], s["q"], s["sel"])
        return s["cache"].attend_rows(s["step"], s["q"], s["out"], s["sel"])
    return plain_select(s) if op == "select" else plain_attend(s)


def plain_select(s):
    """In 64 bits: a page just above the border and one just below it differ by less than 32 bits hold."""
    B, H, P, k = s["table"].shape[0], s["table"].shape[1], s["pages_max"], s["topk"]
    dev = s["q"].device
    N, total = s["new_max"], s["q"].shape[0]
    q = torch.zeros((B, N, H, D), dtype=torch.float64, device=dev)
    q[s["tok_b"], s["tok_i"]] = s["q"].double().view(total, H, -1, D).sum(2)
    score = torch.matmul(q.transpose(1, 2), s["summaries"].double().transpose(2, 3))       # [B][H][N][P]
    seen = (s["past"].long()[:, None] + torch.arange(N, device=dev) + 1) // PAGE           # [B][N]
    score.masked_fill_(torch.arange(P, device=dev) >= seen[:, None, :, None], -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    there = torch.arange(order.shape[-1], device=dev) < seen[:, None, :, None]
    order = torch.where(there, order, P).sort(-1).values
    out = torch.full((B, H, N, k), -1, dtype=torch.int32, device=dev)
    out[..., : order.shape[-1]] = torch.where(order < P, order, -1)
    return out.transpose(1, 2)[s["tok_b"], s["tok_i"]].contiguous()


def plain_attend(s):
    dev = s["q"].device
    H, G, total = s["table"].shape[1], s["group"], s["q"].shape[0]
    past = s["past"].long()
    length = past + (s["cu"][1:] - s["cu"][:-1])
    heads, row = torch.arange(H, device=dev), torch.arange(PAGE, device=dev)
    out = torch.empty((total, H * G, D), dtype=torch.bfloat16, device=dev)
    step = max(1, 16384 // (H * (s["topk"] + 2)))  # tokens at a time: a gigabyte of keys and values
    for a in range(0, total, step):
        b, i = s["tok_b"][a:a + step], s["tok_i"][a:a + step]
        see = past[b] + i + 1
        sel = s["sel"][a:a + step].long()
        last = (see // PAGE)[:, None, None].expand(-1, H, 1)   # the page that the token itself is in, or the next one
        in_pool = last < (length[b] // PAGE)[:, None, None]
        sel = torch.cat([torch.where((sel >= 0) & (sel < last), sel, -1), torch.where(in_pool, last, -1)], -1)
        page = s["table"][b[:, None, None], heads[None, :, None], sel.clamp(min=0)].long().clamp(min=0)
        x = s["pages"][page].view(F8).float() * s["scales"][page][..., None, None]         # [T][H][k + 1][2][64][128]
        x = torch.cat([x, s["tails"][b][:, :, None].float()], 2)
        pos = torch.cat([sel, torch.where(in_pool, -1, last)], -1)
        tok = pos[..., None] * PAGE + row
        hidden = ((pos < 0)[..., None] | (tok >= see[:, None, None, None])).flatten(2)
        key, val = x[:, :, :, 0].flatten(2, 3), x[:, :, :, 1].flatten(2, 3).masked_fill(hidden[..., None], 0.0)
        q = s["q"][a:a + step].float().view(-1, H, G, D)
        w = torch.matmul(q, key.transpose(2, 3)) * (1.0 / math.sqrt(D))
        w = w.masked_fill_(hidden[:, :, None, :], -math.inf)
        top = w.amax(-1, keepdim=True)
        w = w.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
        sums = w.sum(-1, keepdim=True)
        out[a:a + step] = (torch.matmul(w, val) / torch.where(sums == 0, 1.0, sums)).view(-1, H * G, D).to(torch.bfloat16)
    return out


def plain_reserve(s):
    past, table, refs = s["past"].long(), s["table"], s["refs"]
    length = past + (s["cu"][1:] - s["cu"][:-1])
    p = torch.arange(s["pages_max"], device=refs.device)
    want = ((p >= (past // PAGE)[:, None]) & (p < (length // PAGE)[:, None]))[:, None, :] & (table < 0)
    rank = torch.cumsum(want.flatten(), 0).view_as(want)
    free = torch.cumsum(refs == 0, 0)
    want &= rank[-1, -1, -1] <= free[-1]
    page = torch.searchsorted(free, rank).clamp(max=refs.numel() - 1)
    refs.scatter_add_(0, page.flatten(), want.flatten().to(torch.int32))
    table.copy_(torch.where(want, page.to(torch.int32), table))
    s["free"].copy_((refs == 0).sum())


def plain_fork(s):
    past, table, refs, src = s["past"], s["table"], s["refs"], s["src"].long()
    B = src.numel()
    moved, there, a = src != torch.arange(B, device=src.device), src >= 0, src.clamp(min=0)
    length = torch.where(there, past[a], 0)
    p, row = torch.arange(s["pages_max"], device=src.device), torch.arange(PAGE, device=src.device)
    whole = (p < (length // PAGE)[:, None])[:, None, :]
    new = torch.where(whole, table[a], -1)
    at = moved[:, None, None]
    refs.scatter_add_(0, table.flatten().long().clamp(min=0), -(at & (table >= 0)).flatten().to(torch.int32))
    refs.scatter_add_(0, new.flatten().long().clamp(min=0), (at & (new >= 0)).flatten().to(torch.int32))
    s["summaries"].copy_(torch.where((at & whole)[..., None], s["summaries"][a], s["summaries"]))
    table.copy_(torch.where(at, new, table))
    kept = (moved[:, None] & (row < (length % PAGE)[:, None]))[:, None, None, :, None]
    s["tails"].copy_(torch.where(kept, s["tails"][a], s["tails"]))
    past.copy_(torch.where(moved, length, past))


def plain_compact(s):
    table, refs = s["table"], s["refs"]
    used = refs > 0
    n = used.sum()
    at = torch.arange(refs.numel(), device=refs.device)
    go = torch.nonzero(used & (at >= n))[:, 0]
    to = torch.nonzero(~used)[:, 0][: go.numel()]
    place = at.to(torch.int32)
    place[go] = to.to(torch.int32)
    s["pages"][to], s["scales"][to], refs[to] = s["pages"][go], s["scales"][go], refs[go]
    refs[go] = 0
    table.copy_(torch.where(table >= 0, place[table.clamp(min=0).long()], table))
    s["free"].copy_(refs.numel() - n)


# ---------------------------------------------------------------------------------------------------------------
# the operators' definition, in 64 bits, request by request
# ---------------------------------------------------------------------------------------------------------------
def _exact_select(case, s):
    H, G, k = case["kv_heads"], case["group"], case["topk"]
    out = torch.full((s["q"].shape[0], H, k), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, (past, new) in enumerate(lengths(case)):
        pages = (past + new) // PAGE
        for h in range(H if pages else 0):
            key = s["summaries"][b, h, :pages].double()
            for i in range(0, new, 256):
                m = min(256, new - i)
                q = s["q"][at + i:at + i + m, h * G:(h + 1) * G].double()
                score = torch.einsum("tgd,pd->tp", q, key)
                last = (past + i + 1 + torch.arange(m, device="cuda")) // PAGE
                score[torch.arange(pages, device="cuda")[None] >= last[:, None]] = -math.inf
                # the k-th largest, then all above it and the first of those that equal it
                n = min(k, pages)
                border = score.topk(n, -1).values[:, -1:]
                above, equal = score > border, score == border
                take = above | (equal & (torch.cumsum(equal, -1) <= n - above.sum(-1, keepdim=True)))
                take &= score > -math.inf
                t, p = torch.nonzero(take, as_tuple=True)
                out[at + i + t, h, torch.cumsum(take, -1)[t, p] - 1] = p.to(torch.int32)
        at += new
    return out


def _exact_attend(case, s):
    H, G = case["kv_heads"], case["group"]
    out = torch.zeros((s["q"].shape[0], H * G, D), dtype=torch.float64, device="cuda")
    at = 0
    for b, (past, new) in enumerate(lengths(case)):
        n = past + new
        whole, rest = n // PAGE, n % PAGE
        for h in range(H):
            where = s["table"][b, h, :whole].long()
            x = s["pages"][where].view(F8).double() * s["scales"][where].double()[:, :, None, None]
            key = torch.cat([x[:, 0].reshape(-1, D), s["tails"][b, h, 0, :rest].double()])
            val = torch.cat([x[:, 1].reshape(-1, D), s["tails"][b, h, 1, :rest].double()])
            for i in range(0, new, 256):
                m = min(256, new - i)
                see = past + i + 1 + torch.arange(m, device="cuda")
                may = torch.zeros((m, whole + 2), dtype=torch.bool, device="cuda")
                sel = s["sel"][at + i:at + i + m, h].long()
                sel = torch.where((sel >= 0) & (sel < (see // PAGE)[:, None]), sel, whole + 1)
                may.scatter_(1, sel, True)
                may.scatter_(1, (see // PAGE)[:, None], True)  # the newest tokens
                may = may[:, : whole + 1].repeat_interleave(PAGE, 1)[:, :n] & (torch.arange(n, device="cuda") < see[:, None])
                q = s["q"][at + i:at + i + m, h * G:(h + 1) * G].double()
                w = torch.einsum("igd,jd->igj", q, key) / math.sqrt(D)
                w.masked_fill_(~may[:, None, :], -math.inf)
                w = torch.nan_to_num(torch.softmax(w, -1))
                out[at + i:at + i + m, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", w, val)
        at += new
    return out


def _exact_pool(case, s):
    """Page by page, in plain Python."""
    B, H, P = s["table"].shape
    table, refs = s["table"].cpu().tolist(), s["refs"].cpu().tolist()
    ints = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "reserve":
        wanted = [(b, h, p) for b, (past, new) in enumerate(lengths(case)) for h in range(H)
                  for p in range(past // PAGE, (past + new) // PAGE) if table[b][h][p] < 0]
        free = [i for i, r in enumerate(refs) if r == 0]
        if len(wanted) <= len(free):
            for (b, h, p), i in zip(wanted, free):
                table[b][h][p], refs[i] = i, 1
        return {"table": torch.tensor(table, **ints), "refs": torch.tensor(refs, **ints),
                "free": torch.tensor([refs.count(0)], **ints)}
    if case["op"] == "compact":
        n = sum(r > 0 for r in refs)
        holes = iter([i for i in range(n) if refs[i] == 0])
        place = {i: next(holes) for i in range(n, len(refs)) if refs[i] > 0}
        pages, scales = s["pages"].view(F8).double(), s["scales"].double()
        if place:
            a, z = torch.tensor(list(place), device="cuda"), torch.tensor(list(place.values()), device="cuda")
            pages[z], scales[z] = pages[a], scales[a]
        for a, z in place.items():
            refs[z], refs[a] = refs[a], 0
        table = [[[place.get(x, x) for x in row] for row in head] for head in table]
        return {"table": torch.tensor(table, **ints), "refs": torch.tensor(refs, **ints),
                "free": torch.tensor([len(refs) - n], **ints), "pages": pages, "scales": scales}
    past = s["past"].cpu().tolist()
    now, tails, summaries = list(past), s["tails"].double(), s["summaries"].double()
    new_table = [[list(row) for row in head] for head in table]
    for b, a in enumerate(s["src"].cpu().tolist()):
        if a == b:
            continue
        n = now[b] = past[a] if a >= 0 else 0
        for h in range(H):
            for p in range(P):
                x, y = table[b][h][p], table[a][h][p] if p < n // PAGE else -1
                if x >= 0:
                    refs[x] -= 1
                if y >= 0:
                    refs[y] += 1
                new_table[b][h][p] = y
        if a >= 0:
            tails[b, :, :, : n % PAGE] = s["tails"][a, :, :, : n % PAGE].double()
            summaries[b, :, : n // PAGE] = s["summaries"][a, :, : n // PAGE].double()
    return {"table": torch.tensor(new_table, **ints), "refs": torch.tensor(refs, **ints), "lengths": torch.tensor(now, **ints),
            "tails": tails, "summaries": summaries}


def exact(case, seed):
    s = prepare(case, seed)
    return {"select": _exact_select, "attend": _exact_attend}.get(case["op"], _exact_pool)(case, s)
