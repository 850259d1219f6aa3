"""The cases on which the operators of the 8-bit paged cache are measured.

Two operators: `append` rotates the new tokens' queries and keys and appends keys and values to the cache (a page of 64
tokens of one KV head goes to 8 bits, with a power-of-two scale for its keys and one for its values, once it is complete;
the newest tokens stay in bf16), `attend` is exact attention over that cache. A case says how many requests there are, how
many tokens each has in the cache and how many are new; where these are ranges, `lengths` spreads them over the requests.
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
def _case(name, op, batch, kv_heads, group, past, new, rot=D, interleaved=False, topk=0):
    c = {"op": op, "batch": batch, "kv_heads": kv_heads, "group": group, "past_lo": past[0], "past_hi": past[1],
         "new_lo": new[0], "new_hi": new[1], "rot": rot, "interleaved": interleaved, "topk": topk}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a single user's next token: nothing but latency
        _case("append one token", "append", 1, 8, 5, (777, 777), (1, 1)),
        # a full serving batch with mixed contexts: one token each, some of them completing a page
        _case("append batch of 256", "append", 256, 8, 8, (8192, 32768), (1, 1)),
        # one prompt, as long as a chunk gets, ending inside a page
        _case("append prompt 8191", "append", 1, 8, 5, (0, 0), (8191, 8191)),
        # prompt chunks of many requests at once, onto contexts of any length; half of the head rotated, in pairs
        _case("append ragged chunks", "append", 24, 2, 7, (0, 20000), (1, 2048), rot=64, interleaved=True),
        # the tiny configuration: one request, four heads of their own
        _case("decode 4K, one request", "attend", 1, 4, 1, (4095, 4095), (1, 1)),
        # the measured serving configuration, dense: 32 requests of 32K
        _case("decode 32K, 32 requests", "attend", 32, 8, 5, (32767, 32767), (1, 1)),
        # one very long request: the work has to be split over the context
        _case("decode 1M, one request", "attend", 1, 8, 5, (1048575, 1048575), (1, 1)),
        # contexts from one token to 16K in one batch, the largest group
        _case("decode ragged, 48 requests", "attend", 48, 2, 16, (0, 16383), (1, 1)),
        # the sparse step: 32 pages a head that Select chose, and the newest tokens
        _case("decode 32 pages of 32K", "attend", 32, 8, 5, (32700, 32767), (1, 1), topk=32),
        # five drafted tokens verified at once
        _case("verify 5 tokens", "attend", 16, 8, 8, (4000, 16384), (5, 5)),
        # prompts from their start, of mixed lengths
        _case("prompts to 6000", "attend", 4, 8, 5, (0, 0), (300, 6000)),
        # one chunk of a long prompt onto the 30,000 tokens before it
        _case("chunk 2048 onto 30000", "attend", 1, 8, 8, (30000, 30000), (2048, 2048)),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm where that spans more than a factor of ten."""
    if hi > 10 * max(lo, 1):
        return min(hi, int(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi + 1)))))
    return rng.randint(lo, hi)


def draw(rng):
    op = rng.choice(["append", "attend"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    kind = rng.choice(["one", "few", "many"])
    if kind == "one":
        batch, new = _spread(rng, 1, 256), (1, 1)
    elif kind == "few":
        n = rng.randint(2, 12)
        batch, new = _spread(rng, 1, 64), (rng.randint(1, n), n)
    else:
        n = _spread(rng, 13, 4096)
        batch, new = _spread(rng, 1, 16), (rng.randint(1, n), n)
    hi = _spread(rng, 1, 400000)
    if op == "append":  # what is cached costs nothing there; the new rows do
        batch = max(1, min(batch, 30000 // new[1]))
    else:               # keys in all, and pairs of queries and keys in all
        hi = max(1, min(hi, 6000000 // (batch * kv_heads) - new[1], 1500000000 // (batch * kv_heads * group * new[1])))
        while batch * kv_heads * group * new[1] * (hi + new[1]) > 1700000000 and batch > 1:
            batch //= 2
    lo = rng.choice([0, hi // 2, hi])
    rot = rng.choice([D, D, 96, 64, 32])
    topk = rng.choice([0, 0, _spread(rng, 1, 128)]) if op == "attend" and kind == "one" else 0
    return _case("", op, batch, kv_heads, group, (lo, hi), new, rot, rng.random() < 0.5, topk)


def lengths(case):
    """(tokens in the cache before the call, new tokens) of each request: they follow from the case alone."""
    rng = random.Random("%(op)s %(batch)d %(past_lo)d %(past_hi)d %(new_lo)d %(new_hi)d" % case)
    out = []
    for _ in range(case["batch"]):
        past, new = _spread(rng, case["past_lo"], case["past_hi"]), rng.randint(case["new_lo"], case["new_hi"])
        # An append that both completes the open page and opens another replaces the rows that it started from. So
        # that a pass finds the state that the last one found, such a request's new tokens end with a page here.
        if case["op"] == "append" and past % PAGE and past % PAGE + new > PAGE:
            new -= (past + new) % PAGE
        out.append((past, new))
    return out


def work(case):
    hkv, hq = case["kv_heads"], case["kv_heads"] * case["group"]
    read = written = flops = 0
    for past, new in lengths(case):
        n = past + new
        if case["op"] == "append":
            full = n // PAGE - past // PAGE
            kept = n % PAGE if full else new       # rows that stay in bf16
            old = past % PAGE if full else 0       # rows read back from there
            read += (hq + 2 * hkv) * new * D * 2 + 2 * old * hkv * D * 2
            written += hq * new * D * 2 + 2 * full * hkv * (PAGE * D + 4) + 2 * kept * hkv * D * 2
            flops += 3 * (hq + hkv) * new * case["rot"]
        else:
            full, tail = n // PAGE, n % PAGE
            if case["topk"]:
                full = min(full, case["topk"])
            read += hkv * (2 * full * (PAGE * D + 4) + 2 * tail * D * 2) + hq * new * D * 2
            written += hq * new * D * 2
            seen = full * PAGE + tail
            flops += 4 * D * hq * (new * seen - new * (new - 1) // 2)
    return {"bytes": read + written, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _inv_freq(rot):
    return [1e6 ** (-2.0 * j / rot) for j in range(rot // 2)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, H, G = case["batch"], case["kv_heads"], case["group"]
    both = lengths(case)
    past, new = [p for p, _ in both], [n for _, n in both]
    total, cu = sum(new), [0]
    for n in new:
        cu.append(cu[-1] + n)
    full = [(p + n) // PAGE for p, n in both]
    first = [p // PAGE if case["op"] == "append" else 0 for p in past]   # pages before it lie outside the pool
    P = max(1, max(full))
    ints = dict(dtype=torch.int32, device=dev)
    s = {"op": case["op"], "group": G, "rot": case["rot"], "interleaved": case["interleaved"], "pages_max": P,
         "new_max": max(new), "past": torch.tensor(past, **ints), "cu": torch.tensor(cu, **ints), "inv_freq": _inv_freq(case["rot"])}

    # The pool: every page of every head once, in an order of its own. Pages outside it are -1 in the table.
    per_b = [f - a for a, f in zip(first, full)]
    n_pages = max(1, H * sum(per_b))
    place = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    held = (torch.arange(P, device=dev)[None, :] >= torch.tensor(first, device=dev)[:, None]) & (
        torch.arange(P, device=dev)[None, :] < torch.tensor(full, device=dev)[:, None])
    held = held[:, None, :].expand(B, H, P)
    table = torch.full((B, H, P), -1, **ints)
    table[held] = place[: int(held.sum())]
    s["table"] = table

    # Keys have channels that are larger than others; values do not.
    loud = torch.exp(0.7 * torch.randn((H, 1, D), generator=g, device=dev))
    width = (H * G + 2 * H) * D
    s["tails"] = torch.randn((B, H, 2, PAGE, D), generator=g, device=dev).mul_(
        torch.stack([loud, torch.ones_like(loud)], 1)).to(torch.bfloat16)
    if case["op"] == "append":
        rows = torch.randn((total, width), generator=g, device=dev, dtype=torch.float32)
        rows[:, H * G * D:(H * G + H) * D] *= loud.expand(H, 1, D).reshape(-1)
        rows = rows.to(torch.bfloat16)           # one projection's output: q, k and v lie side by side
        s["q"] = rows[:, : H * G * D].view(total, H * G, D)
        s["k"] = rows[:, H * G * D:(H * G + H) * D].view(total, H, D)
        s["v"] = rows[:, (H * G + H) * D:].view(total, H, D)
        s["pages"] = torch.zeros((n_pages, 2, PAGE, D), dtype=torch.uint8, device=dev)
        s["scales"] = torch.ones((n_pages, 2), device=dev)
        s["q_out"] = torch.empty((total, H * G, D), dtype=torch.bfloat16, device=dev)
    else:
        pages = torch.empty((n_pages, 2, PAGE, D), dtype=torch.uint8, device=dev)
        scales = torch.empty((n_pages, 2), device=dev)
        tone = torch.exp(0.7 * torch.randn((1, 1, 1, D), generator=g, device=dev))
        for a in range(0, n_pages, 16384):
            x = torch.randn((min(16384, n_pages - a), 2, PAGE, D), generator=g, device=dev)
            x[:, 0:1] *= tone
            x *= torch.exp(0.3 * torch.randn((x.shape[0], 2, 1, 1), generator=g, device=dev))
            sc = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / TOP)))
            pages[a:a + 16384] = (x / sc[:, :, None, None]).to(F8).view(torch.uint8)
            scales[a:a + 16384] = sc
        s["pages"], s["scales"] = pages, scales
        s["q"] = (1.3 * torch.randn((total, H * G, D), generator=g, device=dev)).to(torch.bfloat16)
        s["out"] = torch.empty((total, H * G, D), dtype=torch.bfloat16, device=dev)
        s["sel"] = None
        if case["topk"]:
            k = case["topk"]
            rank = torch.rand((B, H, P), generator=g, device=dev).masked_fill_(~held, 2.0)
            val, idx = rank.sort(-1)
            idx = torch.where(val < 2.0, idx, P)[..., :k].sort(-1).values
            idx = torch.cat([idx, torch.full((B, H, max(0, k - P)), P, device=dev, dtype=idx.dtype)], -1)
            s["sel"] = torch.where(idx < P, idx, -1).to(torch.int32).reshape(B * H, k).contiguous()

    # Where each new token and each page that gets new tokens belongs.
    n_t, p_t = torch.tensor(new, device=dev), torch.tensor(past, device=dev)
    s["tok_b"] = torch.repeat_interleave(torch.arange(B, device=dev), n_t)
    s["tok_i"] = torch.arange(total, device=dev) - torch.tensor(cu[:-1], device=dev)[s["tok_b"]]
    if case["op"] == "append":
        touched = (p_t + n_t - 1) // PAGE - p_t // PAGE + 1
        base = torch.cumsum(touched, 0) - touched
        s["tp_b"] = torch.repeat_interleave(torch.arange(B, device=dev), touched)
        s["tp_p"] = torch.arange(int(touched.sum()), device=dev) - (base - p_t // PAGE)[s["tp_b"]]
        s["tp_first"] = base
        at = p_t[s["tok_b"]] + s["tok_i"]
        s["tok_tp"], s["tok_row"] = base[s["tok_b"]] + at // PAGE - (p_t // PAGE)[s["tok_b"]], at % PAGE
        s["tp_rows"] = torch.clamp((p_t + n_t)[s["tp_b"]] - s["tp_p"] * PAGE, max=PAGE)
        s["tp_full"] = torch.nonzero(s["tp_rows"] == PAGE)[:, 0]
        s["tp_open"] = torch.nonzero(s["tp_rows"] < PAGE)[:, 0]
    if own:
        import sparse_attention_tiered_gb300 as spin

        rope = spin.SpinRope(s["inv_freq"], interleaved=case["interleaved"])
        s["cache"] = spin.SpinKV8(B, H * G, H, P, pages=s["pages"], scales=s["scales"], tails=s["tails"], table=table, rope=rope)
        s["step"] = spin.SpinKV8Step(s["past"], s["cu"], total_new=total, max_new=max(new))
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(s):
    if own:
        if s["op"] == "append":
            s["cache"].append(s["step"], s["q"], s["k"], s["v"], s["q_out"])
            return {"q": s["q_out"], "pages": s["pages"].view(F8), "scales": s["scales"], "tails": s["tails"]}
        s["cache"].attend(s["step"], s["q"], s["out"], sel=s["sel"])
        return s["out"]
    return plain_append(s) if s["op"] == "append" else plain_attend(s)


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2:rot])
    y, z = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def plain_append(s):
    angle = (s["past"][s["tok_b"]].double() + s["tok_i"].double())[:, None] * torch.tensor(
        s["inv_freq"], dtype=torch.float64, device=s["q"].device)
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    q = _rotate(s["q"], cos, sin, s["rot"], s["interleaved"])
    k = _rotate(s["k"], cos, sin, s["rot"], s["interleaved"])
    H = k.shape[1]
    held = torch.zeros((s["tp_b"].numel(), 2, PAGE, H, D), dtype=torch.bfloat16, device=k.device)
    held[s["tp_first"]] = s["tails"].permute(0, 2, 3, 1, 4)
    held[s["tok_tp"], 0, s["tok_row"]] = k
    held[s["tok_tp"], 1, s["tok_row"]] = s["v"]
    done = held[s["tp_full"]].float().permute(0, 3, 1, 2, 4)                 # [pages][H][2][64][128]
    frac, exp = torch.frexp(done.abs().amax((3, 4)))
    scale = torch.exp2(torch.clamp(exp - 9 + (frac > 0.875).int(), min=-64).float())
    at = s["table"][s["tp_b"][s["tp_full"]], :, s["tp_p"][s["tp_full"]]].long()
    s["pages"][at] = (done / scale[..., None, None]).to(F8).view(torch.uint8)
    s["scales"][at] = scale
    open_b = s["tp_b"][s["tp_open"]]
    rows = torch.arange(PAGE, device=k.device)[None, :] < s["tp_rows"][s["tp_open"]][:, None]
    s["tails"][open_b] = torch.where(rows[:, None, None, :, None], held[s["tp_open"]].permute(0, 3, 1, 2, 4), s["tails"][open_b])
    return {"q": q, "pages": s["pages"].view(F8), "scales": s["scales"], "tails": s["tails"]}


def plain_attend(s):
    dev = s["q"].device
    table, B, H = s["table"], s["table"].shape[0], s["table"].shape[1]
    new = s["cu"][1:] - s["cu"][:-1]
    n = (s["past"] + new).long()
    full = n // PAGE
    sel = torch.arange(s["pages_max"], device=dev).expand(B, H, -1) if s["sel"] is None else s["sel"].view(B, H, -1).long()
    there = (sel >= 0) & (sel < full[:, None, None])
    at = torch.where(there, table.gather(2, sel.clamp(min=0)).long(), 0)
    x = s["pages"][at].view(F8).float() * s["scales"][at][..., None, None]   # [B][H][P][2][64][128]
    tail = s["tails"].float()[:, :, None]
    x = torch.cat([x, tail], 2)
    row = torch.arange(PAGE, device=dev)
    pos = torch.cat([sel[..., None] * PAGE + row, (full * PAGE)[:, None, None, None] + row.expand(B, H, 1, PAGE)], 2)
    seen = torch.cat([there[..., None].expand(-1, -1, -1, PAGE), (pos[:, :, -1:] < n[:, None, None, None])], 2)
    M = pos.shape[2] * PAGE
    pos, seen = pos.reshape(B, H, 1, M), seen.reshape(B, H, 1, M)
    key, val = x[:, :, :, 0].reshape(B, H, M, D), x[:, :, :, 1].reshape(B, H, M, D)
    val = torch.where(seen.transpose(2, 3), val, 0.0)
    N, G = s["new_max"], s["group"]
    q = torch.zeros((B, N, H, G, D), device=dev)
    q[s["tok_b"], s["tok_i"]] = s["q"].float().view(-1, H, G, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    w = torch.matmul(q, key.transpose(2, 3)) * (1.0 / math.sqrt(D))
    upto = (s["past"].long()[:, None] + torch.arange(N, device=dev))[:, None, :, None].expand(B, 1, N, G).reshape(B, 1, N * G, 1)
    w = w.masked_fill_(~(seen & (pos <= upto)), -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, val) / torch.where(total == 0, 1.0, total)
    o = o.view(B, H, N, G, D).permute(0, 2, 1, 3, 4)[s["tok_b"], s["tok_i"]]
    return o.reshape(-1, H * G, D).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------------------
# the operators' definition, in 64 bits, request by request
# ---------------------------------------------------------------------------------------------------------------
def _to_e4m3(x):
    """x (float64, |x| <= 448) to the nearest e4m3 value, ties to the even one."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6.0)
    unit = torch.exp2(e - 3.0)
    return torch.round(x / unit) * unit


def _exact_append(case, s):
    B, H, hq, rot = case["batch"], case["kv_heads"], case["kv_heads"] * case["group"], case["rot"]
    q_out = torch.empty((s["q"].shape[0], hq, D), dtype=torch.float64, device="cuda")
    pages, scales, tails = s["pages"].view(F8).double(), s["scales"].double(), s["tails"].double()
    freq = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
    at = 0
    for b, (past, new) in enumerate(lengths(case)):
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.arange(past, past + new, device="cuda").double()[:, None] * freq)

        def turned(x):
            x = x.double()
            if case["interleaved"]:
                z = torch.view_as_real(torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2).contiguous()) * turn[:, None]).flatten(-2)
            else:
                z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn[:, None]
                z = torch.cat([z.real, z.imag], -1)
            return torch.cat([z, x[..., rot:]], -1)

        q_out[at:at + new] = turned(s["q"][at:at + new])
        k, v = turned(s["k"][at:at + new]).to(torch.bfloat16).double(), s["v"][at:at + new].double()
        at += new
        for h in range(H):
            old = past % PAGE
            rows = torch.stack([torch.cat([tails[b, h, 0, :old], k[:, h]]), torch.cat([tails[b, h, 1, :old], v[:, h]])])
            whole = rows.shape[1] // PAGE
            for c in range(0, whole, 4096):
                m = min(4096, whole - c)
                x = rows[:, c * PAGE:(c + m) * PAGE].reshape(2, m, PAGE, D).transpose(0, 1)
                sc = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / TOP)).clamp(min=-64.0))
                where = s["table"][b, h, past // PAGE + c:past // PAGE + c + m].long()
                pages[where], scales[where] = _to_e4m3(x / sc[..., None, None]), sc
            tails[b, h, :, : rows.shape[1] - whole * PAGE] = rows[:, whole * PAGE:]
    return {"q": q_out, "pages": pages, "scales": scales, "tails": tails}


def _exact_attend(case, s):
    H, G, k = case["kv_heads"], case["group"], case["topk"]
    out = torch.zeros((s["q"].shape[0], H * G, D), dtype=torch.float64, device="cuda")
    at = 0
    for b, (past, new) in enumerate(lengths(case)):
        n = past + new
        whole, rest = n // PAGE, n % PAGE
        for h in range(H):
            which = torch.arange(whole, device="cuda")
            if k:
                which = s["sel"][b * H + h].long()
                which = which[which >= 0]
            where = s["table"][b, h, which].long()
            x = s["pages"][where].view(F8).double() * s["scales"][where].double()[:, :, None, None]
            key = torch.cat([x[:, 0].reshape(-1, D), s["tails"][b, h, 0, :rest].double()])
            val = torch.cat([x[:, 1].reshape(-1, D), s["tails"][b, h, 1, :rest].double()])
            pos = torch.cat([(which[:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1),
                             whole * PAGE + torch.arange(rest, device="cuda")])
            for i in range(0, new, 1024):
                m = min(1024, new - i)
                q = s["q"][at + i:at + i + m, h * G:(h + 1) * G].double()
                w = torch.einsum("igd,jd->gij", q, key) / math.sqrt(D)
                w.masked_fill_(pos[None, None, :] > past + i + torch.arange(m, device="cuda")[None, :, None], -math.inf)
                w = torch.nan_to_num(torch.softmax(w, -1)) if pos.numel() else w
                out[at + i:at + i + m, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", w, val)
        at += new
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attend(case, s)
