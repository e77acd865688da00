"""The paged 4-bit key/value cache and the sparse attention over it: the cases
that are measured, and the operators' plain forms.

The cache holds, per position and key/value head, one record of 144 bytes:
64 bytes of key codes (two e2m1 numbers a byte, the even dim in the low
nibble), 64 bytes of value codes, 8 e4m3 key scales and 8 e4m3 value scales
(one per 16 dims).  Position p of a request is record
tables[request, p // page_size] * page_size + p % page_size.
"""
import math

import torch

own = False  # True: `run` calls the framework's operators

DIM = 128
REC = 144
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CUDA = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # a speculative decode step: 48 requests, two tokens each, the drafts taken back after it
        dict(name="plan 48x2", op="plan", requests=48, decode=48, step=2, prompt=0, page=64, longest=16384),
        # a mixed step: 480 decoding requests beside 32 prompts of 2,048 tokens
        dict(name="plan 512 mixed", op="plan", requests=512, decode=480, step=1, prompt=2048, page=64,
             longest=65536),
        # a decode step's new rows stored, and read back as the cache holds them
        dict(name="store 96", op="store", tokens=96, kv_heads=1, page=64, dtype="bf16"),
        # several prompts' rows of one layer stored and handed on rounded
        dict(name="store 65536x2", op="store", tokens=65536, kv_heads=2, page=64, dtype="f16"),
        # part of a context fetched, an odd count from small pages
        dict(name="fetch 4097", op="fetch", tokens=4097, kv_heads=1, page=16, dtype="bf16"),
        # a whole 256K context fetched
        dict(name="fetch 262144", op="fetch", tokens=262144, kv_heads=1, page=64, dtype="bf16"),
        # one decoding request of a million positions: latency
        dict(name="attend 1x8 1M", op="attend", tokens=1, step=1, heads=8, kv_heads=1, select=2048, context=1 << 20,
             page=64, dtype="bf16"),
        # 48 requests x 2 tokens, the row top-k joined with a 128-position window
        dict(name="attend 96x8", op="attend", tokens=96, step=2, heads=8, kv_heads=1, select=2176, context=16384,
             page=64, dtype="bf16"),
        # all 64 heads of a layer on one device
        dict(name="attend 64x64", op="attend", tokens=64, step=1, heads=64, kv_heads=1, select=2048, context=32768,
             page=64, dtype="f16"),
        # four key/value heads, an odd list, small pages, a large batch
        dict(name="attend 512x32/4", op="attend", tokens=512, step=1, heads=32, kv_heads=4, select=1001,
             context=8192, page=16, dtype="bf16"),
        # a prompt chunk over a million positions
        dict(name="prompt 2048x8 1M", op="prompt", tokens=2048, heads=8, select=2048, context=1 << 20, page=64,
             dtype="bf16"),
        # a ragged chunk of a shorter prompt, 16 heads
        dict(name="prompt 777x16", op="prompt", tokens=777, heads=16, select=640, context=40000, page=64,
             dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "fetch", "attend", "attend", "attend", "prompt", "prompt"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if op == "plan":
        requests = _log(rng, 1, 512)
        prompts = rng.randint(0, min(requests, 32))
        return dict(op=op, requests=requests, decode=requests - prompts, step=rng.randint(1, 4),
                    prompt=_log(rng, 16, 2048), page=page, longest=_log(rng, 2048, 65536))
    if op in ("store", "fetch"):
        kv_heads = rng.choice([1, 2, 4])
        return dict(op=op, tokens=_log(rng, 1, 131072 // kv_heads), kv_heads=kv_heads, page=page,
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "attend":
        kv_heads = rng.choice([1, 1, 1, 2, 4])
        group = rng.choice([1, 5, 8, 12, 16, 32, 64, 128])
        heads = kv_heads * group
        select = _log(rng, 1, 4096)
        step = rng.choice([1, 1, 2, 3])
        most = max(1, min(512, (1 << 27) // (heads * select * 8), (1 << 21) // (select * kv_heads)))
        tokens = max(step, _log(rng, 1, most) // step * step)
        return dict(op=op, tokens=tokens, step=step, heads=heads, kv_heads=kv_heads, select=select,
                    context=_log(rng, 16, max(17, min(1 << 17, (1 << 23) // (tokens * kv_heads)))), page=page,
                    dtype=dtype)
    heads = rng.choice([8, 16])
    select = _log(rng, 1, 2048)
    return dict(op=op, tokens=_log(rng, 1, 2048), heads=heads, select=select, context=_log(rng, 64, 1 << 19),
                page=page, dtype=dtype)


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=CUDA)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=CUDA)


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _tables(g, lens, page, width=None):
    """Block tables over a pool whose pages are in no order: (tables [R, P], pages)."""
    need = _pages_of(lens, page)
    total = int(need.sum())
    width = int(need.max()) if width is None else width
    order = torch.randperm(max(total, 1), generator=g, device=CUDA).int()
    j = torch.arange(width, device=CUDA)
    first = torch.cumsum(need, 0) - need
    at = (first[:, None] + j[None, :]).clamp(max=max(total, 1) - 1)
    tables = torch.where(j[None, :] < need[:, None], order[at], torch.full_like(order[at], -1))
    return tables.contiguous(), total


def _random_cache(g, records):
    """`records` records of quantised normal numbers."""
    cache = torch.empty(records, REC, dtype=torch.uint8, device=CUDA)
    for r0 in range(0, records, 1 << 18):
        n = min(1 << 18, records - r0)
        kc, ks = _quantise(_normal(g, n, DIM))
        vc, vs = _quantise(_normal(g, n, DIM))
        cache[r0:r0 + n] = _pack(kc, vc, ks, vs)
    return cache


def prepare(case, seed):
    return {"plan": _prepare_plan, "store": _prepare_rows, "fetch": _prepare_rows, "attend": _prepare_attend,
            "prompt": _prepare_prompt}[case["op"]](case, _gen(seed))


def _prepare_plan(c, g):
    R, page = c["requests"], c["page"]
    u = torch.rand(R, generator=g, device=CUDA, dtype=torch.float64)
    before = torch.exp(u * math.log(c["longest"])).int().clamp(min=1)
    new = torch.full((R,), c["step"], dtype=torch.int32, device=CUDA)
    is_prompt = torch.zeros(R, dtype=torch.bool, device=CUDA)
    is_prompt[torch.randperm(R, generator=g, device=CUDA)[:R - c["decode"]]] = True
    new[is_prompt] = c["prompt"]
    before[is_prompt] = 0
    lens = before + new
    T = int(new.sum())
    held = _pages_of(before, page).int()
    width = (c["longest"] + max(c["prompt"], c["step"]) + page - 1) // page
    tables, used = _tables(g, before, page, width)
    spare = c["decode"] * (c["step"] // page + 2) + (R - c["decode"]) * (c["prompt"] // page + 2) + 7
    pages = used + spare
    free = used + torch.randperm(spare, generator=g, device=CUDA).int()
    i32 = dict(dtype=torch.int32, device=CUDA)
    return dict(op="plan", pages=pages, page=page, lens=lens, new=new, back=before, none=torch.zeros_like(new),
                tables=tables, held=held, free=free, count=torch.tensor([spare], **i32),
                first=torch.empty(R + 1, **i32), token_req=torch.empty(T, **i32), ends=torch.empty(T, **i32),
                slots=torch.empty(T, **i32), status=torch.empty(4, **i32), back_first=torch.empty(R + 1, **i32),
                no_tokens=torch.empty(0, **i32), back_status=torch.empty(4, **i32))


def _prepare_rows(c, g):
    T, H, page = c["tokens"], c["kv_heads"], c["page"]
    pages = (T + page - 1) // page + 3
    slots = torch.randperm(pages, generator=g, device=CUDA)[:, None] * page + torch.arange(page, device=CUDA)
    slots = slots.reshape(-1)[:T].int().contiguous()
    dt = DTYPES[c["dtype"]]
    s = dict(op=c["op"], pages=pages, page=page, kv_heads=H, slots=slots,
             k_out=torch.empty(T, H, DIM, dtype=dt, device=CUDA), v_out=torch.empty(T, H, DIM, dtype=dt, device=CUDA))
    if c["op"] == "fetch":
        s["cache"] = _random_cache(g, pages * page * H)
    else:
        # keys and values are the two halves of a projection's output
        kv = (_normal(g, T, 2, H, DIM) * torch.exp(_normal(g, 1, 2, H, DIM) * 0.5)).to(dt)
        s.update(k=kv[:, 0], v=kv[:, 1], cache=torch.zeros(pages * page * H, REC, dtype=torch.uint8, device=CUDA))
    return s


def _lists(g, ends, select, base=None):
    """Ascending distinct positions below each end, -1 after them: `select` of them, or all where there are fewer."""
    T = ends.numel()
    u = torch.rand(T, select, generator=g, device=CUDA, dtype=torch.float64)
    j = torch.arange(select, device=CUDA, dtype=torch.float64)
    if base is not None:  # most positions from the group's own draws, the others from the token's
        mine = torch.rand(T, select, generator=g, device=CUDA) < 0.05
        u = torch.where(mine, u, base)
    # one position of each of `select` stretches of whole positions
    w = ends.double()[:, None] / select
    lo, hi = torch.floor(j[None, :] * w), torch.floor((j[None, :] + 1) * w)
    spread = (lo + torch.floor(u * (hi - lo))).long()
    low = torch.arange(select, device=CUDA)[None, :]
    idx = torch.where(ends[:, None] > select, torch.minimum(spread, ends.long()[:, None] - 1),
                      torch.where(low < ends[:, None], low, torch.full_like(low, -1)))
    return idx.int().contiguous()


def _prepare_attend(c, g):
    T, H, page, step = c["tokens"], c["heads"], c["page"], c["step"]
    R = T // step
    u = torch.rand(R, generator=g, device=CUDA, dtype=torch.float64)
    lens = torch.exp(u * math.log(8.0)) * (c["context"] / 8.0)
    lens = lens.int().clamp(min=step) if R > 1 else torch.full((1,), max(step, c["context"]), dtype=torch.int32,
                                                               device=CUDA)
    tables, pages = _tables(g, lens, page)
    req = torch.arange(R, device=CUDA).repeat_interleave(step).int()
    ends = lens[req.long()] - (step - 1) + torch.arange(step, device=CUDA).repeat(R).int()
    dt = DTYPES[c["dtype"]]
    return dict(op="attend", pages=pages, page=page, kv_heads=c["kv_heads"], tables=tables, token_req=req,
                cache=_random_cache(g, pages * page * c["kv_heads"]), q=_normal(g, T, H, DIM).to(dt),
                idx=_lists(g, ends, c["select"]), o=torch.empty(T, H, DIM, dtype=dt, device=CUDA),
                lse=torch.empty(T, H, dtype=torch.float32, device=CUDA))


def _prepare_prompt(c, g):
    T, H, page = c["tokens"], c["heads"], c["page"]
    total = max(c["context"], T)
    tables, pages = _tables(g, torch.tensor([total], dtype=torch.int32, device=CUDA), page)
    ends = total - T + 1 + torch.arange(T, device=CUDA, dtype=torch.int32)
    G = 128 // H
    base = torch.rand((T + G - 1) // G, c["select"], generator=g, device=CUDA, dtype=torch.float64)
    base = base.repeat_interleave(G, 0)[:T]
    # a group's tokens see the same positions but for the last few
    seen = torch.minimum(ends, ends[torch.arange(T, device=CUDA) // G * G])
    dt = DTYPES[c["dtype"]]
    return dict(op="prompt", pages=pages, page=page, kv_heads=1, tables=tables,
                token_req=torch.zeros(T, dtype=torch.int32, device=CUDA), cache=_random_cache(g, pages * page),
                q=_normal(g, T, H, DIM).to(dt), idx=_lists(g, seen, c["select"], base),
                o=torch.empty(T, H, DIM, dtype=dt, device=CUDA),
                lse=torch.empty(T, H, dtype=torch.float32, device=CUDA))


# ---------------------------------------------------------------------------
# the plain forms

def _quantise(x):
    """Codes and scale bytes of x [n, 128] (float32): one e4m3 scale per 16 dims, e2m1 codes, ties to even."""
    y = x.reshape(-1, 8, 16)
    # divided by a tensor: a scalar divisor becomes a product with its rounded reciprocal
    largest = y.abs().amax(-1)
    scale = (largest / torch.full_like(largest, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()
    m = torch.where(s[..., None] > 0, y.abs() / s[..., None], torch.zeros_like(y))
    code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int()
            + (m >= 3.5).int() + (m > 5.0).int())
    code = code + 8 * torch.signbit(y).int()
    return code.to(torch.uint8).reshape(-1, DIM), scale.view(torch.uint8).reshape(-1, 8)


def _pack(kc, vc, ks, vs):
    return torch.cat([kc[:, 0::2] | (kc[:, 1::2] << 4), vc[:, 0::2] | (vc[:, 1::2] << 4), ks, vs], 1)


def _expand(codes, scales):
    """float32 values of code bytes [..., 64] and scale bytes [..., 8]."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    value = table[code.long()].unflatten(-1, (8, 16))
    return (value * scales.contiguous().view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _plan_plain(page, pages, lens, new, tables, held, free, count, first, token_req, ends, slots, status):
    R, P = tables.shape
    T, dev = token_req.numel(), lens.device
    need = _pages_of(lens, page)
    grow, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    a, p = grow.sum(), back.sum()
    total = new.sum()
    bad = ((lens < 0) | (new < 0) | (new > lens) | (held < 0) | (held > P)).any()
    zero = torch.zeros_like(total)
    code = torch.where(bad, zero + 4, torch.where((need > P).any(), zero + 2, torch.where(
        total > T, zero + 3, torch.where((a > count[0]) | (count[0] - a + p > free.numel()), zero + 1, zero))))
    ok = code == 0
    c = count[0].long()
    j = torch.arange(P, device=dev)[None, :]
    is_new = ok & (j >= held[:, None]) & (j < need[:, None])
    rank = (torch.cumsum(grow, 0) - grow)[:, None] + j - held[:, None]
    taken = free[(c - 1 - rank).clamp(0, free.numel() - 1)]
    gone = ok & (j >= need[:, None]) & (j < held[:, None])
    place = c - a + p - 1 - ((torch.cumsum(back, 0) - back)[:, None] + j - need[:, None])
    spill = torch.cat([free, free[:1]])  # one place more for what is not given back
    spill[torch.where(gone, place, torch.full_like(place, free.numel())).reshape(-1)] = tables.reshape(-1)
    free.copy_(spill[:-1])
    tables.copy_(torch.where(is_new, taken, torch.where(gone, torch.full_like(tables, -1), tables)))
    held.copy_(torch.where(ok, need, held))
    count.copy_(torch.where(ok, c - a + p, c)[None])
    cu = torch.where(ok, torch.cumsum(new, 0), torch.zeros_like(torch.cumsum(new, 0)))
    first[0] = 0
    first[1:] = cu
    i = torch.arange(T, device=dev)
    r = torch.searchsorted(cu, i, right=True)
    live = r < R
    r = r.clamp(max=R - 1)
    pos = (lens - new)[r] + i - (cu - new)[r]
    pg = tables.reshape(-1)[r * P + (pos // page).clamp(0, P - 1)]
    token_req.copy_(torch.where(live, r, torch.full_like(r, -1)))
    ends.copy_(torch.where(live, pos + 1, torch.zeros_like(pos)))
    slots.copy_(torch.where(live & (pg >= 0) & (pg < pages), pg * page + pos % page, torch.full_like(pos, -1)))
    status.copy_(torch.stack([code, torch.where(code == 1, (a - c).clamp(min=0), zero),
                              torch.where(ok, total, zero), count[0].long()]))


def _attend_plain(s):
    q, idx, H = s["q"].float(), s["idx"], s["kv_heads"]
    T, heads, Kc = q.shape[0], q.shape[1], idx.shape[1]
    seen = idx >= 0
    at = idx.clamp(min=0).long()
    page = s["tables"][s["token_req"].long()[:, None], at // s["page"]].long()
    rec = s["cache"].view(-1, H, REC)[page * s["page"] + at % s["page"]]  # [T, Kc, H, 144]
    rec = rec.permute(0, 2, 1, 3)
    k = _expand(rec[..., 0:64], rec[..., 128:136])
    v = _expand(rec[..., 64:128], rec[..., 136:144])
    qg = q.view(T, H, heads // H, DIM)
    x = (qg @ k.transpose(-1, -2)) * (DIM ** -0.5)
    x = torch.where(seen[:, None, None, :], x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    z = w.sum(-1, keepdim=True)
    o = torch.where(z > 0, (w @ v) / z, torch.zeros_like(z))
    s["o"].copy_(o.reshape(T, heads, DIM))
    s["lse"].copy_((top + torch.log(z)).reshape(T, heads))


# ---------------------------------------------------------------------------
# one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_plain(s):
    if s["op"] == "plan":
        state = (s["tables"], s["held"], s["free"], s["count"])
        _plan_plain(s["page"], s["pages"], s["lens"], s["new"], *state, s["first"], s["token_req"], s["ends"],
                    s["slots"], s["status"])
        _plan_plain(s["page"], s["pages"], s["back"], s["none"], *state, s["back_first"], s["no_tokens"],
                    s["no_tokens"], s["no_tokens"], s["back_status"])
    elif s["op"] == "store":
        H = s["kv_heads"]
        kc, ks = _quantise(s["k"].float())
        vc, vs = _quantise(s["v"].float())
        s["cache"].view(-1, H, REC)[s["slots"].long()] = _pack(kc, vc, ks, vs).view(-1, H, REC)
    if s["op"] in ("store", "fetch"):
        rec = s["cache"].view(-1, s["kv_heads"], REC)[s["slots"].long()]
        s["k_out"].copy_(_expand(rec[..., 0:64], rec[..., 128:136]))
        s["v_out"].copy_(_expand(rec[..., 64:128], rec[..., 136:144]))
    elif s["op"] in ("attend", "prompt"):
        _attend_plain(s)
    return _outputs(s)


def _outputs(s):
    if s["op"] == "plan":
        return {n: s[n] for n in ("first", "token_req", "ends", "slots", "status", "tables", "held", "free", "count",
                                  "back_first", "back_status")}
    if s["op"] in ("store", "fetch"):
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"o": s["o"], "lse": s["lse"]}


def _run_own(s):
    import sparse_attention_indexer_live_gb300 as dsa
    cfg = s.get("cfg")
    if cfg is None:  # the cache's description and the union's workspace, which a program makes once
        cfg = s["cfg"] = dsa.cache_cfg(pages=s["pages"], page_size=s["page"], kv_heads=s.get("kv_heads", 1))
        if s["op"] == "prompt":
            n = dsa.dsa_cache_attention_prompt_workspace(cfg, s["q"], s["idx"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=CUDA)
    if s["op"] == "plan":
        state = (s["tables"], s["held"], s["free"], s["count"])
        dsa.dsa_cache_plan(cfg, s["lens"], s["new"], *state, s["first"], s["token_req"], s["ends"], s["slots"],
                           s["status"])
        dsa.dsa_cache_plan(cfg, s["back"], s["none"], *state, s["back_first"], s["no_tokens"], s["no_tokens"],
                           s["no_tokens"], s["back_status"])
    elif s["op"] == "store":
        dsa.dsa_cache_write(cfg, s["k"], s["v"], s["slots"], s["cache"])
    if s["op"] in ("store", "fetch"):
        dsa.dsa_cache_read(cfg, s["cache"], s["slots"], s["k_out"], s["v_out"])
    elif s["op"] == "attend":
        dsa.dsa_cache_attention(cfg, s["cache"], s["q"], s["idx"], s["token_req"], s["tables"], DIM ** -0.5, s["o"],
                                s["lse"])
    elif s["op"] == "prompt":
        dsa.dsa_cache_attention_prompt(cfg, s["cache"], s["q"], s["idx"], s["tables"], DIM ** -0.5, s["workspace"],
                                       s["o"], s["lse"])
    return _outputs(s)


def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}.get(c.get("dtype"), 0)
    if c["op"] == "plan":
        R = c["requests"]
        T = c["decode"] * c["step"] + (R - c["decode"]) * c["prompt"]
        # both calls: lengths, counts held, tokens' maps, about a page id each way per page's worth of new tokens
        moved = R + T // c["page"]
        return {"bytes": 2 * 4 * (3 * R + 1) + 3 * 4 * T + 2 * 16 * moved + 2 * R * 4, "flops": 0}
    if c["op"] in ("store", "fetch"):
        rows = c["tokens"] * c["kv_heads"]
        once = rows * (2 * DIM * size + REC) + 4 * c["tokens"]
        return {"bytes": once * (2 if c["op"] == "store" else 1), "flops": 0}
    T, H, Kc = c["tokens"], c["heads"], c["select"]
    kv_heads = c.get("kv_heads", 1)
    if c["op"] == "attend":
        # lengths are log-uniform over [context / 8, context]; the listed lists are about full
        mean = c["context"] if T == c["step"] else c["context"] * (7.0 / 8.0) / math.log(8.0)
        per = min(Kc, mean)
        seen = min(T * per, (T // c["step"]) * mean)
        pairs = T * per
    else:
        total = max(c["context"], T)
        per = min(Kc, total)
        # distinct positions: each group's lists and the 5 % of its tokens' own, spread over the context
        groups = -(-T // (128 // H))
        seen = total * -math.expm1(-groups * per * (1 + 0.05 * min(T, 128 // H)) / total)
        pairs = T * per
    io = T * H * (2 * DIM * size + 4) + 4 * T * Kc
    return {"bytes": seen * REC * kv_heads + io, "flops": 4.0 * DIM * H * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _plan_exact(s)
    if case["op"] == "store":
        return {"k": _rounded_exact(s["k"]), "v": _rounded_exact(s["v"])}
    values = _codes_exact(s["cache"])
    H = s["kv_heads"]
    if case["op"] == "fetch":
        at = s["slots"].long()[:, None] * H + torch.arange(H, device=CUDA)[None, :]
        return {"k": values(at, 0), "v": values(at, 1)}
    T, heads = s["q"].shape[:2]
    o = torch.zeros(T, heads, DIM, dtype=torch.float64, device=CUDA)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64, device=CUDA)
    few = max(1, (1 << 20) // (s["idx"].shape[1] * H))
    for t0 in range(0, T, few):  # a few tokens at a time: 64-bit rows are large
        idx = s["idx"][t0:t0 + few].long()
        n = idx.shape[0]
        keep = idx >= 0
        pos = torch.where(keep, idx, torch.zeros_like(idx))
        row = s["tables"][s["token_req"][t0:t0 + few].long()].long()
        slot = torch.gather(row, 1, pos // s["page"]) * s["page"] + pos % s["page"]
        for h in range(H):
            k, v = values(slot * H + h, 0), values(slot * H + h, 1)
            qh = s["q"][t0:t0 + few].double().view(n, H, heads // H, DIM)[:, h]
            x = torch.einsum("tgd,tjd->tgj", qh, k) / math.sqrt(DIM)
            x = x.masked_fill(~keep[:, None, :], -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - z[..., None]).nan_to_num(0.0)
            a, b = h * (heads // H), (h + 1) * (heads // H)
            o[t0:t0 + few, a:b] = torch.einsum("tgj,tjd->tgd", w, v)
            lse[t0:t0 + few, a:b] = z
    return {"o": o, "lse": lse}


def _codes_exact(cache):
    """values(records, which): 64-bit rows of the keys (0) or values (1) of records of the cache."""
    byte = torch.arange(256, device=CUDA, dtype=torch.float64)
    e, m, sign = torch.floor(byte / 8) % 16, byte % 8, torch.where(byte >= 128, -1.0, 1.0)
    scale_of = sign * torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)
    nibble = byte[:16]
    e, m, sign = torch.floor(nibble / 2) % 4, nibble % 2, torch.where(nibble >= 8, -1.0, 1.0)
    code_of = sign * torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1), m / 2)

    def values(records, which):
        rows = cache[records.reshape(-1)]
        b = rows[:, 64 * which:64 * which + 64].long()
        out = torch.empty(rows.shape[0], DIM, dtype=torch.float64, device=CUDA)
        out[:, 0::2], out[:, 1::2] = code_of[b % 16], code_of[b // 16]
        scale = scale_of[rows[:, 128 + 8 * which:136 + 8 * which].long()]
        return (out * scale.repeat_interleave(16, 1)).view(*records.shape, DIM)

    return values


def _rounded_exact(x):
    """The rows of x as the cache holds them, from the nearest e4m3 and e2m1 numbers."""
    y = x.double().reshape(*x.shape[:-1], 8, 16)
    a = y.abs().amax(-1)
    a = torch.clamp(a / torch.full_like(a, 6.0), max=448.0)
    one = torch.ones_like(a)
    # 3 bits after the leading one; from a table, since powers computed on a GPU are not exact
    powers = torch.tensor([2.0 ** e for e in range(-9, 6)], dtype=torch.float64, device=a.device)
    step = powers[(torch.frexp(a.clamp(min=2.0 ** -6)).exponent + 5).long()]
    s = torch.clamp(torch.round(a / step) * step, max=448.0)
    m = (y / torch.where(s > 0, s, one)[..., None]).clamp(-6, 6)
    step = torch.where(m.abs() < 2, 0.5, torch.where(m.abs() < 4, 1.0, 2.0)).double()
    return (torch.round(m / step) * step * s[..., None]).reshape(x.shape)


def _plan_exact(s):
    page, pages, T = s["page"], s["pages"], s["token_req"].numel()
    lens, new = s["lens"].tolist(), s["new"].tolist()
    tables, held, stack = s["tables"].cpu(), s["held"].tolist(), s["free"].tolist()
    count = int(s["count"][0])
    req, ends, slots, first = [], [], [], [0]
    rows = [t[:h].tolist() for t, h in zip(tables, held)]
    top = count
    for r, (n, k) in enumerate(zip(lens, new)):
        while len(rows[r]) < -(-n // page):
            top -= 1
            rows[r].append(stack[top])
        for p in range(n - k, n):
            req.append(r)
            ends.append(p + 1)
            slots.append(rows[r][p // page] * page + p % page)
        first.append(len(req))
    # the step back leaves the tables and the list as they were
    t = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"first": t(first), "token_req": t(req), "ends": t(ends), "slots": t(slots), "status": t([0, 0, T, top]),
            "tables": tables, "held": t(held), "free": t(stack), "count": t([count]),
            "back_first": t([0] * len(first)), "back_status": t([0, 0, 0, count])}
