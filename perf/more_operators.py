"""The paged key/value cache in 16 bits: the cases that are measured, and the
operators' plain forms.

The cache is two tensors [pages, page_size, kv_heads, 128]: position p of a
request is row p % page_size of page tables[request, p // page_size].  A third
one, [pages, kv_heads, 128], holds each full page's mean key.  Four operators:

    append  a step's rotated keys and its values stored, its queries rotated,
            the means of the pages that it fills
    attend  causal attention of a step's tokens (single ones, drafts, prompt
            chunks, in one batch) to everything before them
    select  the pages that each token's queries score highest, by the mean keys
    blocks  attention to a selection of pages
"""
import math

import torch

own = False  # True: `run` calls the framework's operators

DIM = 128
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
CUDA = "cuda"


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # a speculative decode step: 48 requests, two tokens each
        dict(name="append 48x2", op="append", decode=48, step=2, prompts=0, prompt=0, context=512, heads=32, kv_heads=8,
             page=64, rot=128, neighbours=False, theta=1e6, dtype="bf16"),
        # a prompt chunk of one layer, far into a long context
        dict(name="append 8192", op="append", decode=0, step=1, prompts=1, prompt=8192, context=16384, heads=32,
             kv_heads=8, page=64, rot=128, neighbours=False, theta=1e6, dtype="bf16"),
        # decoding requests beside ragged prompts, half of the dims rotated, neighbours paired, small pages
        dict(name="append mixed", op="append", decode=29, step=1, prompts=3, prompt=777, context=2000, heads=24,
             kv_heads=2, page=16, rot=64, neighbours=True, theta=1e4, dtype="f16"),
        # one short request: latency
        dict(name="attend 1x8 300", op="attend", decode=1, step=1, prompts=0, prompt=0, context=300, heads=8, kv_heads=1,
             page=64, dtype="bf16"),
        # one token of a long request, all SMs on one key/value head
        dict(name="attend 1x8 128K", op="attend", decode=1, step=1, prompts=0, prompt=0, context=131072, heads=8,
             kv_heads=1, page=64, dtype="bf16"),
        # a decode step of 64 requests of all lengths
        dict(name="attend 64x32/8", op="attend", decode=64, step=1, prompts=0, prompt=0, context=16384, heads=32,
             kv_heads=8, page=64, dtype="bf16"),
        # a mixed step: drafts of three tokens beside ragged prompt chunks, an odd group, small pages
        dict(name="attend mixed", op="attend", decode=31, step=3, prompts=3, prompt=777, context=5000, heads=24,
             kv_heads=2, page=16, dtype="f16"),
        # a prompt chunk over 32K positions
        dict(name="attend 4096x32/8", op="attend", decode=0, step=1, prompts=1, prompt=4096, context=32768, heads=32,
             kv_heads=8, page=64, dtype="bf16"),
        # the pages of a decode step's requests of up to 128K positions
        dict(name="select 64", op="select", decode=64, step=1, prompts=0, prompt=0, context=131072, heads=32, kv_heads=4,
             page=64, select=16, lead=1, trail=2, dtype="bf16"),
        # the pages of a prompt chunk over 128K positions
        dict(name="select 2048", op="select", decode=0, step=1, prompts=1, prompt=2048, context=131072, heads=32,
             kv_heads=4, page=64, select=16, lead=1, trail=2, dtype="bf16"),
        # the same step's attention
        dict(name="blocks 64", op="blocks", decode=64, step=1, prompts=0, prompt=0, context=131072, heads=32, kv_heads=4,
             page=64, select=16, dtype="bf16"),
        # a prompt chunk's: neighbours share most of their pages
        dict(name="blocks 2048", op="blocks", decode=0, step=1, prompts=1, prompt=2048, context=131072, heads=32,
             kv_heads=4, page=64, select=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "select", "select", "blocks", "blocks"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 5, 8, 8, 12, 16])
    heads = kv_heads * group
    c = dict(op=op, heads=heads, kv_heads=kv_heads, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "f16"]))
    kind = rng.choice(["decode", "decode", "prompt", "mixed"])
    c["step"] = rng.choice([1, 1, 2, 3])
    c["decode"] = 0 if kind == "prompt" else _log(rng, 1, 64)
    c["prompts"] = 0 if kind == "decode" else 1 if kind == "prompt" else rng.randint(1, 3)
    c["prompt"] = 0 if kind == "decode" else _log(rng, 2, 2048)
    requests = c["decode"] + c["prompts"]
    if op == "append":
        c["context"] = max(c["step"], c["prompt"], _log(rng, 16, max(17, 32768 // requests)))
        c["rot"] = rng.choice([32, 64, 96, 128, 128, 128])
        c["neighbours"] = rng.random() < 0.3
        c["theta"] = rng.choice([1e4, 5e5, 1e6])
        return c
    # keys held: at most 2^20 positions of all heads; work: at most a quarter of the largest listed chunk's
    most = min(131072, (1 << 20) // (requests * kv_heads), (1 << 30) // (heads * (c["prompts"] * c["prompt"] + 1)))
    c["context"] = max(c["step"], c["prompt"], _log(rng, 16, max(17, most)))
    if op in ("select", "blocks"):
        c["select"] = rng.choice([7, 8, 8, 16, 16, 32])
        if op == "select":
            # pages to choose from: four times as many as are chosen
            c["select"] = max(7, min(c["select"], most // (4 * c["page"])))
            c["context"] = max(c["context"], 4 * c["select"] * c["page"])
            c["lead"] = rng.choice([0, 1, 1, 2])
            c["trail"] = rng.choice([1, 1, 2])
    return c


def _shape(c):
    """(lengths after the step, new tokens) of every request: ragged, and of the case alone."""
    lens, new = [], []
    for r in range(c["decode"]):
        part = 1.0 if c["decode"] == 1 else 8.0 ** -((r * 0.6180339887498949) % 1.0)
        lens.append(max(c["step"], int(c["context"] * part)))
        new.append(c["step"])
    for r in range(c["prompts"]):
        n = max(1, c["prompt"] - r * 37 % (c["prompt"] // 4 + 1))
        new.append(n)
        lens.append(max(n, c["context"] - r * 101 % (c["context"] // 8 + 1)))
    return lens, new


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=CUDA)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=CUDA)


def _rows(g, n, heads, dt, channel):
    """Rows of heads whose channels differ in size, as trained projections' do."""
    out = torch.empty(n, heads, DIM, dtype=dt, device=CUDA)
    for a in range(0, n, 1 << 16):
        b = min(n, a + (1 << 16))
        out[a:b] = (_normal(g, b - a, heads, DIM) * channel).to(dt)
    return out


def prepare(case, seed):
    c, g = case, _gen(seed)
    lens, new = _shape(c)
    page, H, Hk, dt = c["page"], c["heads"], c["kv_heads"], DTYPES[c["dtype"]]
    i32 = dict(dtype=torch.int32, device=CUDA)
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=g, device=CUDA).int()
    tables = torch.full((len(lens), width), -1, **i32)
    at = 0
    for r, n in enumerate(need):
        tables[r, :n] = order[at:at + n]
        at += n
    first = [0]
    for n in new:
        first.append(first[-1] + n)
    T = first[-1]
    s = dict(op=c["op"], page=page, pages=pages, kv_heads=Hk, heads=H, dt=dt, lens_list=lens, new_list=new,
             first_list=first, tables=tables, lens=torch.tensor(lens, **i32), first=torch.tensor(first, **i32),
             scale=DIM ** -0.5)
    k_size = torch.exp(_normal(g, Hk, DIM) * 0.4)
    if c["op"] == "append":
        # queries, keys and values lie side by side, as one projection leaves them
        qkv = _rows(g, T, H + 2 * Hk, dt, torch.exp(_normal(g, H + 2 * Hk, DIM) * 0.4))
        ends, slots = [], []
        host = tables.cpu().tolist()
        for r, (n, f) in enumerate(zip(lens, new)):
            for p in range(n - f, n):
                ends.append(p + 1)
                slots.append(host[r][p // page] * page + p % page)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:], ends=torch.tensor(ends, **i32),
                 slots=torch.tensor(slots, **i32), neighbours=c["neighbours"],
                 inv_freq=c["theta"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=CUDA) / c["rot"]),
                 q_out=torch.empty(T, H, DIM, dtype=dt, device=CUDA), means=_rows(g, pages, Hk, dt, k_size))
    else:
        q_size = torch.exp(_normal(g, H, DIM) * 0.4)
        s["q"] = _rows(g, T, H, dt, q_size)
    if c["op"] == "select":
        # mean keys: what a head's keys share, and what the page's own add
        shared = _normal(g, Hk, DIM) * k_size * 0.3
        s["means"] = (_rows(g, pages, Hk, torch.float32, k_size * 0.25) + shared).to(dt)
        s.update(lead=c["lead"], trail=c["trail"], idx=torch.empty(T, Hk, c["select"], **i32))
        return s
    s["k_cache"] = _rows(g, pages * page, Hk, dt, k_size).view(pages, page, Hk, DIM)
    s["v_cache"] = _rows(g, pages * page, Hk, dt, 1.0).view(pages, page, Hk, DIM)
    if c["op"] in ("attend", "blocks"):
        s.update(o=torch.empty(T, H, DIM, dtype=dt, device=CUDA), lse=torch.empty(T, H, dtype=torch.float32, device=CUDA))
    if c["op"] == "blocks":
        s["idx"] = torch.cat([_page_lists(g, n, f, page, Hk, c["select"]) for n, f in zip(lens, new)]).contiguous()
    return s


def _page_lists(g, n, f, page, kv_heads, select):
    """Ascending pages [f, kv_heads, select] of a request's last f tokens, -1 after them: the first page, the token's
    own, and others, of which runs of 64 neighbours share most."""
    own_page = (torch.arange(n - f, n, device=CUDA) // page)[:, None, None]
    most = (n - 1) // page + 1
    score = torch.rand(-(-f // 64), kv_heads, most, generator=g, device=CUDA).repeat_interleave(64, 0)[:f]
    mine = torch.rand(f, kv_heads, most, generator=g, device=CUDA)
    score = torch.where(mine < 0.002, mine + 1.0, score)
    j = torch.arange(most, device=CUDA)
    score = torch.where((j == 0) | (j == own_page), torch.full_like(score, 3.0), score)
    score = torch.where(j > own_page, torch.full_like(score, -1.0), score)
    best, at = torch.topk(score, min(select, most), dim=-1)
    at = torch.where(best < 0, torch.full_like(at, 1 << 30), at).sort(-1).values
    out = torch.full((f, kv_heads, select), -1, dtype=torch.int32, device=CUDA)
    out[..., :at.shape[-1]] = torch.where(at == 1 << 30, torch.full_like(at, -1), at).int()
    return out


# ---------------------------------------------------------------------------
# the plain forms

def _rotate(x, ends, inv_freq, neighbours):
    """Rows x [T, heads, 128] (float32) turned by their positions; the angles in 64 bits."""
    half = inv_freq.numel()
    angle = (ends.double() - 1)[:, None] * inv_freq
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    turned = x[..., :2 * half]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if neighbours else (turned[..., :half], turned[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if neighbours else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _append_plain(s):
    page, Hk = s["page"], s["kv_heads"]
    slots = s["slots"].long()
    s["q_out"].copy_(_rotate(s["q"].float(), s["ends"], s["inv_freq"], s["neighbours"]))
    k = _rotate(s["k"].float(), s["ends"], s["inv_freq"], s["neighbours"])
    s["k_cache"].view(-1, Hk, DIM)[slots] = k.to(s["dt"])
    s["v_cache"].view(-1, Hk, DIM)[slots] = s["v"]
    filled = slots[slots % page == page - 1] // page
    s["means"][filled] = s["k_cache"][filled].float().mean(1).to(s["dt"])


def _gathered(s, r, h, pages=None):
    """Keys and values [positions, 128] of request r's head h (float32)."""
    n = s["lens_list"][r]
    ids = s["tables"][r, :-(-n // s["page"])].long()
    k = s["k_cache"][ids, :, h].reshape(-1, DIM)[:n]
    v = s["v_cache"][ids, :, h].reshape(-1, DIM)[:n]
    return k.float(), v.float()


def _softmax_plain(x, seen, v):
    """(o, lse) of scores x [.., n], of which those seen count, and values v [n, 128]."""
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    w = torch.exp(x - top)
    z = w.sum(-1, keepdim=True)
    return torch.where(z > 0, (w @ v) / z, torch.zeros_like(z)), (top + torch.log(z))[..., 0]


def _attend_plain(s):
    group = s["heads"] // s["kv_heads"]
    for r, (n, f) in enumerate(zip(s["lens_list"], s["new_list"])):
        a, b = s["first_list"][r], s["first_list"][r + 1]
        pos = torch.arange(n - f, n, device=CUDA)
        for h in range(s["kv_heads"]):
            k, v = _gathered(s, r, h)
            q = s["q"][a:b, h * group:(h + 1) * group].float().transpose(0, 1)
            seen = torch.arange(n, device=CUDA)[None, :] <= pos[:, None]
            if s["op"] == "blocks":
                own_pages = torch.zeros(f, -(-n // s["page"]) + 1, dtype=torch.bool, device=CUDA)
                own_pages.scatter_(1, s["idx"][a:b, h].long() + 1, True)  # the column before the first takes the -1s
                seen = seen & own_pages[:, 1:].repeat_interleave(s["page"], 1)[:, :n]
            o, lse = _softmax_plain((q @ k.transpose(0, 1)) * s["scale"], seen, v)
            s["o"][a:b, h * group:(h + 1) * group] = o.transpose(0, 1).to(s["dt"])
            s["lse"][a:b, h * group:(h + 1) * group] = lse.transpose(0, 1)


def _select_plain(s):
    page, Hk, n_out = s["page"], s["kv_heads"], s["idx"].shape[2]
    group = s["heads"] // Hk
    s["idx"].fill_(-1)
    for r, (n, f) in enumerate(zip(s["lens_list"], s["new_list"])):
        a, b = s["first_list"][r], s["first_list"][r + 1]
        ids = s["tables"][r, :-(-n // page)].long()
        own_page = (torch.arange(n - f, n, device=CUDA) // page)[:, None, None]
        q = s["q"][a:b].double().view(f, Hk, group, DIM).sum(2)
        # in 64 bits: neighbours in rank may differ by less than 32 bits hold
        score = torch.einsum("thd,jhd->thj", q, s["means"][ids].double())
        j = torch.arange(ids.numel(), device=CUDA)
        pinned = (j < s["lead"]) | (j > own_page - s["trail"])
        score = torch.where(pinned, torch.full_like(score, math.inf), score)
        score = torch.where(j > own_page, torch.full_like(score, -math.inf), score)
        best = torch.argsort(score, dim=-1, descending=True, stable=True)[..., :n_out]
        gone = best > own_page
        best = torch.where(gone, torch.full_like(best, 1 << 30), best).sort(-1).values
        best = torch.where(best == 1 << 30, torch.full_like(best, -1), best)
        s["idx"][a:b, :, :best.shape[-1]] = best.int()


# ---------------------------------------------------------------------------
# one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_plain(s):
    {"append": _append_plain, "attend": _attend_plain, "select": _select_plain, "blocks": _attend_plain}[s["op"]](s)
    return _outputs(s)


def _outputs(s):
    return {n: s[n] for n in {"append": ("q_out", "k_cache", "v_cache", "means"), "attend": ("o", "lse"),
                              "select": ("idx",), "blocks": ("o", "lse")}[s["op"]]}


def _run_own(s):
    import sparse_attention_indexer_live_gb300 as dsa
    op, cfg = s["op"], s.get("cfg")
    if cfg is None:  # what a program makes once: the cache's description, frequencies, workspaces
        cfg = s["cfg"] = dsa.kv_cfg(pages=s["pages"], page_size=s["page"], kv_heads=s["kv_heads"], dtype=s["dt"])
        if op == "append":
            s["turns"] = dsa.rotary_turns(s["inv_freq"])
        else:
            n = (dsa.dsa_kv_attention_workspace(cfg, s["q"], s["tables"]) if op == "attend" else
                 dsa.dsa_kv_select_workspace(cfg, s["q"], s["tables"]) if op == "select" else
                 dsa.dsa_kv_block_attention_workspace(cfg, s["q"], s["idx"], s["tables"]))
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=CUDA)
    if op == "append":
        dsa.dsa_kv_append(cfg, s["q"], s["k"], s["v"], s["ends"], s["slots"], s["turns"], s["neighbours"], 1.0,
                          s["q_out"], s["k_cache"], s["v_cache"], s["means"])
    elif op == "attend":
        dsa.dsa_kv_attention(cfg, s["k_cache"], s["v_cache"], s["q"], s["first"], s["lens"], s["tables"], s["scale"],
                             s["workspace"], s["o"], s["lse"])
    elif op == "select":
        dsa.dsa_kv_select(cfg, s["means"], s["q"], s["first"], s["lens"], s["tables"], s["lead"], s["trail"],
                          s["workspace"], s["idx"])
    else:
        dsa.dsa_kv_block_attention(cfg, s["k_cache"], s["v_cache"], s["q"], s["idx"], s["first"], s["lens"],
                                   s["tables"], s["scale"], s["workspace"], s["o"], s["lse"])
    return _outputs(s)


def work(case):
    c = case
    lens, new = _shape(c)
    H, Hk, page, T = c["heads"], c["kv_heads"], c["page"], sum(new)
    row = 2 * DIM
    if c["op"] == "append":
        filled = sum(n // page - (n - f) // page for n, f in zip(lens, new))
        before = sum(min((n - f) % page, n - f) for n, f in zip(lens, new) if n // page > (n - f) // page)
        return {"bytes": row * (2 * T * (H + 2 * Hk) + (filled + before) * Hk) + 8 * T + 4 * c["rot"],
                "flops": 3 * c["rot"] * T * (H + Hk) + filled * page * Hk * DIM}
    pages = [-(-n // page) for n in lens]
    if c["op"] == "select":
        # pages that are scored: before the trailing pinned ones
        pairs = sum(max(0, (p // page) + 1 - c["trail"] - c["lead"]) for n, f in zip(lens, new) for p in range(n - f, n))
        return {"bytes": row * Hk * sum(pages) + row * T * H + 4 * T * Hk * c["select"] + 4 * sum(pages),
                "flops": 2.0 * DIM * Hk * pairs + T * H * DIM}
    io = T * H * (2 * row + 4)
    if c["op"] == "attend":
        pairs = sum(f * (n - f) + f * (f + 1) / 2 for n, f in zip(lens, new))
        return {"bytes": 2 * row * Hk * sum(lens) + io, "flops": 4.0 * DIM * H * pairs}
    pairs = seen = 0.0
    for n, f, p in zip(lens, new, pages):
        per = min(c["select"], p)
        pairs += f * min(per * page - page / 2, n - f / 2)
        # distinct pages: runs of 64 tokens share theirs but for 1 in 500 of all pages
        lists = -(-f // 64) * per + 0.002 * f * min(p, per / 0.002)
        seen += p * -math.expm1(-lists / p) if f > 1 else per
    return {"bytes": 2 * row * Hk * page * seen + io + 4 * T * Hk * c["select"], "flops": 4.0 * DIM * H * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _append_exact, "attend": _attend_exact, "select": _select_exact, "blocks": _attend_exact}[
        s["op"]](s)


def _append_exact(s):
    half = s["inv_freq"].numel()
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=CUDA), (s["ends"].double() - 1)[:, None] * s["inv_freq"])

    def rotated(x):
        y = x.double().clone()
        i = torch.arange(half, device=CUDA)
        re, im = (2 * i, 2 * i + 1) if s["neighbours"] else (i, i + half)
        z = torch.complex(y[..., re], y[..., im]) * turn[:, None]
        y[..., re], y[..., im] = z.real, z.imag
        return y

    page, Hk = s["page"], s["kv_heads"]
    k, v, means = s["k_cache"].double(), s["v_cache"].double(), s["means"].double()
    new = rotated(s["k"])
    held = s["k_cache"].clone()
    held.view(-1, Hk, DIM)[s["slots"].long()] = new.to(s["dt"])
    k.view(-1, Hk, DIM)[s["slots"].long()] = new
    v.view(-1, Hk, DIM)[s["slots"].long()] = s["v"].double()
    for slot in s["slots"].tolist():
        if (slot + 1) % page == 0:
            means[slot // page] = held[slot // page].double().sum(0) / page
    return {"q_out": rotated(s["q"]), "k_cache": k, "v_cache": v, "means": means}


def _attend_exact(s):
    T, H, Hk, page = s["q"].shape[0], s["heads"], s["kv_heads"], s["page"]
    group = H // Hk
    o = torch.zeros(T, H, DIM, dtype=torch.float64, device=CUDA)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=CUDA)
    for r, n in enumerate(s["lens_list"]):
        a, b = s["first_list"][r], s["first_list"][r + 1]
        slot = s["tables"][r].long().repeat_interleave(page)[:n] * page + torch.arange(n, device=CUDA) % page
        few = max(1, (1 << 25) // n)  # tokens at a time: 64-bit scores are large
        for h in range(Hk):
            k = s["k_cache"].view(-1, Hk, DIM)[slot, h].double()
            v = s["v_cache"].view(-1, Hk, DIM)[slot, h].double()
            for t0 in range(a, b, few):
                t = torch.arange(t0, min(b, t0 + few), device=CUDA)
                last = n - b + t  # a token's own position
                late = torch.arange(n, device=CUDA)[None, :] > last[:, None]
                if s["op"] == "blocks":
                    mine = (s["idx"][t, h][:, :, None] == torch.arange(-(-n // page), device=CUDA)).any(1)
                    late = late | ~mine[:, torch.arange(n, device=CUDA) // page]
                for g in range(h * group, (h + 1) * group):
                    x = (s["q"][t, g].double() @ k.T * s["scale"]).masked_fill(late, -math.inf)
                    z = torch.logsumexp(x, -1)
                    lse[t, g] = z
                    o[t, g] = torch.exp(x - z[:, None]).nan_to_num(0.0) @ v
    return {"o": o, "lse": lse}


def _select_exact(s):
    page, Hk, n_out = s["page"], s["kv_heads"], s["idx"].shape[2]
    group = s["heads"] // Hk
    idx = torch.full_like(s["idx"], -1)
    for r, (n, f) in enumerate(zip(s["lens_list"], s["new_list"])):
        t = torch.arange(s["first_list"][r], s["first_list"][r + 1], device=CUDA)
        here = (t - t[0] + n - f) // page
        for h in range(Hk):
            means = s["means"][s["tables"][r, :(n - 1) // page + 1].long(), h].double()
            score = sum(s["q"][t, g].double() @ means.T for g in range(h * group, (h + 1) * group))
            j = torch.arange(means.shape[0], device=CUDA).expand_as(score)
            free = (j >= s["lead"]) & (j <= here[:, None] - s["trail"])
            pinned = (j <= here[:, None]) & ~free
            room = n_out - pinned.sum(-1)
            order = torch.sort(score.masked_fill(~free, -math.inf), dim=-1, descending=True, stable=True).indices
            rank = torch.empty_like(order).scatter_(1, order, j.contiguous())
            keep = pinned | (free & (rank < room[:, None]))
            place = torch.cumsum(keep, -1) - 1
            at = keep.nonzero(as_tuple=True)
            idx[t[at[0]], h, place[at]] = at[1].int()
    return {"idx": idx}
