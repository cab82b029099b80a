"""The serving operators around the paged KV cache, as they are timed and compared:

plan    block tables and slot maps of a step, from the requests' lengths on the GPU
append  a step's key and value rows written into the paged pools through the slot map
attend  causal attention of packed queries over the paged cache (whole prompts, chunks, single tokens)

`run` computes them in plain torch, or, where `own` is true, with the library's entry points.
"""
import math

import torch

own = False

SCORES = 1 << 28      # score entries the plain attention holds at a time
SPARE_PAGES = 5       # pages of a pool that no request has


# ------------------------------------------------------------------ cases

def _text(xs):
    return ",".join(str(int(x)) for x in xs)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _case(op, lens, new, **over):
    """lens: tokens of each request once this step's are in; new: the step's own tokens of each."""
    c = {"op": op, "dtype": "bf16", "hq": 32, "hkv": 8, "d": 128, "page": 16, "fused": True, "pad": 0,
         "lens": _text(lens), "new": _text(new)}
    c.update(over)
    return c


def listed():
    # lengths log-uniform in [4096, 262144]: the ragged batch this library is benchmarked on
    ragged = [116503, 117936, 34924, 13445, 5125, 20174, 22394, 4944]
    # a serving batch between a fresh request and a full context
    batch = [1 + (131071 * i * i) // 3969 for i in range(64)]
    return [
        # one decode step of a running batch: every request grows by a token
        _case("plan", batch, [1] * 64, name="plan_step"),
        # a batch of prompts admitted at once, every token new; the slot map is padded to a fixed capacity
        _case("plan", ragged, ragged, pad=2233, name="plan_prompts"),
        # one decode step's rows of 16 requests
        _case("append", [32768] * 16, [1] * 16, name="append_step"),
        # a whole prompt's rows, from the fused projection that made them
        _case("append", [131072], [131072], name="append_prompt"),
        # short prompts of a chat batch: latency, odd lengths, one tile or less each
        _case("attend", [1, 17, 200, 129, 64, 333, 5, 90], [1, 17, 200, 129, 64, 333, 5, 90], name="attend_short"),
        # one segment of the index as a prompt
        _case("attend", [8192], [8192], name="attend_segment"),
        # the longest prompt here
        _case("attend", [32768], [32768], name="attend_prompt"),
        # the next chunk of three prompts whose earlier chunks are in the cache
        _case("attend", [131072, 40001, 5000], [512, 1024, 77], name="attend_chunk"),
        # a decode step without an index: one token for each of 16 requests
        _case("attend", [32768] * 16, [1] * 16, name="attend_step"),
        # one request decoding over a long context
        _case("attend", [131072], [1], name="attend_single"),
        # a head for each key head, small heads, larger pages, an odd length
        _case("attend", [4111, 2500], [4111, 2500], hq=8, hkv=8, d=64, page=64, fused=False, name="attend_d64"),
        # the fp32 workload's shape
        _case("attend", [4096], [4096], dtype="f32", hq=1, hkv=1, d=64, fused=False, name="attend_f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend"])
    page = rng.choice([1, 8, 16, 16, 32, 64, 256])
    hkv = rng.choice([1, 2, 4, 8])
    c = {"page": page, "hkv": hkv, "hq": hkv * rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128]),
         "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]), "fused": rng.random() < 0.5}
    if op == "plan":
        n = _log(rng, 1, 256)
        lens = [_log(rng, 1, 131072) for _ in range(n)]
        if rng.random() < 0.5:      # single tokens, some requests idle
            new = [rng.choice([0, 1, 1, 1]) for _ in lens]
        else:                       # chunks of any length up to the whole
            new = [_log(rng, 1, x) for x in lens]
            over = sum(new) / 400000
            new = [max(1, int(x / over)) for x in new] if over > 1 else new
        return _case(op, lens, new, pad=rng.choice([0, rng.randrange(1, 512)]), **c)
    if op == "append":
        new = [_log(rng, 1, 8192) for _ in range(_log(rng, 1, 12))]
        return _case(op, [x + rng.randrange(0, 2000) for x in new], new, pad=rng.choice([0, rng.randrange(1, 64)]), **c)
    kind = rng.choice(["prompt", "chunk", "step"])
    most = 3000 if c["dtype"] == "f32" else 12000
    if kind == "prompt":
        new = [_log(rng, 1, most) for _ in range(_log(rng, 1, 6))]
        lens = new
    elif kind == "chunk":
        new = [_log(rng, 1, most // 8) for _ in range(_log(rng, 1, 4))]
        lens = [x + _log(rng, 1, 4 * most) for x in new]
    else:
        lens = [_log(rng, 1, 10 * most) for _ in range(_log(rng, 1, 16))]
        new = [1] * len(lens)
    return _case(op, lens, new, **c)


# ------------------------------------------------------------------ inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _mixture(gen, centers, scale, rows, per_head):
    """[rows][heads][d] rows near the centres of their key head, per-channel scaled."""
    h, n, d = centers.shape
    ids = torch.randint(0, n, (rows, h, per_head), generator=gen, device="cuda")
    x = centers[torch.arange(h, device="cuda")[None, :, None], ids]
    x = x.add_(torch.randn(x.shape, generator=gen, device="cuda"), alpha=0.3)
    return x.mul_(scale).reshape(rows, h * per_head, d)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens, new, page = _ints(case["lens"]), _ints(case["new"]), case["page"]
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], _dtype(case)
    batch, total = len(lens), sum(new)
    have = [a - b for a, b in zip(lens, new)]
    first = [-(-x // page) for x in have]        # pages in use before the step
    last = [-(-x // page) for x in lens]         # and after it
    used, n_pages = sum(last), sum(last) + SPARE_PAGES
    max_pages = max(max(last), 1)
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(max_pages, device="cuda")
    lasts = torch.tensor(last, device="cuda")
    starts = torch.cumsum(lasts, 0) - lasts
    at = (starts[:, None] + col).clamp(max=n_pages - 1)
    table = torch.where(col < lasts[:, None], order[at], -1).to(torch.int32)
    int32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"op": case["op"], "page": page, "n_pages": n_pages, "lens": lens, "new": new}
    if case["op"] == "plan":
        firsts = torch.tensor(first, device="cuda")
        free = torch.cat([table[(col >= firsts[:, None]) & (col < lasts[:, None])], order[used:]])
        free = free[torch.randperm(free.numel(), generator=gen, device="cuda")]
        table = torch.where(col < firsts[:, None], table, -1)
        s.update(table=table, free=free, n_free=int32([free.numel()]), seq_lens=int32(have), new_lens=int32(new),
                 capacity=total + case["pad"], work=torch.zeros(1024, dtype=torch.uint8, device="cuda"))
        return s
    centers = torch.randn(hkv, 256, d, generator=gen, device="cuda")
    scale = torch.exp(0.5 * torch.randn(hkv, 1, d, generator=gen, device="cuda"))
    q_rows = hq * d if case["fused"] else 0      # a fused projection's row: q, then k, then v
    if case["op"] == "append":
        tokens = total + case["pad"]
        rows = torch.empty(tokens, q_rows + 2 * hkv * d, dtype=dt, device="cuda")
        rows[:, :q_rows] = 0
        k = rows[:, q_rows:q_rows + hkv * d].view(tokens, hkv, d)
        v = rows[:, q_rows + hkv * d:].view(tokens, hkv, d)
        k.copy_(_mixture(gen, centers, scale, tokens, 1))
        v.copy_(torch.randn(tokens, hkv, d, generator=gen, device="cuda"))
        req = torch.repeat_interleave(torch.arange(batch, device="cuda"), torch.tensor(new, device="cuda"))
        begin = torch.tensor(new, device="cuda").cumsum(0) - torch.tensor(new, device="cuda")
        pos = torch.arange(total, device="cuda") - begin[req] + torch.tensor(have, device="cuda")[req]
        slots = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
        slots[:total] = table[req, pos // page] * page + (pos % page).to(torch.int32)
        pools = torch.randn(2, n_pages, hkv, page, d, generator=gen, device="cuda").to(dt)
        s.update(k=k, v=v, slots=slots, k_pool=pools[0], v_pool=pools[1],
                 work=torch.zeros(1024, dtype=torch.uint8, device="cuda"))
        return s
    k_pool = torch.empty(n_pages, hkv, page, d, dtype=dt, device="cuda")
    step = max(1, (1 << 22) // (hkv * page * d))
    for i in range(0, n_pages, step):            # the pool's rows, a few pages at a time
        n = min(step, n_pages - i)
        k_pool[i:i + n] = _mixture(gen, centers, scale, n * page, 1).view(n, page, hkv, d).transpose(1, 2)
    v_pool = torch.empty_like(k_pool)
    for i in range(0, n_pages, step):
        v_pool[i:i + step] = torch.randn(v_pool[i:i + step].shape, generator=gen, device="cuda")
    rows = torch.zeros(total, hq * d + (2 * hkv * d if case["fused"] else 0), dtype=dt, device="cuda")
    q = rows[:, :hq * d].view(total, hq, d)
    q.copy_(_mixture(gen, centers, scale, total, hq // hkv))
    s.update(q=q, k_pool=k_pool, v_pool=v_pool, table=table,
             out=torch.empty(total, hq, d, dtype=dt, device="cuda"),
             lse=torch.empty(total, hq, dtype=torch.float32, device="cuda"))
    return s


# ------------------------------------------------------------------ plain forms

def _plan(s):
    page, dev = s["page"], s["table"].device
    have, new = s["seq_lens"].long(), s["new_lens"].long()
    first, last = (have + page - 1) // page, (have + new + page - 1) // page
    need = last - first
    before = need.cumsum(0) - need                             # pages the requests before take
    col = torch.arange(s["table"].shape[1], device=dev)
    taken = before[:, None] + col - first[:, None]             # the stack is taken from its end
    at = (s["n_free"].long() - 1 - taken).clamp(0, s["free"].numel() - 1)
    fresh = (col >= first[:, None]) & (col < last[:, None])
    table = torch.where(fresh, s["free"][at], s["table"])
    s["table"].copy_(table)
    ends = new.cumsum(0)
    token = torch.arange(s["capacity"], device=dev)
    req = torch.searchsorted(ends, token, right=True)
    real = req < new.numel()
    req = req.clamp(max=new.numel() - 1)
    pos = token - (ends - new)[req] + have[req]
    row = (pos // page).clamp(0, s["table"].shape[1] - 1)
    slot = table[req, row].long() * page + pos % page
    none = torch.full_like(slot, -1)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    return {"slot_map": torch.where(real, slot, none).int(), "positions": torch.where(real, pos, none).int(),
            "starts": starts.int(), "seq_lens": (have + new).int(),
            "n_free": (s["n_free"] - need.sum()).int(), "block_table": s["table"]}


def _append(s):
    n = sum(s["new"])                                          # the rows behind are padding
    slot = s["slots"][:n].long()
    s["k_pool"][slot // s["page"], :, slot % s["page"]] = s["k"][:n]
    s["v_pool"][slot // s["page"], :, slot % s["page"]] = s["v"][:n]
    return [s["k_pool"], s["v_pool"]]


def _attend(s):
    q, page = s["q"], s["page"]
    total, hq, d = q.shape
    hkv = s["k_pool"].shape[1]
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    begin = 0
    for b, (T, n) in enumerate(zip(s["lens"], s["new"])):
        pages = s["table"][b, :-(-T // page)].long()
        k = s["k_pool"][pages].transpose(0, 1).reshape(hkv, 1, -1, d)[:, :, :T].float()
        v = s["v_pool"][pages].transpose(0, 1).reshape(hkv, 1, -1, d)[:, :, :T].float()
        some = max(1, SCORES // (hq * T))
        for i in range(0, n, some):
            m = min(some, n - i)
            high = T - n + i + m                               # keys some of these queries see
            rows = q[begin + i:begin + i + m].float().view(m, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            x = (rows @ k[:, :, :high].transpose(2, 3)) / math.sqrt(d)
            seen = torch.arange(high, device=q.device) <= torch.arange(high - m, high, device=q.device)[:, None]
            x = x.masked_fill_(~seen, -math.inf)
            top = x.amax(3, keepdim=True)
            x = x.sub_(top).exp_()
            mass = x.sum(3, keepdim=True)
            o = (x @ v[:, :, :high]) / mass
            out[begin + i:begin + i + m] = o.permute(2, 0, 1, 3).reshape(m, hq, d).to(out.dtype)
            lse[begin + i:begin + i + m] = (top + mass.log()).permute(2, 0, 1, 3).reshape(m, hq)
        begin += n
    return [out, lse]


# ------------------------------------------------------------------ the library's calls

def _own(s):
    """One call of the library; what a program keeps between its calls is made at the first."""
    import retrieval_sparse_attention_wave_b200 as W
    if s["op"] == "plan":
        if "kept" not in s:
            pages = W.PageTable(s["table"], s["seq_lens"], s["free"], s["n_free"], s["page"], s["n_pages"])
            s["kept"] = (pages, W.PagePlan.empty(pages, s["capacity"]))
        pages, into = s["kept"]
        p = W.plan_pages(pages, s["new_lens"], s["capacity"], out=into, ws=s["work"])
        return {"slot_map": p.slot_map, "positions": p.positions, "starts": p.starts, "seq_lens": p.seq_lens,
                "n_free": p.n_free, "block_table": pages.block_table}
    if s["op"] == "append":
        W.append_kv(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], ws=s["work"])
        return [s["k_pool"], s["v_pool"]]
    if "kept" not in s:
        kv = W.KVCache(s["k_pool"], s["v_pool"], s["table"], s["lens"])
        params = W.AttendParams(n_q_heads=s["q"].shape[1], q_lens=s["new"])
        s["kept"] = (kv, params, W.attend_workspace(kv, params))
    kv, params, ws = s["kept"]
    out, lse = W.attend(s["q"], kv, params, out=s["out"], lse=s["lse"], ws=ws)
    return [out, lse]


def run(state):
    if own:
        return _own(state)
    return {"plan": _plan, "append": _append, "attend": _attend}[state["op"]](state)


# ------------------------------------------------------------------ floors and 64-bit values

def work(case):
    lens, new, page = _ints(case["lens"]), _ints(case["new"]), case["page"]
    hq, hkv, d, e = case["hq"], case["hkv"], case["d"], 2 if case["dtype"] == "bf16" else 4
    total, batch = sum(new), len(lens)
    if case["op"] == "plan":
        have = [a - b for a, b in zip(lens, new)]
        need = sum(-(-a // page) + (-b // page) for a, b in zip(lens, have))
        open_pages = sum(1 for b, n in zip(have, new) if n and b % page)
        return {"bytes": 4 * (2 * batch + 1 + need + open_pages) + 4 * (need + 2 * (total + case["pad"]) + 2 * batch + 2),
                "flops": 0}
    if case["op"] == "append":
        return {"bytes": 4 * total * hkv * d * e + 4 * (total + case["pad"]), "flops": 0}
    pairs = sum(n * T - n * (n - 1) // 2 for T, n in zip(lens, new))
    tokens = sum(T for T, n in zip(lens, new) if n)
    return {"bytes": 2 * total * hq * d * e + 4 * total * hq + 2 * tokens * hkv * d * e + 4 * sum(-(-T // page) for T in lens),
            "flops": 4 * d * hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    page, lens, new = s["page"], s["lens"], s["new"]
    if case["op"] == "plan":
        table, free = s["table"].tolist(), s["free"].tolist()
        slots, positions, starts = [], [], [0]
        for row, T, n in zip(table, lens, new):
            for i in range(-(-(T - n) // page), -(-T // page)):
                row[i] = free.pop()
            where = torch.arange(T - n, T)
            positions.append(where)
            slots.append(torch.tensor(row)[where // page] * page + where % page)
            starts.append(starts[-1] + n)
        pad = [torch.full((case["pad"],), -1)]
        int32 = lambda x: x.to(torch.int32)  # noqa: E731
        return {"slot_map": int32(torch.cat(slots + pad)), "positions": int32(torch.cat(positions + pad)),
                "starts": int32(torch.tensor(starts)), "seq_lens": int32(torch.tensor(lens)),
                "n_free": int32(torch.tensor([len(free)])), "block_table": int32(torch.tensor(table))}
    if case["op"] == "append":
        got = []
        for x, pool in ((s["k"], s["k_pool"]), (s["v"], s["v_pool"])):
            by_slot = pool.double().transpose(1, 2).reshape(-1, *x.shape[1:])     # a row for each slot
            n = sum(new)
            by_slot.index_copy_(0, s["slots"][:n].long(), x[:n].double())
            got.append(by_slot.view(s["n_pages"], page, *x.shape[1:]).transpose(1, 2).contiguous())
        return got
    q = s["q"]
    total, hq, d = q.shape
    hkv = s["k_pool"].shape[1]
    group = hq // hkv
    out = torch.zeros(total, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(total, hq, dtype=torch.float64, device="cuda")
    ends = torch.tensor(new).cumsum(0).tolist()
    for b, T in enumerate(lens):
        where = torch.arange(T, device="cuda")
        page_of, row_of = s["table"][b].long()[where // page], where % page
        for h in range(hkv):
            keys, values = s["k_pool"][page_of, h, row_of].double(), s["v_pool"][page_of, h, row_of].double()
            for lo in range(0, new[b], 1024):
                hi = min(new[b], lo + 1024)
                token = torch.arange(ends[b] - new[b] + lo, ends[b] - new[b] + hi, device="cuda")
                position = torch.arange(T - new[b] + lo, T - new[b] + hi, device="cuda")
                limit = T - new[b] + hi
                score = torch.einsum("igd,kd->gik", q[token, h * group:(h + 1) * group].double(), keys[:limit]) * d ** -0.5
                score[:, where[None, :limit] > position[:, None]] = -math.inf
                total_mass = torch.logsumexp(score, 2)
                weight = torch.exp(score - total_mass[..., None])
                out[token, h * group:(h + 1) * group] = torch.einsum("gik,kd->igd", weight, values[:limit])
                lse[token, h * group:(h + 1) * group] = total_mass.T
    return [out, lse]
