"""Cases of the token-by-token operators: the recurrent KDA step on a cache of states, and latent
attention over a paged cache of latents (append, query absorption, attention, output expansion).

Sizes are those of the repository's hybrid layer group (16 or 32 heads of 128, 64 rotary dimensions,
a latent of 512) and of its odd test shapes.  Each case is one operator's call on one batch of
sequences; the rows of a batch are ragged wherever ``rows_max`` is above one.
"""
import math

import torch

own = False

LAT, ROPE, HEAD = 512, 64, 128          # latent, rotary and per-head widths of the layer group
WIDTH = LAT + ROPE                      # one cached token
SCALE = 1.0 / math.sqrt(HEAD + ROPE)
BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one rollout being sampled: the latency of a single token through a KDA layer's state
        {"name": "kda_step_one", "op": "kda_step", "seqs": 1, "heads": 16, "dim": 128, "rows_max": 1, "fork": False, "dtype": "bf16"},
        # drafted tokens and rollouts that branch from shared states, fp32 layer, odd sizes
        {"name": "kda_step_fork_runs", "op": "kda_step", "seqs": 37, "heads": 5, "dim": 64, "rows_max": 6, "fork": True, "dtype": "f32"},
        # a full sampling batch of the 32-head layer: bound by reading and writing the states
        {"name": "kda_step_batch", "op": "kda_step", "seqs": 512, "heads": 32, "dim": 128, "rows_max": 1, "fork": False, "dtype": "bf16"},
        # one token each for a sampling batch
        {"name": "append_tokens", "op": "append", "seqs": 96, "heads": 16, "rows_max": 1, "kv_max": 8192, "page": 64, "dtype": "bf16"},
        # tool answers read into the cache: long ragged runs from the fp32 projections, small pages
        {"name": "append_runs", "op": "append", "seqs": 24, "heads": 16, "rows_max": 1021, "kv_max": 4096, "page": 16, "dtype": "f32"},
        # queries of one token, and of a long ragged run of tokens
        {"name": "absorb_one", "op": "absorb", "seqs": 1, "heads": 16, "rows_max": 1, "kv_max": 40000},
        {"name": "absorb_runs", "op": "absorb", "seqs": 11, "heads": 16, "rows_max": 720, "kv_max": 40000},
        # attention outputs of a sampling batch, and of long runs of the 32-head layer
        {"name": "expand_tokens", "op": "expand", "rows": 96, "heads": 16},
        {"name": "expand_runs", "op": "expand", "rows": 2047, "heads": 32},
        # one rollout with a long context: latency, the context split over the whole GPU
        {"name": "attn_one", "op": "attn", "seqs": 1, "heads": 16, "rows_max": 1, "kv_max": 6000, "page": 64},
        # drafted tokens: several queries a sequence, causal among themselves, odd head count
        {"name": "attn_drafts", "op": "attn", "seqs": 19, "heads": 5, "rows_max": 7, "kv_max": 3001, "page": 16},
        # a sampling batch of agentic contexts, ragged from empty to 32768 tokens
        {"name": "attn_batch", "op": "attn", "seqs": 64, "heads": 16, "rows_max": 1, "kv_max": 32768, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kda_step", "append", "absorb", "expand", "attn"])
    if op == "kda_step":
        dim = rng.choice([32, 64, 128])
        heads = _log(rng, 1, 32)
        runs = rng.random() < 0.4
        return {"op": op, "seqs": _log(rng, 1, 200 if runs else 512), "heads": heads, "dim": dim, "rows_max": rng.randint(2, 6) if runs else 1,
                "fork": rng.random() < 0.4, "dtype": rng.choice(["bf16", "f32"])}
    if op == "append":
        rows_max = _log(rng, 2, 1024) if rng.random() < 0.5 else 1
        return {"op": op, "seqs": _log(rng, 1, 24 if rows_max > 1 else 256), "heads": rng.choice([1, 5, 16, 32]), "rows_max": rows_max,
                "kv_max": _log(rng, 1100, 4096), "page": rng.choice([16, 32, 64, 128]), "dtype": rng.choice(["bf16", "f32"])}
    if op == "absorb":
        rows_max = _log(rng, 2, 720) if rng.random() < 0.5 else 1
        return {"op": op, "seqs": _log(rng, 1, 11 if rows_max > 1 else 500), "heads": rng.choice([1, 3, 5, 8, 16]), "rows_max": rows_max,
                "kv_max": _log(rng, 1000, 200000)}
    if op == "expand":
        return {"op": op, "rows": _log(rng, 1, 2047), "heads": _log(rng, 1, 32)}
    rows_max = rng.randint(2, 8) if rng.random() < 0.5 else 1
    kv_max = _log(rng, 16, 32768)
    heads = rng.choice([1, 3, 5, 8, 16, 24, 32])
    most = (64 * 32768 * 16) // (kv_max * rows_max * heads)
    return {"op": op, "seqs": max(1, min(_log(rng, 1, 96), 64 * 32768 // kv_max, most)), "heads": heads, "rows_max": rows_max, "kv_max": kv_max,
            "page": rng.choice([16, 32, 64, 128])}


# ------------------------------------------------------------------------------------ inputs
def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _spread(n, top):
    """n whole numbers spread evenly over 0 .. top, top itself first."""
    return [top] + [int(i * 0.6180339887498949 % 1 * (top + 1)) for i in range(1, n)]


def _ragged(gen, n, top):
    return torch.tensor(_spread(n, top), device="cuda")[torch.randperm(n, generator=gen, device="cuda")]


def _runs(gen, seqs, rows_max):
    """row_start of a ragged batch: the longest run has rows_max new rows, some have none."""
    m = _ragged(gen, seqs, rows_max)
    return torch.cat([m.new_zeros(1), m.cumsum(0)]).to(torch.int32)


def _pages(gen, seqs, kv_max, page):
    """Every sequence's pages, scattered over the cache."""
    per = -(-kv_max // page)
    perm = torch.randperm(seqs * per + 1, generator=gen, device="cuda")[: seqs * per]
    return perm.view(seqs, per).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    op = case["op"]
    if op == "expand":
        st["o"] = _randn(gen, case["rows"], case["heads"], LAT) * 0.2
        st["w_b"] = _randn(gen, 2 * case["heads"] * HEAD, LAT, dtype=torch.float32).mul_(0.02).to(torch.bfloat16)
        return st
    seqs, H, rows_max = case["seqs"], case["heads"], case["rows_max"]
    st["row_start"] = _runs(gen, seqs, rows_max) if rows_max > 1 else None
    n = int(st["row_start"][-1]) if rows_max > 1 else seqs
    st["n_rows"] = n
    if op == "kda_step":
        d, dt = case["dim"], DTYPES[case["dtype"]]
        k = _randn(gen, n, H, d, dtype=torch.float32)
        st["q"], st["k"], st["v"] = _randn(gen, n, H, d, dtype=dt), (k / k.norm(dim=-1, keepdim=True)).to(dt), _randn(gen, n, H, d, dtype=dt)
        st["g"] = (-0.1 * torch.nn.functional.softplus(_randn(gen, n, H, d, dtype=torch.float32))).to(dt)
        st["beta"] = torch.sigmoid(_randn(gen, n, H, dtype=torch.float32)).to(dt)
        slots = seqs + (seqs if case["fork"] else 1)
        st["state"] = _randn(gen, slots, H, d, d, dtype=torch.float32).mul_(0.3)
        perm = torch.randperm(slots, generator=gen, device="cuda")
        if case["fork"]:  # branches read shared states and keep their own
            st["src"] = perm[torch.randint(0, max(1, seqs // 3), (seqs,), generator=gen, device="cuda")].to(torch.int32)
            st["dst"] = perm[seqs:].to(torch.int32)
        else:
            st["src"], st["dst"] = perm[:seqs].to(torch.int32), None
        return st
    kv = _ragged(gen, seqs, case["kv_max"])
    m = torch.diff(st["row_start"]) if rows_max > 1 else torch.ones_like(kv)
    kv = torch.maximum(kv, m)
    if op == "attn" and seqs > 2:
        kv[seqs // 2] = 0  # a padding entry of the batch
    st["kv_len"] = kv.to(torch.int32)
    if op == "absorb":
        st["q"] = _randn(gen, n, H * (HEAD + ROPE) + WIDTH)[:, : H * (HEAD + ROPE)].unflatten(1, (H, HEAD + ROPE))
        st["w_b"] = _randn(gen, 2 * H * HEAD, LAT, dtype=torch.float32).mul_(0.02).to(torch.bfloat16)
        return st
    most = max(case["kv_max"], rows_max)
    st["block_table"] = _pages(gen, seqs, most, case["page"])
    n_pages = seqs * (-(-most // case["page"])) + 1
    st["cache"] = torch.randn(n_pages, case["page"], WIDTH, generator=gen, device="cuda", dtype=torch.bfloat16)
    if op == "append":
        proj = _randn(gen, n, H * (HEAD + ROPE) + WIDTH, dtype=DTYPES[case["dtype"]])  # [q | c | kr] of the projection
        st["c"], st["kr"] = proj[:, -WIDTH:-ROPE], proj[:, -ROPE:]
        return st
    st["qa"] = _randn(gen, n, H, WIDTH)
    return st


# ------------------------------------------------------------------------------------ plain forms
def _rows(st):
    """(sequence, position) of every new row: row i of a run of m ends the kv_len cached tokens."""
    if st["row_start"] is None:
        b = torch.arange(st["n_rows"], device="cuda")
        return b, st["kv_len"].long() - 1
    start = st["row_start"].long()
    t = torch.arange(st["n_rows"], device="cuda")
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return b, st["kv_len"].long()[b] - start[b + 1] + t


def _padded(st):
    """[seqs, rows_max] row numbers of a ragged batch, n_rows where a sequence has no such row."""
    start = (st["row_start"] if st["row_start"] is not None else torch.arange(st["n_rows"] + 1, device="cuda")).long()
    i = torch.arange(st["rows_max"], device="cuda")
    t = start[:-1, None] + i
    return torch.where(t < start[1:, None], t, st["n_rows"])


def _rotate(x, pos):
    """Half-split rotation of the last dimension at `pos`, which broadcasts over x's other dimensions."""
    half = x.shape[-1] // 2
    inv = BASE ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / x.shape[-1])
    angle = pos.double()[..., None] * inv
    cs, sn = angle.cos().float(), angle.sin().float()
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cs - b * sn, a * sn + b * cs], -1)


def _plain_kda_step(st):
    src = st["src"].long()
    dst = st["dst"].long() if st["dst"] is not None else src
    S = st["state"][src]
    if st["row_start"] is None:
        q, k, v, g, beta = (st[x].float() for x in ("q", "k", "v", "g", "beta"))
        S = S * torch.exp(g)[..., None]
        u = torch.einsum("bhij,bhi->bhj", S, k)
        S = S + k[..., None] * (beta[..., None] * (v - u))[..., None, :]
        o = torch.einsum("bhij,bhi->bhj", S, q)
    else:
        at = _padded(st)
        q, k, v, g, beta = (torch.cat([st[x].float(), torch.zeros_like(st[x][:1], dtype=torch.float32)])[at] for x in ("q", "k", "v", "g", "beta"))
        o = q.new_zeros(st["n_rows"] + 1, *st["q"].shape[1:])
        for t in range(st["rows_max"]):  # the recurrence; rows past a run's end have g = 0 and beta = 0 and change nothing
            S = S * torch.exp(g[:, t])[..., None]
            u = torch.einsum("bhij,bhi->bhj", S, k[:, t])
            S = S + k[:, t][..., None] * (beta[:, t][..., None] * (v[:, t] - u))[..., None, :]
            o[at[:, t]] = torch.einsum("bhij,bhi->bhj", S, q[:, t])
        o = o[: st["n_rows"]]
    st["state"][dst] = S
    return o.to(st["q"].dtype), st["state"]


def _plain_append(st):
    b, pos = _rows(st)
    page = st["page"]
    x = torch.cat([st["c"].float(), _rotate(st["kr"].float(), pos)], -1)
    st["cache"][st["block_table"][b, pos // page].long(), pos % page] = x.to(st["cache"].dtype)
    return st["cache"]


def _plain_absorb(st):
    _, pos = _rows(st)
    q = st["q"].float()
    w = st["w_b"][: st["heads"] * HEAD].float().view(st["heads"], HEAD, LAT)
    lat = torch.einsum("thi,hil->thl", q[..., :HEAD], w)
    return torch.cat([lat, _rotate(q[..., HEAD:], pos[:, None])], -1).to(st["q"].dtype)


def _plain_expand(st):
    w = st["w_b"][st["heads"] * HEAD:].float().view(st["heads"], HEAD, LAT)
    return torch.einsum("thl,hil->thi", st["o"].float(), w).to(st["o"].dtype)


def _plain_attn(st):
    n, H = st["n_rows"], st["heads"]
    at = _padded(st)  # [B, R]
    m = (at < n).sum(1)
    B, R = at.shape
    keys = st["cache"][st["block_table"].long()].view(B, -1, WIDTH).float()
    q = torch.cat([st["qa"], torch.zeros_like(st["qa"][:1])])[at].float()
    s = torch.einsum("brhe,ble->brhl", q, keys) * SCALE
    pos = st["kv_len"].long()[:, None] - m[:, None] + torch.arange(R, device="cuda")
    s = torch.where(torch.arange(keys.shape[1], device="cuda") <= pos[:, :, None, None], s, -math.inf)
    mx = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(mx == -math.inf, 0.0, mx))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("brhl,ble->brhe", p, keys[..., :LAT]) / torch.where(total == 0, 1.0, total)
    lse = (mx + torch.log(total)).squeeze(-1)
    out, l = o.new_zeros(n + 1, H, LAT), o.new_zeros(n + 1, H)
    out[at], l[at] = o, lse
    return out[:n].to(st["qa"].dtype), l[:n]


def run(st):
    op = st["op"]
    if not own:
        return {"kda_step": _plain_kda_step, "append": _plain_append, "absorb": _plain_absorb, "expand": _plain_expand, "attn": _plain_attn}[op](st)
    import tree_packed_chunkwise_b200 as tpc
    if op == "kda_step":
        o = tpc.tpc_kda_step(st["state"], st["src"], st["q"], st["k"], st["v"], st["g"], st["beta"], dst=st["dst"], row_start=st["row_start"])
        return o, st["state"]
    if op == "append":
        tpc.tpc_latent_append(st["cache"], st["block_table"], st["kv_len"], st["c"], st["kr"], row_start=st["row_start"])
        return st["cache"]
    if op == "absorb":
        return tpc.tpc_latent_absorb(st["q"], st["w_b"], st["kv_len"], row_start=st["row_start"])
    if op == "expand":
        return tpc.tpc_latent_expand(st["o"], st["w_b"])
    return tpc.tpc_latent_attn(st["qa"], st["cache"], st["block_table"], st["kv_len"], SCALE, row_start=st["row_start"])


# ------------------------------------------------------------------------------------ 64-bit definition
def _exact_runs(st):
    """[(sequence, first row, rows)] on the host."""
    if st["row_start"] is None:
        return [(b, b, 1) for b in range(st["n_rows"])]
    s = st["row_start"].tolist()
    return [(b, s[b], s[b + 1] - s[b]) for b in range(len(s) - 1)]


def _exact_rotation(x, first, m):
    """x [m, ..., ROPE] as complex pairs (i, i + 32), row r turned by (first + r) * BASE^(-2i/ROPE)."""
    half = ROPE // 2
    inv = torch.tensor([BASE ** (-2.0 * i / ROPE) for i in range(half)], dtype=torch.float64, device="cuda")
    turn = torch.arange(first, first + m, device="cuda").double()[:, None] * inv
    turn = turn.view(m, *[1] * (x.dim() - 2), half)
    z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * torch.polar(torch.ones_like(turn), turn)
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op, H = case["op"], case["heads"]
    if op == "expand":
        w, o = st["w_b"].double(), st["o"].double()
        return torch.stack([o[:, h] @ w[(H + h) * HEAD:(H + h + 1) * HEAD].T for h in range(H)], 1)
    runs = _exact_runs(st)
    if op == "kda_step":
        old, new = st["state"], st["state"].double()
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        src = st["src"].tolist()
        dst = st["dst"].tolist() if st["dst"] is not None else src
        eye = torch.eye(case["dim"], dtype=torch.float64, device="cuda")
        for b, first, m in runs:
            S = old[src[b]].double()
            for t in range(first, first + m):
                q, k, v, a, beta = st["q"][t].double(), st["k"][t].double(), st["v"][t].double(), st["g"][t].double().exp(), st["beta"][t].double()
                # S <- (I - beta k k^T) Diag(a) S + beta k v^T,  o = S^T q
                step = eye - beta[:, None, None] * k[:, :, None] * k[:, None, :]
                S = step @ (a[:, :, None] * S) + beta[:, None, None] * k[:, :, None] * v[:, None, :]
                o[t] = (S.transpose(1, 2) @ q[:, :, None]).squeeze(2)
            new[dst[b]] = S
        return o, new
    kv = st["kv_len"].tolist()
    if op == "absorb":
        w, q = st["w_b"].double(), st["q"].double()
        lat = torch.stack([q[:, h, :HEAD] @ w[h * HEAD:(h + 1) * HEAD] for h in range(H)], 1)
        rot = torch.cat([_exact_rotation(q[first:first + m, :, HEAD:], kv[b] - m, m) for b, first, m in runs])
        return torch.cat([lat, rot], -1)
    if op == "append":
        cache, c, kr = st["cache"].double(), st["c"].double(), st["kr"].double()
        for b, first, m in runs:
            p = torch.arange(kv[b] - m, kv[b], device="cuda")
            at = st["block_table"][b].long()[p // case["page"]]
            cache[at, p % case["page"]] = torch.cat([c[first:first + m], _exact_rotation(kr[first:first + m], kv[b] - m, m)], -1)
        return cache
    o = torch.zeros(st["n_rows"], H, LAT, dtype=torch.float64, device="cuda")
    lse = torch.full((st["n_rows"], H), -math.inf, dtype=torch.float64, device="cuda")
    for b, first, m in runs:
        if m == 0 or kv[b] == 0:
            continue
        mem = st["cache"][st["block_table"][b].long()].reshape(-1, WIDTH)[: kv[b]].double()
        for i in range(m):
            seen = mem[: kv[b] - m + 1 + i]
            z = (st["qa"][first + i].double() @ seen.T) * SCALE
            lse[first + i] = torch.logsumexp(z, -1)
            o[first + i] = torch.softmax(z, -1) @ seen[:, :LAT]
    return o, lse


# ------------------------------------------------------------------------------------ work
def work(case):
    op, H = case["op"], case["heads"]
    if op == "expand":
        n = case["rows"]
        return {"bytes": 2 * (n * H * (LAT + HEAD) + H * HEAD * LAT), "flops": 2 * n * H * LAT * HEAD}
    n = case["seqs"] if case["rows_max"] == 1 else sum(_spread(case["seqs"], case["rows_max"]))
    if op == "kda_step":
        d, e = case["dim"], 2 if case["dtype"] == "bf16" else 4
        read = max(1, case["seqs"] // 3) if case["fork"] else case["seqs"]
        return {"bytes": 4 * d * d * H * (read + case["seqs"]) + n * H * (5 * d + 1) * e, "flops": 7 * n * H * d * d}
    if op == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * WIDTH * (e + 2), "flops": n * ROPE * 3}
    if op == "absorb":
        return {"bytes": 2 * (n * H * (HEAD + ROPE + WIDTH) + H * HEAD * LAT), "flops": 2 * n * H * HEAD * LAT}
    tokens = sum(_spread(case["seqs"], case["kv_max"]))
    return {"bytes": 2 * (tokens * WIDTH + n * H * (WIDTH + LAT)) + 4 * n * H, "flops": 2 * tokens * n / case["seqs"] * H * (WIDTH + LAT)}
