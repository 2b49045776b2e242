"""Measured cases of the paged serving operators.

A serving step over a paged KV cache runs, in this order:
  tables   paged_build_tables: block tables, slot map, positions and prefix sums from the request lengths
  release  paged_release_pages: the pages of finished or shortened requests back onto the free list
  append   paged_norm_rope_append: per-head norms of q and k, rotation, rows written into the pages
  attn     gqa_paged_attn: attention of each request's new tokens over its pages, one token or a chunk

`run` computes an operator in plain torch where `own` is false, and calls the library where it is true.
"""
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a batch of 32 requests: every request brings one token, few need a page
        dict(name="tables decode b32", op="tables", batch=32, lo=1024, hi=4096, new=1, chunks=0, chunk=0, pad=0, S=16, ls=1),
        # admission of a large ragged batch: 16 prompts of up to 4K tokens among 240 decoding requests
        dict(name="tables mixed b256", op="tables", batch=256, lo=0, hi=8192, new=1, chunks=16, chunk=4096, pad=333, S=16, ls=2),
        # a few requests of a small batch end, or lose a rejected tail
        dict(name="release b32", op="release", batch=32, lo=1024, hi=4096, S=16, ls=3),
        # many long requests end at once (a batch job is cancelled), small pages
        dict(name="release b500 long", op="release", batch=500, lo=1, hi=32768, S=8, ls=4),
        # new rows of a decode step: 32 query heads, 8 KV heads of 64 channels
        dict(name="append decode b32", op="append", tokens=32, pad=0, Hq=32, Hkv=8, D=64, S=16, rope=64, inter=False, norm=True,
             dtype="f16", fused=True),
        # an odd-sized step with padding rows behind it and half of each head rotated in adjacent pairs
        dict(name="append ragged 1031", op="append", tokens=1031, pad=25, Hq=16, Hkv=2, D=128, S=32, rope=64, inter=True, norm=False,
             dtype="bf16", fused=False),
        # prefill of 8192 tokens: 32 query heads, 8 KV heads of 128 channels
        dict(name="append prefill 8192", op="append", tokens=8192, pad=0, Hq=32, Hkv=8, D=128, S=16, rope=128, inter=False, norm=True,
             dtype="bf16", fused=True),
        # a single request decoding at a 4K context: latency
        dict(name="attn decode b1 4k", op="attn", batch=1, lo=4096, hi=4096, new=1, chunks=0, chunk=0, Hq=32, Hkv=8, D=64, S=16,
             dtype="f16", ls=5),
        # decoding batch of 8 at up to 64K: the cache's bytes
        dict(name="attn decode b8 64k", op="attn", batch=8, lo=30001, hi=65536, new=1, chunks=0, chunk=0, Hq=32, Hkv=8, D=128, S=16,
             dtype="bf16", ls=6),
        # chunked prefill among decoding requests: two chunks of 500 tokens, 30 single tokens, contexts up to 4K
        dict(name="attn mixed b32", op="attn", batch=32, lo=600, hi=4096, new=1, chunks=2, chunk=500, Hq=32, Hkv=8, D=64, S=16,
             dtype="f16", ls=7),
        # drafted tokens: 5 new tokens of each of 16 requests scored at once, odd lengths
        dict(name="attn draft b16", op="attn", batch=16, lo=777, hi=9001, new=5, chunks=0, chunk=0, Hq=32, Hkv=8, D=128, S=32,
             dtype="bf16", ls=8),
        # a 1024-token chunk at the end of a 32K context, 32 heads of 128 channels: matrix products
        dict(name="attn chunk 1k of 32k", op="attn", batch=1, lo=32768, hi=32768, new=1, chunks=1, chunk=1024, Hq=32, Hkv=32, D=128,
             S=16, dtype="f16", ls=9),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["tables", "release", "append", "append", "attn", "attn", "attn", "attn"])
    S = rng.choice([8, 16, 32, 64, 128])
    ls = rng.randrange(1 << 30)
    if op == "tables":
        batch = _log(rng, 1, 512)
        hi = _log(rng, 1, 32768)
        chunks = rng.randint(0, min(batch, 16))
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, new=rng.randint(0, 8), chunks=chunks,
                    chunk=_log(rng, 1, 4096), pad=rng.choice([0, rng.randint(1, 500)]), S=S, ls=ls)
    if op == "release":
        hi = _log(rng, 1, 32768)
        return dict(op=op, batch=_log(rng, 1, 512), lo=rng.randint(0, hi), hi=hi, S=S, ls=ls)
    D = rng.choice([64, 128])
    G = rng.choice([1, 2, 4, 8])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32] if G == 1 else [1, 2, 3, 4, 8])
    dtype = rng.choice(["f16", "bf16"])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8192), pad=rng.choice([0, rng.randint(1, 60)]), Hq=G * Hkv, Hkv=Hkv, D=D, S=S,
                    rope=rng.choice([0, 32, D // 2, D, D]), inter=rng.random() < 0.4, norm=rng.random() < 0.7, dtype=dtype,
                    fused=rng.random() < 0.6)
    kind = rng.choice(["decode", "draft", "mixed", "chunk"])
    batch = 1 if kind == "chunk" and rng.random() < 0.4 else _log(rng, 1, 48)
    new = rng.randint(2, 9) if kind == "draft" else 1
    chunks = rng.randint(1, min(batch, 4)) if kind == "mixed" else batch if kind == "chunk" else 0
    chunk = _log(rng, 16, 1024) if chunks else 0
    # the padded plain form holds batch x rows x context scores, in 32 bits, and each context's rows: keep both under what
    # the largest listed case holds
    hi = _log(rng, max(1, new, chunk), 65536)
    most = max(chunk, new)
    hi = max(most, min(hi, (1 << 29) // (batch * most * G * Hkv), (1 << 28) // (batch * Hkv * D)))
    return dict(op=op, batch=batch, lo=rng.randint(most, hi), hi=hi, new=new, chunks=chunks, chunk=chunk, Hq=G * Hkv, Hkv=Hkv, D=D,
                S=S, dtype=dtype, ls=ls)


def lengths(case):
    """Per request: the tokens in the cache before the step, and the step's new tokens. For `attn`, lo and hi bound the
    context with the new tokens."""
    r = random.Random(case["ls"])
    whole = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    new = [case["new"]] * case["batch"]
    for i in r.sample(range(case["batch"]), case["chunks"]):
        new[i] = case["chunk"] if case["chunks"] == 1 or case["op"] == "attn" else r.randint(1, case["chunk"])
    if case["op"] == "attn":
        return [w - n for w, n in zip(whole, new)], new
    return whole, new


def kept(case):
    """Per request of a release: its tokens, and how many of them stay (none, all, or all but a tail)."""
    r = random.Random(case["ls"])
    whole = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    return whole, [r.choice([0, w, max(0, w - r.randint(1, 40))]) for w in whole]


def pages(n, S):
    return (n + S - 1) // S


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tables(counts, width, pool, gen):
    """A block table whose rows hold counts[b] distinct pages in shuffled order, and the pages that are left."""
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    n = torch.tensor(counts, device=DEV)
    used = torch.arange(width, device=DEV)[None, :] < n[:, None]
    table[used] = order[:sum(counts)]
    return table, order[sum(counts):]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, S = case["op"], case.get("S")
    s = dict(case)
    if op == "tables":
        cached, new = lengths(case)
        width = max(pages(c + n, S) for c, n in zip(cached, new)) + 1
        held = [pages(c, S) for c in cached]
        need = sum(pages(c + n, S) for c, n in zip(cached, new)) - sum(held)
        pool = sum(held) + need + 17
        s["table"], left = _tables(held, width, pool, gen)
        s["free"] = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
        s["free"][:left.numel()] = left
        s["count"] = _ints([left.numel()])
        s["cached"], s["new_len"] = _ints(cached), _ints(new)
        T = s["T"] = sum(new) + case["pad"] + (0 if sum(new) + case["pad"] else 1)
        s["out"] = dict(kv_len=_ints([0] * case["batch"]), cu_q=_ints([0] * (case["batch"] + 1)), positions=_ints([0] * T),
                        slots=_ints([0] * T), free_count_out=_ints([0]))
    elif op == "release":
        whole, keep = kept(case)
        held = [pages(w, S) for w in whole]
        pool = sum(held) + 11
        s["table"], left = _tables(held, max(held) + 1, pool, gen)
        s["free"] = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
        s["free"][:left.numel()] = left
        s["count"], s["kv_len"], s["keep"] = _ints([left.numel()]), _ints(whole), _ints(keep)
        s["count_out"] = _ints([0])
    elif op == "append":
        dt, T, Hq, Hkv, D, R = DTYPES[case["dtype"]], case["tokens"] + case["pad"], case["Hq"], case["Hkv"], case["D"], case["rope"]
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=gen, device=DEV).to(dt)  # the projection's output
        s["q"], s["k"], s["v"] = x.split([Hq, Hkv, Hkv], dim=1)
        if not case["fused"]:
            s["q"], s["k"], s["v"] = (t.contiguous() for t in (s["q"], s["k"], s["v"]))
        s["qw"] = s["kw"] = None
        if case["norm"]:
            s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(dt) for _ in range(2))
        s["cos_sin"] = None
        most = 65536
        if R:  # angles of far positions need more than 32 bits; the table is rounded once
            inv = 1.0 / 500000.0 ** (torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
            angle = torch.arange(most, dtype=torch.float64, device=DEV)[:, None] * inv
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        rows = pages(case["tokens"] * 3 // 2 + 1, S) * S
        s["positions"] = torch.randint(0, most, (T,), generator=gen, device=DEV).to(torch.int32)
        s["slots"] = torch.randperm(rows, generator=gen, device=DEV)[:T].to(torch.int32)
        s["slots"][case["tokens"]:] = -1
        pool = (rows // S, Hkv, S, D)
        s["kp"], s["vp"] = (torch.randn(pool, generator=gen, device=DEV).to(dt) for _ in range(2))
        s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
    else:
        dt, Hq, Hkv, D = DTYPES[case["dtype"]], case["Hq"], case["Hkv"], case["D"]
        cached, new = lengths(case)
        whole = [c + n for c, n in zip(cached, new)]
        held = [pages(w, S) for w in whole]
        pool = sum(held) + 3
        s["table"], _ = _tables(held, max(held), pool, gen)
        s["kp"], s["vp"] = (torch.randn(pool, Hkv, S, D, generator=gen, device=DEV, dtype=dt) for _ in range(2))
        s["q"] = torch.randn(sum(new), Hq, D, generator=gen, device=DEV, dtype=dt)
        s["kv_len"] = _ints(whole)
        s["cu_q"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
        s["max_q"], s["max_kv"] = max(new), max(whole)  # what a scheduler on the host knows
        s["scale"] = D ** -0.5
        s["out"] = torch.empty_like(s["q"])
        if own:  # the library's scratch, kept from step to step
            import gqa_head_folding_gb300 as g
            s["ws"] = g.alloc_paged_workspace(g.paged_dims_of(s["q"], s["kp"], s["table"]), DEV)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"tables": _plain_tables, "release": _plain_release, "append": _plain_append, "attn": _plain_attn}[s["op"]](s)


def _run_own(s):
    import gqa_head_folding_gb300 as g
    if s["op"] == "tables":
        kv_len, cu_q, positions, slots, count = g.paged_build_tables(s["cached"], s["new_len"], s["free"], s["count"], s["table"],
                                                                     s["T"], s["S"], **s["out"])
        return dict(table=s["table"], kv_len=kv_len, cu_q=cu_q, positions=positions, slots=slots, count=count)
    if s["op"] == "release":
        count = g.paged_release_pages(s["kv_len"], s["keep"], s["table"], s["free"], s["count"], s["S"], free_count_out=s["count_out"])
        return dict(free=s["free"], count=count)
    if s["op"] == "append":
        q = g.paged_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["kp"], s["vp"], q_weight=s["qw"],
                                     k_weight=s["kw"], eps=1e-6, cos_sin=s["cos_sin"], interleaved=s["inter"], q_out=s["q_out"])
        return dict(q=q, k_pages=s["kp"], v_pages=s["vp"])
    return dict(out=g.gqa_paged_attn(s["q"], s["kp"], s["vp"], s["table"], s["cu_q"], s["kv_len"], s["scale"], s["max_q"],
                                     out=s["out"], workspace=s["ws"]))


def _plain_tables(s):
    S, T, table, free = s["S"], s["T"], s["table"], s["free"]
    cached, new = s["cached"].long(), s["new_len"].long()
    held, want = (cached + S - 1) // S, (cached + new + S - 1) // S
    taken = torch.cumsum(want - held, 0)
    before = taken - (want - held)
    cu = torch.zeros(cached.numel() + 1, dtype=torch.int64, device=DEV)
    cu[1:] = torch.cumsum(new, 0)
    count = s["count"].long()
    # page p of request b, where it is new, is the next one off the end of the free list
    p = torch.arange(table.shape[1], device=DEV)[None, :]
    fresh = (p >= held[:, None]) & (p < want[:, None])
    at = (count - 1 - (before[:, None] + p - held[:, None])).clamp(0, free.numel() - 1)
    table.copy_(torch.where(fresh, free[at], table))
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=cached.numel() - 1)
    live = t < cu[-1]
    pos = torch.where(live, cached[b] + t - cu[b], 0)
    slot = torch.where(live, table[b, pos // S].long() * S + pos % S, -1)
    return dict(table=table, kv_len=(cached + new).int(), cu_q=cu.int(), positions=pos.int(), slots=slot.int(),
                count=(count - taken[-1]).int())


def _plain_release(s):
    S, table, free = s["S"], s["table"], s["free"]
    held, keep = (s["kv_len"].long() + S - 1) // S, (s["keep"].long() + S - 1) // S
    p = torch.arange(table.shape[1], device=DEV)[None, :]
    gone = (p >= keep[:, None]) & (p < held[:, None])
    at = torch.cumsum(gone.reshape(-1).long(), 0).reshape(gone.shape) - 1 + s["count"].long()
    place = torch.where(gone, at, free.numel())
    longer = torch.cat([free, free.new_zeros(1)])  # the last place takes what stays
    longer.scatter_(0, place.reshape(-1), table.reshape(-1))
    free.copy_(longer[:-1])
    return dict(free=free, count=(s["count"].long() + gone.sum()).int())


def _plain_append(s):
    def norm(x, w):
        x = x.float()
        return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()

    def rotate(x):
        if s["cos_sin"] is None:
            return x
        R = s["cos_sin"].shape[1]
        cos, sin = s["cos_sin"][s["positions"].long()][:, None].chunk(2, dim=-1)
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["inter"] else (x[..., :R // 2], x[..., R // 2:R])
        y = (a * cos - b * sin, b * cos + a * sin)
        y = torch.stack(y, dim=-1).flatten(-2) if s["inter"] else torch.cat(y, dim=-1)
        return torch.cat([y, x[..., R:]], dim=-1)

    live = s["slots"] >= 0
    S, n = s["kp"].shape[2], s["tokens"]
    q, k = rotate(norm(s["q"], s["qw"])), rotate(norm(s["k"], s["kw"]))
    s["q_out"].copy_(torch.where(live[:, None, None], q.to(s["q_out"].dtype), s["q_out"]))
    page, row = s["slots"][:n].long() // S, s["slots"][:n].long() % S  # the rows behind the tokens are padding
    s["kp"][page, :, row] = k[:n].to(s["kp"].dtype)
    s["vp"][page, :, row] = s["v"][:n]
    return dict(q=s["q_out"], k_pages=s["kp"], v_pages=s["vp"])


def _plain_attn(s):
    q, cu, kv_len = s["q"], s["cu_q"].long(), s["kv_len"].long()
    B, (T, Hq, D), Hkv, S, Q = kv_len.numel(), q.shape, s["kp"].shape[1], s["kp"].shape[2], s["max_q"]
    G, P = Hq // Hkv, (s["max_kv"] + S - 1) // S
    table = s["table"][:, :P].clamp(min=0).long()
    k, v = (c[table].transpose(1, 2).reshape(B, Hkv, P * S, D).float() for c in (s["kp"], s["vp"]))
    t = torch.arange(Q, device=DEV)[None, :]
    n = (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + t).clamp(max=T - 1)
    x = q[rows].float().reshape(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D)
    key = torch.arange(P * S, device=DEV)
    last = (kv_len[:, None] - n + t)[:, None, :, None].expand(B, 1, Q, G).reshape(B, 1, Q * G, 1)  # a row's own position
    v = torch.where((key[None, :] < kv_len[:, None])[:, None, :, None], v, 0.0)
    p = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(key > last, float("-inf"))
    p.sub_(p.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    o = o.reshape(B, Hkv, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B, Q, Hq, D)
    return dict(out=o[t < n].to(q.dtype))


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("tables", "release"):
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    k, v, q = s["kp"], s["vp"], s["q"].double()
    out, S = torch.zeros_like(q), case["S"]
    Hkv, G = case["Hkv"], case["Hq"] // case["Hkv"]
    for b, (c, n) in enumerate(zip(*lengths(case))):
        first, held = int(s["cu_q"][b]), s["table"][b, :pages(c + n, S)].long()
        seen = torch.ones(n, c + n, dtype=torch.bool, device=DEV).tril(c)
        for h in range(Hkv):
            kh, vh = (x[held, h].reshape(-1, case["D"])[:c + n].double() for x in (k, v))
            for g in range(G):
                a = (q[first:first + n, h * G + g] @ kh.T) * s["scale"]
                a = torch.softmax(torch.where(seen, a, -torch.inf), dim=1)
                out[first:first + n, h * G + g] = a @ vh
    return dict(out=out)


def _exact_append(s):
    D, R, n, S = s["D"], s["rope"], s["tokens"], s["S"]

    def head(x, w):
        y = x[:n].double()
        if w is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        if R:
            row = s["cos_sin"].double()[s["positions"][:n].long()]
            z = torch.complex(row[:, None, :R // 2], row[:, None, R // 2:])
            i = torch.arange(R // 2, device=DEV)
            i, j = (2 * i, 2 * i + 1) if s["inter"] else (i, i + R // 2)
            turned = torch.complex(y[..., i], y[..., j]) * z
            y[..., i], y[..., j] = turned.real, turned.imag
        return y

    q = s["q_out"].double()
    q[:n] = head(s["q"], s["qw"])
    kp, vp = s["kp"].double(), s["vp"].double()
    flat = s["slots"][:n].long()
    for pool, rows in ((kp, head(s["k"], s["kw"])), (vp, s["v"][:n].double())):
        pool.transpose(1, 2)[flat // S, flat % S] = rows
    return dict(q=q, k_pages=kp, v_pages=vp)


def work(case):
    op = case["op"]
    if op == "tables":
        cached, new = lengths(case)
        fresh = sum(pages(c + n, case["S"]) - pages(c, case["S"]) for c, n in zip(cached, new))
        tokens = sum(new) + case["pad"]
        # both lengths in; kv_len, cu_q out; a page in and out of the list; a position and a slot for each row
        return {"bytes": 4 * (4 * case["batch"] + 2 * fresh + 2 * tokens + 3), "flops": 2 * tokens}
    if op == "release":
        whole, keep = kept(case)
        gone = sum(pages(w, case["S"]) - pages(k, case["S"]) for w, k in zip(whole, keep))
        return {"bytes": 4 * (2 * case["batch"] + 2 * gone + 2), "flops": gone}
    if op == "append":
        n, D, heads = case["tokens"], case["D"], case["Hq"] + 2 * case["Hkv"]
        return {"bytes": n * (2 * heads * D * 2 + 4 * case["rope"] + 8), "flops": n * (case["Hq"] + case["Hkv"]) * D * 8}
    cached, new = lengths(case)
    keys = sum(c + n for c, n in zip(cached, new))
    seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
    return {"bytes": 4 * (sum(new) * case["Hq"] + keys * case["Hkv"]) * case["D"] + 4 * sum(pages(c + n, case["S"]) for c, n in zip(cached, new)),
            "flops": 4 * seen * case["Hq"] * case["D"]}
