"""The operators of a decode step that does not read all of every sequence's cache, as they are measured.

All four work on the paged bf16 cache: pools [n_pages, 128, 8, 128] of keys (rotated) and values, and a block table
[B, max_pages]. A page holds two blocks of 64 tokens.

- bounds: for each block and KV head the largest and the smallest key of each feature, in 8 bits with a power of two
  as scale: codes int8 [n_pages, 2, 8, 2, 128] (block of the page, KV head, upper and lower, feature) and scale
  [n_pages, 2, 8]. Recomputed for the blocks that new rows touch. With a = max |key| of the block's rows and head,
  scale = 2^e, e the least integer with a <= 127 * 2^e, kept within [-32, 16]; upper = ceil(max key / 2^e), lower =
  floor(min key / 2^e), kept within [-127, 127].
- select: a query in 8 bits the same way (rounded to nearest, ties to even), q = c * 2^f; the score of a block is the
  largest over the KV head's six query heads of 2^(e + f) * sum over features of max(c * upper, c * lower), a bound of
  the product with any key of the block. These are whole numbers times powers of two, exact in fp32 in any order. The
  first `sink` and the last `recent` blocks of a sequence are chosen, then those with the largest scores (the lower
  index first among equals), `budget` in all: their numbers in order, -1 behind the last.
- sparse: attention of one token per sequence over the rows of the blocks in its lists.
- shared: attention of one token per sequence where the sequences of a group have their first pages in common.
"""
import math
import random

import torch

own = False

HEADS, KV, GROUP, D, PAGE, BLOCK = 48, 8, 6, 128, 128, 64
MULT, CAP = 1.0 / math.sqrt(128.0), 30.0
LEAST, MOST = -32, 16  # exponents of the bounds' and the queries' scales
MAX_ROWS = 65536


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step of a serving batch: each sequence's last block takes one more row
        dict(name="bounds_step_b32", op="bounds", B=32, T=1, rows=16383, spread=True, valid_min=0),
        # a long prompt that was appended at once
        dict(name="bounds_prompt_8192", op="bounds", B=1, T=8192, rows=0, spread=False, valid_min=0),
        # one conversation: latency
        dict(name="select_b1_8192", op="select", B=1, rows=8192, spread=False, budget=32, sink=1, recent=2),
        # a serving batch at the longest context
        dict(name="select_b32_65536", op="select", B=32, rows=65536, spread=False, budget=64, sink=1, recent=4),
        # one conversation, 1024 of its 8192 rows: latency
        dict(name="sparse_b1_16", op="sparse", B=1, rows=8192, spread=False, budget=16, holes=0.0),
        # a serving batch, lengths from a few rows to 16384, 2048 rows read of each
        dict(name="sparse_b32_32", op="sparse", B=32, rows=16384, spread=True, budget=32, holes=0.0),
        # few very long contexts, 8192 rows read of each
        dict(name="sparse_b8_128", op="sparse", B=8, rows=65536, spread=False, budget=128, holes=0.0),
        # four answers to one short question: latency
        dict(name="shared_b4_512", op="shared", B=4, groups=1, even=True, prefix=512, own_rows=96, spread=True),
        # a system prompt of 8192 rows before short conversations
        dict(name="shared_b32_8192", op="shared", B=32, groups=1, even=True, prefix=8192, own_rows=300, spread=True),
        # four long documents with sixteen questions to each
        dict(name="shared_4x16_16384", op="shared", B=64, groups=4, even=True, prefix=16384, own_rows=200, spread=True),
        # a large batch whose own rows weigh as much as the prefix
        dict(name="shared_b128_4096", op="shared", B=128, groups=1, even=True, prefix=4096, own_rows=1024, spread=True),
        # many samples behind one long document
        dict(name="shared_b256_16384", op="shared", B=256, groups=1, even=True, prefix=16384, own_rows=128, spread=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["bounds", "select", "sparse", "shared"])
    spread = rng.random() < 0.5
    if op == "bounds":
        T = rng.choice([1, _log_int(rng, 2, 8192)])
        rows = _log_int(rng, 1, 16384)
        B = _log_int(rng, 1, max(1, min(64, 262144 // (rows + T), 16384 // T)))
        return dict(op=op, B=B, T=T, rows=rows, spread=spread, valid_min=rng.choice([0, 1 + T // 8]))
    if op == "shared":
        groups = rng.choice([1, 1, 2, 5])
        prefix = PAGE * _log_int(rng, 1, 128)
        B = _log_int(rng, groups, 256)
        return dict(op=op, B=B, groups=groups, even=rng.random() < 0.5, prefix=prefix,
                    own_rows=_log_int(rng, 1, max(1, min(4096, 131072 // B))), spread=spread)
    rows = _log_int(rng, 1, MAX_ROWS)
    budget = _log_int(rng, 1, 256)
    if op == "select":
        B = _log_int(rng, 1, max(1, min(64, 32 * MAX_ROWS // rows)))
        sink = rng.randint(0, min(4, budget))
        return dict(op=op, B=B, rows=rows, spread=spread, budget=budget, sink=sink,
                    recent=rng.randint(0, min(8, budget - sink)))
    B = _log_int(rng, 1, max(1, min(64, 8 * MAX_ROWS // rows, 1024 // budget)))
    return dict(op=op, B=B, rows=rows, spread=spread, budget=budget, holes=rng.choice([0.0, 0.0, 0.3]))


# ------------------------------------------------------------------------------------------------- the inputs
def _random(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _keys(g, pages):
    """Keys of `pages` pages: a block's rows lie around a point of their own, as those of a passage of text do."""
    near = _random(g, pages, 2, 1, KV, D)
    return (near + 1.5 * _random(g, pages, 2, BLOCK, KV, D)).bfloat16().view(pages, PAGE, KV, D)


def _pool(g, n, make):
    pool = torch.empty(n, PAGE, KV, D, dtype=torch.bfloat16, device="cuda")
    for i in range(0, n, 512):
        m = min(512, n - i)
        pool[i:i + m] = make(g, m)
    return pool


def _values(g, pages):
    return _random(g, pages, PAGE, KV, D).bfloat16()


def _table(g, counts, max_pages, common=(), of=None):
    """A table and the pages in the pool: `counts` pages of each sequence's own, anywhere in the pool, behind the
    common[i] pages of its group i = of[b]."""
    n = sum(common) + len(counts) * (max_pages - min(common, default=0))
    order = torch.randperm(n, generator=g, device="cuda").tolist()
    take = lambda m: [order.pop() for _ in range(m)]  # noqa: E731
    shared = [take(m) for m in common]
    rows = [(shared[of[b]] if common else []) + take(c) for b, c in enumerate(counts)]
    return _ints([row + [-1] * (max_pages - len(row)) for row in rows]), n


def _lengths(case, seed):
    r = random.Random(seed * 7919 + 17)
    least = 0 if case["op"] == "bounds" else 1
    return [r.randint(least, case["rows"]) if case["spread"] else case["rows"] for _ in range(case["B"])], r


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    op, B = case["op"], case["B"]
    if op == "shared":
        return _prepare_shared(case, seed, g)
    rows, r = _lengths(case, seed)
    state = {"case": case}
    if op == "bounds":
        T = case["T"]
        valid = [r.randint(case["valid_min"], T) if case["valid_min"] else T for _ in range(B)]
        max_pages = -(-(case["rows"] + T) // PAGE)
        state["table"], n = _table(g, [-(-(a + T) // PAGE) for a in rows], max_pages)
        state |= {"k_pool": _pool(g, n, _keys), "start_pos": _ints(rows), "valid_len": _ints(valid),
                  "codes": torch.zeros(n, 2, KV, 2, D, dtype=torch.int8, device="cuda"),
                  "scale": torch.zeros(n, 2, KV, device="cuda")}
        return state
    max_pages = -(-case["rows"] // PAGE)
    state["table"], n = _table(g, [-(-a // PAGE) for a in rows], max_pages)
    state |= {"kv_len": _ints(rows), "q_rot": (1.5 * _random(g, B, HEADS, D)).bfloat16()}
    if op == "select":
        # (the bounds of whole blocks: what a sequence's last block holds behind its last row matters little)
        made = [_bounds(_keys(g, min(512, n - i)).view(-1, BLOCK, KV, D)) for i in range(0, n, 512)]
        state |= {"codes": torch.cat([c for c, _ in made]).view(n, 2, KV, 2, D),
                  "scale": torch.cat([s for _, s in made]).view(n, 2, KV),
                  "score": torch.zeros(B, KV, 2 * max_pages, device="cuda"),
                  "sel": torch.full((B, KV, case["budget"]), -1, dtype=torch.int32, device="cuda")}
        return state
    # sparse: the last block and any others, each head its own
    budget = case["budget"]
    blocks = 2 * max_pages
    i = torch.arange(blocks, device="cuda")
    count = (state["kv_len"].long() + BLOCK - 1)[:, None, None] // BLOCK
    rank = torch.rand(B, KV, blocks, generator=g, device="cuda")
    rank = rank.masked_fill(i == count - 1, -1.0).masked_fill(i >= count, 2.0)
    order = rank.argsort(-1)[..., :budget]
    sel = torch.where(order < count, order, blocks).sort(-1).values
    sel = torch.where(sel < blocks, sel, -1)
    sel = sel.masked_fill(torch.rand(sel.shape, generator=g, device="cuda") < case["holes"], -1)
    full = torch.full((B, KV, budget), -1, dtype=torch.int32, device="cuda")
    full[..., :sel.shape[-1]] = sel
    state |= {"k_pool": _pool(g, n, _keys), "v_pool": _pool(g, n, _values), "sel": full,
              "out": torch.zeros(B, HEADS, D, dtype=torch.bfloat16, device="cuda")}
    return state


def _prepare_shared(case, seed, g):
    B, groups = case["B"], case["groups"]
    r = random.Random(seed * 7919 + 17)
    # sequences of a group follow one another
    cuts = [B * i // groups for i in range(groups + 1)] if case["even"] else \
        [0] + sorted(r.sample(range(1, B), groups - 1)) + [B]
    pages = [case["prefix"] // PAGE if not case["spread"] or i == 0 else r.randint(1, case["prefix"] // PAGE)
             for i in range(groups)]
    of = [max(i for i in range(groups) if cuts[i] <= b) for b in range(B)]
    mine = [r.randint(0, case["own_rows"]) if case["spread"] else case["own_rows"] for _ in range(B)]
    max_pages = max(pages[of[b]] + -(-mine[b] // PAGE) for b in range(B))
    table, n = _table(g, [-(-m // PAGE) for m in mine], max_pages, pages, of)
    return {"case": case, "table": table, "kv_len": _ints([pages[of[b]] * PAGE + mine[b] for b in range(B)]),
            "group_start": _ints(cuts), "shared_pages": _ints(pages),
            "k_pool": _pool(g, n, _keys), "v_pool": _pool(g, n, _values),
            "q_rot": (1.5 * _random(g, B, HEADS, D)).bfloat16(),
            "out": torch.zeros(B, HEADS, D, dtype=torch.bfloat16, device="cuda"),
            "cuts": cuts, "pages": pages, "most": max(mine)}


# ------------------------------------------------------------------------------------------------- one pass
def run(state):
    return {"bounds": _run_bounds, "select": _run_select, "sparse": _run_sparse,
            "shared": _run_shared}[state["case"]["op"]](state)


def _exponent(a):
    """The least e with a <= 127 * 2^e, within [LEAST, MOST]."""
    m, e = torch.frexp(torch.where(torch.isfinite(a), a, 1.0))
    e = torch.where(m <= 127.0 / 128.0, e - 7, e - 6)
    e = torch.where(a == 0, LEAST, torch.where(torch.isfinite(a), e, MOST))
    return e.clamp(LEAST, MOST)


def _two(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _whole(x):
    """fp32 values with a NaN taken as the infinity of its sign."""
    x = x.float()
    return torch.where(torch.isnan(x), torch.copysign(torch.full_like(x, math.inf), x), x)


def _bounds(rows, seen=None):
    """Codes [n, 8, 2, 128] and scales [n, 8] of blocks rows [n, 64, 8, 128] whose rows `seen` [n, 64] count."""
    x = _whole(rows)
    if seen is None:
        hi, lo = x.amax(1), x.amin(1)
    else:
        hi = x.masked_fill(~seen[..., None, None], -math.inf).amax(1)
        lo = x.masked_fill(~seen[..., None, None], math.inf).amin(1)
    e = _exponent(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    inv = _two(-e)[..., None]
    upper, lower = torch.ceil(hi * inv).clamp(-127, 127), torch.floor(lo * inv).clamp(-127, 127)
    return torch.stack((upper, lower), 2).to(torch.int8), _two(e)


def _run_bounds(state):
    if own:
        import grok_gqa_attention_gb300 as G
        G.kv_bounds_paged(state["k_pool"], state["table"], state["start_pos"], state["valid_len"],
                          state["case"]["T"], state["codes"], state["scale"])
        return {"codes": state["codes"], "scale": state["scale"]}
    table, T = state["table"].long(), state["case"]["T"]
    start, valid = state["start_pos"].long(), state["valid_len"].long()
    n = (T + 2 * BLOCK - 2) // BLOCK  # blocks that T rows can touch
    block = (start // BLOCK)[:, None] + torch.arange(n, device=table.device)
    end = (start + valid)[:, None]
    touched = block * BLOCK < end
    page = table.gather(1, (block // 2).clamp(max=table.shape[1] - 1))
    at, block = (2 * page + block % 2)[touched], block[touched]
    left = (end.expand_as(touched)[touched] - block * BLOCK)
    seen = torch.arange(BLOCK, device=table.device) < left[:, None]
    codes, scale = _bounds(state["k_pool"].view(-1, BLOCK, KV, D)[at], seen)
    state["codes"].view(-1, KV, 2, D)[at] = codes
    state["scale"].view(-1, KV)[at] = scale
    return {"codes": state["codes"], "scale": state["scale"]}


def _run_select(state):
    case = state["case"]
    budget, sink, recent = case["budget"], case["sink"], case["recent"]
    if own:
        import grok_gqa_attention_gb300 as G
        G.select_blocks_paged(state["q_rot"], state["codes"], state["scale"], state["table"], state["kv_len"],
                              sink, recent, state["score"], state["sel"])
        return {"score": state["score"], "sel": state["sel"]}
    table, length = state["table"].long().clamp(min=0), state["kv_len"].long()
    B, blocks = table.shape[0], 2 * table.shape[1]
    q = _whole(state["q_rot"]).view(B, KV, GROUP, D)
    f = _exponent(q.abs().amax(-1, keepdim=True))
    c = torch.round(q * _two(-f)).clamp(-127, 127)
    codes = state["codes"][table].flatten(1, 2).permute(0, 2, 3, 4, 1).float()  # [B, 8, 2, 128, blocks]
    total = torch.matmul(c.clamp(min=0), codes[:, :, 0]) + torch.matmul(c.clamp(max=0), codes[:, :, 1])
    score = (total * _two(f)).amax(2) * state["scale"][table].flatten(1, 2).transpose(1, 2)
    i = torch.arange(blocks, device=table.device)
    count = ((length + BLOCK - 1) // BLOCK)[:, None, None]
    ranked = score.masked_fill((i < sink) | (i >= count - recent), math.inf).masked_fill(i >= count, -math.inf)
    order = torch.sort(ranked, dim=-1, descending=True, stable=True).indices[..., :budget]
    chosen = torch.where(order < count, order, blocks).sort(-1).values
    sel = torch.full((B, KV, budget), -1, dtype=torch.int32, device=table.device)
    sel[..., :chosen.shape[-1]] = torch.where(chosen < blocks, chosen, -1)
    return {"score": torch.where(i < count, score, state["score"]), "sel": sel}


def _capped(q, k):
    x = torch.matmul(q, k) * MULT
    return CAP * torch.tanh(x / CAP)


def _run_sparse(state):
    case = state["case"]
    if own:
        import grok_gqa_attention_gb300 as G
        if "ws" not in state:
            state["ws"] = G.alloc_decode_sparse_workspace(case["B"], case["budget"])
        G.decode_sparse_paged(state["q_rot"], state["k_pool"], state["v_pool"], state["table"], state["kv_len"],
                              state["sel"], state["ws"], state["out"])
        return state["out"]
    table, sel = state["table"].long().clamp(min=0), state["sel"].long()
    B = table.shape[0]
    at = torch.arange(BLOCK, device=table.device)
    seen = (sel[..., None] >= 0) & (sel[..., None] * BLOCK + at < state["kv_len"].long()[:, None, None, None])
    block = sel.clamp(min=0)
    page = table.gather(1, (block // 2).flatten(1)).view_as(block)
    head = torch.arange(KV, device=table.device)[:, None]
    by_head = lambda pool: pool.view(-1, BLOCK, KV, D).transpose(1, 2)  # noqa: E731
    pick = lambda pool: by_head(pool)[2 * page + block % 2, head].flatten(2, 3).float()  # noqa: E731
    unseen = ~seen.flatten(2)
    c = _capped(state["q_rot"].float().view(B, KV, GROUP, D), pick(state["k_pool"]).transpose(-1, -2))
    p = torch.exp(c - CAP).masked_fill(unseen[:, :, None], 0.0)
    v = pick(state["v_pool"]).masked_fill(unseen[..., None], 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, torch.matmul(p, v) / total, 0.0)
    return out.view(B, HEADS, D).bfloat16()


def _run_shared(state):
    if own:
        import grok_gqa_attention_gb300 as G
        if "ws" not in state:
            state["ws"] = G.alloc_decode_shared_workspace(state["case"]["B"], state["table"].shape[1],
                                                          state["case"]["groups"])
        G.decode_shared_paged(state["q_rot"], state["k_pool"], state["v_pool"], state["table"], state["kv_len"],
                              state["group_start"], state["shared_pages"], state["ws"], state["out"])
        return state["out"]
    table, length = state["table"].long().clamp(min=0), state["kv_len"].long()
    out = torch.empty_like(state["out"])
    own_pages = -(-state["most"] // PAGE)
    for a, z, pages in zip(state["cuts"], state["cuts"][1:], state["pages"]):
        n = z - a
        q = state["q_rot"][a:z].float().view(n, KV, GROUP, D)
        # the common rows, once for the group's queries
        rows = lambda pool, ids: pool[ids].float().flatten(-4, -3).transpose(-3, -2)  # noqa: E731
        k, v = (rows(state[m], table[a, :pages]) for m in ("k_pool", "v_pool"))  # [8, rows, 128]
        many = q.transpose(0, 1).reshape(KV, n * GROUP, D)
        p = torch.exp(_capped(many, k.transpose(-1, -2)) - CAP)
        total = p.sum(-1, keepdim=True).view(KV, n, GROUP, 1).transpose(0, 1)
        o = torch.matmul(p, v).view(KV, n, GROUP, D).transpose(0, 1)
        if own_pages:
            ids = torch.arange(pages, pages + own_pages, device=table.device)
            tail = table[a:z][:, ids.clamp(max=table.shape[1] - 1)]
            k, v = (rows(state[m], tail) for m in ("k_pool", "v_pool"))  # [n, 8, rows, 128]
            at = torch.arange(own_pages * PAGE, device=table.device)
            unseen = (at >= (length[a:z] - pages * PAGE)[:, None])[:, None, None]
            p = torch.exp(_capped(q, k.transpose(-1, -2)) - CAP).masked_fill(unseen, 0.0)
            total = total + p.sum(-1, keepdim=True)
            o = o + torch.matmul(p, v.masked_fill(unseen[:, :, 0, :, None], 0.0))
        out[a:z] = (o / total).reshape(n, HEADS, D).bfloat16()
    return out


# ------------------------------------------------------------------------------------------------- the least work
def _mean_blocks(case, limit):
    """Blocks per sequence, `limit` at most, in the mean over the seeds."""
    if not case["spread"]:
        return min(limit, -(-case["rows"] // BLOCK))
    n = case["rows"]
    return sum(min(limit, -(-i // BLOCK)) for i in range(1, n + 1)) / n


def work(case):
    op, B = case["op"], case["B"]
    q_out = B * 2 * HEADS * D * 2
    if op == "bounds":
        T = case["T"]
        new = (case["valid_min"] + T) / 2 if case["valid_min"] else T
        before = (BLOCK - 1) / 2 if case["spread"] else case["rows"] % BLOCK
        blocks = (before + new + (BLOCK - 1) / 2) / BLOCK if case["spread"] else math.ceil((before + new) / BLOCK)
        return {"bytes": B * ((before + new) * KV * D * 2 + blocks * KV * (2 * D + 4) + 8), "flops": 0}
    if op == "select":
        blocks = B * KV * _mean_blocks(case, MAX_ROWS)
        return {"bytes": blocks * (2 * D + 8) + q_out / 2 + B * KV * case["budget"] * 4,
                "flops": blocks * GROUP * D * 4.0}
    if op == "sparse":
        blocks = B * KV * _mean_blocks(case, case["budget"]) * (1.0 - case["holes"])
        return {"bytes": blocks * (BLOCK * D * 4 + 4) + q_out, "flops": blocks * BLOCK * GROUP * D * 4.0}
    half = 0.5 if case["spread"] else 1.0
    mine = B * case["own_rows"] * half
    each = case["prefix"] * (1.0 + (case["groups"] - 1) * half) / case["groups"]
    rows = case["groups"] * each + mine
    return {"bytes": rows * KV * D * 4 + q_out, "flops": 4.0 * D * HEADS * (B * each + mine)}


# ------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    return {"bounds": _exact_bounds, "select": _exact_select, "sparse": _exact_sparse,
            "shared": _exact_shared}[case["op"]](state)


def _power(a):
    """Of a float64 array of magnitudes, the scale 2^e by its definition: tried from the least up."""
    e = torch.full(a.shape, float(MOST), dtype=torch.float64, device=a.device)
    for i in range(MOST, LEAST - 1, -1):
        e = torch.where(a <= 127.0 * 2.0 ** i, float(i), e)
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_bounds(state):
    codes, scale = state["codes"].double(), state["scale"].double()
    start, valid = state["start_pos"].tolist(), state["valid_len"].tolist()
    for b in range(state["case"]["B"]):
        ids = state["table"][b].tolist()
        for i in range(start[b] // BLOCK, -(-(start[b] + valid[b]) // BLOCK)):
            first = i % 2 * BLOCK
            rows = state["k_pool"][ids[i // 2], first:min(first + BLOCK, start[b] + valid[b] - i // 2 * PAGE)]
            hi, lo = rows.double().max(0).values, rows.double().min(0).values
            two = _power(torch.maximum(hi.abs().max(-1).values, lo.abs().max(-1).values))
            codes[ids[i // 2], i % 2, :, 0] = torch.ceil(hi / two[:, None]).clamp(-127, 127)
            codes[ids[i // 2], i % 2, :, 1] = torch.floor(lo / two[:, None]).clamp(-127, 127)
            scale[ids[i // 2], i % 2] = two
    return {"codes": codes.to(torch.int8), "scale": scale}


def _exact_select(state):
    case = state["case"]
    budget, sink, recent = case["budget"], case["sink"], case["recent"]
    sel = torch.full((case["B"], KV, budget), -1, dtype=torch.int32)
    score = state["score"].double()
    for b, rows in enumerate(state["kv_len"].tolist()):
        n = -(-rows // BLOCK)
        ids = state["table"][b, :-(-n // 2)].long()
        codes = state["codes"][ids].flatten(0, 1)[:n].double()
        scale = state["scale"][ids].flatten(0, 1)[:n].double()
        q = state["q_rot"][b].double().view(KV, GROUP, D)
        two = _power(q.abs().max(-1).values)
        c = torch.round(q / two[..., None]).clamp(-127, 127)
        for h in range(KV):
            s = torch.stack([torch.maximum(c[h, r] * codes[:, h, 0], c[h, r] * codes[:, h, 1]).sum(-1) * two[h, r]
                             for r in range(GROUP)]).max(0).values * scale[:, h]
            score[b, h, :n] = s
            s = s.tolist()
            must = [i for i in range(n) if i < sink or i >= n - recent]
            rest = sorted((i for i in range(n) if sink <= i < n - recent), key=lambda i: (-s[i], i))
            took = sorted((must + rest[:max(0, budget - len(must))]))
            sel[b, h, :len(took)] = torch.tensor(took, dtype=torch.int32)
    return {"score": score, "sel": sel.cuda()}


def _attend(q, k, v):
    c = CAP * torch.tanh(q @ k.T / math.sqrt(D) / CAP)
    return torch.softmax(c, -1) @ v


def _exact_sparse(state):
    case = state["case"]
    out = torch.zeros(case["B"], HEADS, D, dtype=torch.float64, device="cuda")
    sel, length = state["sel"].tolist(), state["kv_len"].tolist()
    for b in range(case["B"]):
        ids = state["table"][b].tolist()
        for h in range(KV):
            flat = [ids[i // 2] * PAGE + i % 2 * BLOCK + j for i in sel[b][h] if i >= 0
                    for j in range(min(BLOCK, length[b] - i * BLOCK))]
            if not flat:
                continue
            flat = torch.tensor(flat, device="cuda")
            k, v = (state[m].view(-1, KV, D)[flat, h].double() for m in ("k_pool", "v_pool"))
            heads = slice(h * GROUP, (h + 1) * GROUP)
            out[b, heads] = _attend(state["q_rot"][b, heads].double(), k, v)
    return out


def _exact_shared(state):
    """Each sequence by itself, over all the rows that its table names."""
    case = state["case"]
    out = torch.zeros(case["B"], HEADS, D, dtype=torch.float64, device="cuda")
    length = state["kv_len"].tolist()
    for b in range(case["B"]):
        ids = state["table"][b, :-(-length[b] // PAGE)].long()
        k, v = (state[m][ids].flatten(0, 1)[:length[b]] for m in ("k_pool", "v_pool"))
        for h in range(KV):
            heads = slice(h * GROUP, (h + 1) * GROUP)
            out[b, heads] = _attend(state["q_rot"][b, heads].double(), k[:, h].double(), v[:, h].double())
    return out
