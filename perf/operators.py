"""The operators of the 8-bit KV cache, as they are measured.

The cache holds blocks of 64 tokens of one KV head: a pool of K blocks [n, 2, 64, 64] (half of the features,
token, feature) and of V blocks [n, 128, 64] (feature, token) in int8 or e4m3, one fp32 scale per block and pool,
a table [B, 8, max_blocks] that names each sequence's blocks per head, and the bf16 rows of the block that is
still open, [B, 8, 64, 128]. A block with rows x has scale s = RN32(max|x| / Q), Q = 127 (int8) or 448 (e4m3), and
codes round(RN32(x RN32(1 / s))).

Four operators: the append (RoPE and quantisation), single-token attention with the weight that each block
received, attention of many tokens, and the eviction of the blocks with the least accumulated weight.
"""
import math
import random

import torch

own = False

HEADS, KV, GROUP, D, BLOCK = 48, 8, 6, 128, 64
MULT, CAP = 1.0 / math.sqrt(128.0), 30.0
TINY = 2.0 ** -100  # a block whose largest magnitude is below this counts as zero
MAX_ROWS = 65536


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence answering, its new token into a long cache: latency
        dict(name="append_step_b1", op="append", kind="int8", B=1, T=1, rows=8190, spread=False, valid_min=0),
        # a decode batch: 32 sequences at their own lengths
        dict(name="append_step_b32", op="append", kind="e4m3", B=32, T=1, rows=8191, spread=True, valid_min=0),
        # a long prompt into an empty cache
        dict(name="append_prompt_8192", op="append", kind="int8", B=1, T=8192, rows=0, spread=False, valid_min=0),
        # a padded batch of prompts of 256 to 2048 tokens
        dict(name="append_ragged_b8", op="append", kind="e4m3", B=8, T=2048, rows=0, spread=False, valid_min=256),
        # the first tokens of an answer to a short question: latency
        dict(name="decode_b1_300", op="decode", kind="int8", B=1, rows=300, spread=False, weights=False),
        # a serving batch with lengths over the whole context, the blocks' weights kept for eviction
        dict(name="decode_b32_8192_weights", op="decode", kind="int8", B=32, rows=8192, spread=True, weights=True),
        # few sequences with very long contexts
        dict(name="decode_b4_65536", op="decode", kind="e4m3", B=4, rows=65536, spread=True, weights=False),
        # a short prompt: latency
        dict(name="prefill_b1_128", op="prefill", kind="int8", B=1, T=128, rows=0, spread=False, valid_min=0),
        # a chunk of a longer prompt behind a warm cache
        dict(name="prefill_chunk_b4", op="prefill", kind="int8", B=4, T=256, rows=6144, spread=False, valid_min=0),
        # a long prompt at once
        dict(name="prefill_8192", op="prefill", kind="e4m3", B=1, T=8192, rows=0, spread=False, valid_min=0),
        # one conversation that outgrew its budget
        dict(name="evict_b1", op="evict", B=1, blocks=129, keep=96, sink=1, recent=4),
        # a large batch at the longest context
        dict(name="evict_b256", op="evict", B=256, blocks=1024, keep=512, sink=4, recent=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "evict"])
    kind = rng.choice(["int8", "e4m3"])
    if op == "append":
        T = rng.choice([1, _log_int(rng, 2, 8192)])
        B = _log_int(rng, 1, max(1, min(32, 16384 // T)))
        return dict(op=op, kind=kind, B=B, T=T, rows=_log_int(rng, 1, min(16384, MAX_ROWS - T - 512)),
                    spread=rng.random() < 0.5, valid_min=rng.choice([0, 1 + T // 8]))
    if op == "decode":
        rows = _log_int(rng, 1, 65536)
        B = _log_int(rng, 1, max(1, min(64, 131072 // rows)))
        return dict(op=op, kind=kind, B=B, rows=rows, spread=rng.random() < 0.5, weights=rng.random() < 0.5)
    if op == "prefill":
        T = _log_int(rng, 2, 4096)
        B = _log_int(rng, 1, max(1, min(8, 8192 // T)))
        rows = _log_int(rng, 1, max(1, min(16384, 16777216 // (B * T))))
        return dict(op=op, kind=kind, B=B, T=T, rows=rows, spread=rng.random() < 0.5,
                    valid_min=rng.choice([0, 1 + T // 8]))
    blocks = _log_int(rng, 2, 1024)
    keep = rng.randint(1, blocks)
    sink = rng.randint(0, min(4, keep))
    return dict(op=op, B=_log_int(rng, 1, 256), blocks=blocks, keep=keep, sink=sink,
                recent=rng.randint(0, min(64, keep - sink)))


# ------------------------------------------------------------------------------------------------- the inputs
def _lengths(case, seed):
    """Rows in the cache before the new tokens (append, prefill) or in all (decode), and the valid new tokens."""
    r = random.Random(seed * 7919 + 17)
    B, T = case["B"], case.get("T", 0)
    rows = [r.randint(1 if case["op"] == "decode" else 0, case["rows"]) if case["spread"] else case["rows"]
            for _ in range(B)]
    valid = [r.randint(case["valid_min"], T) if case.get("valid_min") else T for _ in range(B)]
    if case["op"] == "append" and T > 1:
        # The pass is run again on the same state: an open block that this call both reads and closes must not
        # be followed by another open one, whose rows would take its place.
        for b in range(B):
            end = rows[b] + valid[b]
            if rows[b] % BLOCK and end // BLOCK > rows[b] // BLOCK and end % BLOCK:
                if end % BLOCK < valid[b]:
                    valid[b] -= end % BLOCK
                else:
                    rows[b] -= rows[b] % BLOCK
    return rows, valid


def _quantise(x, seen, kind):
    """Codes and scales of blocks x [..., 64, 128] (fp32) whose rows `seen` [..., 64] count."""
    top = 127.0 if kind == "int8" else 448.0
    a = torch.where(seen[..., None], x.abs(), 0.0).amax((-1, -2))
    fine = torch.isfinite(a)
    zero = a < TINY
    scale = torch.where(fine, torch.where(zero, 0.0, a / torch.full_like(a, top)), math.nan)
    inv = torch.where(fine & ~zero, torch.ones_like(a) / scale, 0.0)
    y = torch.where((fine & ~zero)[..., None, None], x * inv[..., None, None], 0.0)
    y = torch.where(seen[..., None], y, 0.0)
    return (torch.round(y).to(torch.int8) if kind == "int8" else y.to(torch.float8_e4m3fn)), scale


def _as_k(c):  # [..., 64, 128] -> [..., 2, 64, 64]
    return c.unflatten(-1, (2, 64)).transpose(-3, -2)


def _as_v(c):  # [..., 64, 128] -> [..., 128, 64]
    return c.transpose(-1, -2)


def _dtype(kind):
    return torch.int8 if kind == "int8" else torch.float8_e4m3fn


def _random(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rope_tables(n):
    """cos and sin [n, 64]: fp32 values of the fp32 phase of each position."""
    j = torch.arange(64, dtype=torch.float64, device="cuda")
    base = torch.pow(torch.full_like(j, 10000.0), j / 64.0).float()
    phase = (torch.arange(n, device="cuda").float()[:, None] * (torch.ones_like(base) / base)[None, :]).double()
    return phase.cos().float(), phase.sin().float()


def _table(g, B, max_blocks):
    n = B * KV * max_blocks
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(B, KV, max_blocks), n


def _filled(g, rows, max_blocks, kind):
    """A cache of `rows` tokens a sequence: normal values, a head's keys and values at its own magnitude."""
    B = len(rows)
    table, n = _table(g, B, max_blocks)
    length = torch.tensor(rows, device="cuda")
    at = torch.arange(max_blocks * BLOCK, device="cuda").view(1, max_blocks, BLOCK)
    seen = (at < length[:, None, None])[:, None].expand(B, KV, max_blocks, BLOCK)
    made = []
    for _ in range(2):
        size = 3.0 * (0.5 + 1.0 * torch.rand(B, KV, 1, 1, 1, generator=g, device="cuda"))
        x = (_random(g, B, KV, max_blocks, BLOCK, D) * size).bfloat16().float()
        made.append(_quantise(x, seen, kind))
    flat = table.flatten().long()
    state = {}
    for (codes, scale), name, lay in zip(made, ("k", "v"), (_as_k, _as_v)):
        laid = lay(codes.view(torch.uint8)).flatten(0, 2)
        pool = torch.empty((n,) + tuple(laid.shape[1:]), dtype=torch.uint8, device="cuda")
        pool[flat] = laid
        state[name + "_pool"] = pool.view(_dtype(kind))
        scales = torch.empty(n, device="cuda")
        scales[flat] = scale.flatten()
        state[name + "_scale"] = scales
    state["table"] = table
    state["open_k"] = torch.zeros(B, KV, BLOCK, D, dtype=torch.bfloat16, device="cuda")
    state["open_v"] = torch.zeros_like(state["open_k"])
    return state


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed) * 1000003 + 11)
    op, B = case["op"], case["B"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "evict":
        r = random.Random(seed * 7919 + 17)
        rows = [case["blocks"] * BLOCK - r.randint(0, min(BLOCK * case["blocks"] // 4, 4096)) for _ in range(B)]
        table, n = _table(g, B, case["blocks"])
        # what blocks gather over many steps: a few get most of the weight
        weight = torch.exp(1.5 * _random(g, B, KV, case["blocks"]))
        return {"case": case, "table": table, "kv_len": ints(rows), "weight": weight,
                "table_out": torch.empty_like(table), "weight_out": torch.empty_like(weight),
                "kv_len_out": ints([0] * B)}
    rows, valid = _lengths(case, seed)
    kind = case["kind"]
    if op == "decode":
        max_blocks = -(-case["rows"] // BLOCK)
        state = _filled(g, rows, max_blocks, kind)
        state |= {"case": case, "kv_len": ints(rows), "q_rot": (_random(g, B, HEADS, D) * 3).bfloat16(),
                  "out": torch.zeros(B, HEADS, D, dtype=torch.bfloat16, device="cuda")}
        if case["weights"]:
            state["weight"] = torch.exp(1.5 * _random(g, B, KV, max_blocks))
            state["weight_out"] = torch.zeros_like(state["weight"])
        return state
    T = case["T"]
    if op == "prefill":
        ends = [a + b for a, b in zip(rows, valid)]
        max_blocks = -(-(case["rows"] + T) // BLOCK)
        state = _filled(g, ends, max_blocks, kind)
        state |= {"case": case, "cache_len": ints(rows), "valid_len": ints(valid),
                  "q_rot": (_random(g, B, T, HEADS, D) * 3).bfloat16(),
                  "out": torch.zeros(B, T, HEADS, D, dtype=torch.bfloat16, device="cuda")}
        return state
    # append: an empty pool but for the block that is open, whose rows are at hand in bf16
    max_blocks = -(-(case["rows"] + T) // BLOCK)
    table, n = _table(g, B, max_blocks)
    state = {"case": case, "table": table, "cache_len": ints(rows), "valid_len": ints(valid)}
    # positions run ahead of the rows where blocks were evicted before
    state["start_pos"] = ints([a + 64 * (i % 4) for i, a in enumerate(rows)])
    state["cos"], state["sin"] = _rope_tables(case["rows"] + T + 256)
    for name, heads in (("q", HEADS), ("k", KV), ("v", KV)):
        state[name] = (_random(g, B, T, heads, D) * 3).bfloat16()
    state["q_rot"] = torch.zeros_like(state["q"])
    left = torch.tensor([a % BLOCK for a in rows], device="cuda")
    at = (torch.tensor(rows, device="cuda") // BLOCK).clamp(max=max_blocks - 1)
    seen = (torch.arange(BLOCK, device="cuda")[None, :] < left[:, None])[:, None].expand(B, KV, BLOCK)
    ids = table.gather(2, at[:, None, None].expand(B, KV, 1)).flatten().long()
    for name, lay in (("k", _as_k), ("v", _as_v)):
        rows_open = (_random(g, B, KV, BLOCK, D) * 3).bfloat16()
        codes, scale = _quantise(rows_open.float(), seen, kind)
        laid = lay(codes.view(torch.uint8)).flatten(0, 1)
        pool = torch.zeros((n,) + tuple(laid.shape[1:]), dtype=torch.uint8, device="cuda")
        pool[ids] = laid
        state[name + "_pool"] = pool.view(_dtype(kind))
        state[name + "_scale"] = torch.zeros(n, device="cuda")
        state[name + "_scale"][ids] = scale.flatten()
        state["open_" + name] = rows_open
    return state


# ------------------------------------------------------------------------------------------------- one pass
def _cache(state):
    """The framework's handle of the cache and its workspace, made once and kept, as a user's program keeps them."""
    import grok_gqa_attention_gb300 as G
    if "cache" not in state:
        state["cache"] = G.Kv8Cache(state["k_pool"], state["v_pool"], state["k_scale"], state["v_scale"],
                                    state["table"], state["open_k"], state["open_v"])
        op = state["case"]["op"]
        if op == "decode":
            state["ws"] = G.alloc_kv8_decode_workspace(state["cache"])
        elif op == "prefill":
            state["ws"] = G.alloc_kv8_prefill_workspace(state["cache"])
    return G, state["cache"]


def run(state):
    op = state["case"]["op"]
    if op == "append":
        return _append(state)
    if op == "decode":
        return _decode(state)
    if op == "prefill":
        return _prefill(state)
    return _evict(state)


def _append(state):
    if own:
        G, cache = _cache(state)
        G.kv8_append(cache, state["q"], state["k"], state["v"], state["start_pos"], state["cache_len"],
                     state["valid_len"], state["cos"], state["sin"], state["q_rot"])
        return {n: state[n] for n in ("q_rot", "k_pool", "v_pool", "k_scale", "v_scale", "open_k", "open_v")}
    q, k, v, table = state["q"], state["k"], state["v"], state["table"]
    B, T = q.shape[:2]
    dev = q.device
    length, valid = state["cache_len"].long(), state["valid_len"].long()
    pos = state["start_pos"].long()[:, None] + torch.arange(T, device=dev)
    c, s = state["cos"][pos][:, :, None], state["sin"][pos][:, :, None]  # [B, T, 1, 64]

    def rotate(x):
        a, b = x[..., :64].float(), x[..., 64:].float()
        return torch.cat((a * c - b * s, b * c + a * s), -1).bfloat16()

    q_rot = rotate(q)
    left = length % BLOCK
    n = -(-(T + BLOCK - 1) // BLOCK)  # blocks that T tokens can touch
    rel = torch.arange(n * BLOCK, device=dev)[None, :] - left[:, None]  # new token of each row of those blocks
    is_old = rel < 0
    is_new = (rel >= 0) & (rel < valid[:, None])
    seen = (is_old | is_new).view(B, 1, n, BLOCK).expand(B, KV, n, BLOCK)
    fresh = is_new.view(B, 1, n, BLOCK).expand(B, KV, n, BLOCK)
    first = (length // BLOCK)[:, None] + torch.arange(n, device=dev)
    touched = fresh.any(-1)
    ids = table.long().gather(2, first.clamp(max=table.shape[2] - 1)[:, None].expand(B, KV, n))
    ids = ids[touched]
    end = length + valid
    out = {"q_rot": q_rot}
    for name, x, lay in (("k", rotate(k), _as_k), ("v", v, _as_v)):
        old = state["open_" + name]
        pick = rel.clamp(0, T - 1)[:, :, None, None].expand(B, n * BLOCK, KV, D)
        new = x.gather(1, pick).transpose(1, 2)  # [B, 8, n * 64, 128]
        kept = old[:, :, torch.arange(n * BLOCK, device=dev) % BLOCK]
        rows = torch.where(is_old[:, None, :, None], kept, new).view(B, KV, n, BLOCK, D)
        codes, scale = _quantise(rows.float(), seen, state["case"]["kind"])
        laid = lay(codes.view(torch.uint8))[touched]
        mask = lay(seen[..., None].expand(B, KV, n, BLOCK, D))[touched]
        pool = state[name + "_pool"].view(torch.uint8)
        pool[ids] = torch.where(mask, laid, pool[ids])
        state[name + "_scale"][ids] = scale[touched]
        # the rows of the block that is open afterwards
        last = (end // BLOCK - length // BLOCK).clamp(max=n - 1)[:, None, None, None, None].expand(B, KV, 1, BLOCK, D)
        tail = rows.gather(2, last)[:, :, 0]
        here = fresh.gather(2, last[..., 0])[:, :, 0] & (end % BLOCK != 0)[:, None, None]
        old.copy_(torch.where(here[..., None], tail, old))
    return out | {m: state[m] for m in ("k_pool", "v_pool", "k_scale", "v_scale", "open_k", "open_v")}


def _values(state):
    """Keys and values [B, 8, max_blocks * 64, 128] in fp32, as the cache holds them."""
    table = state["table"].long()
    k = state["k_pool"].view(torch.uint8)[table].view(state["k_pool"].dtype).float()
    k = (k * state["k_scale"][table][..., None, None, None]).transpose(-3, -2).flatten(-2).flatten(2, 3)
    v = state["v_pool"].view(torch.uint8)[table].view(state["v_pool"].dtype).float()
    v = (v * state["v_scale"][table][..., None, None]).transpose(-1, -2).flatten(2, 3)
    return k, v


def _decode(state):
    weights = "weight" in state
    if own:
        G, cache = _cache(state)
        G.kv8_decode(cache, state["q_rot"], state["kv_len"], state["ws"], state["out"], state.get("weight"),
                     state.get("weight_out"))
        return {"out": state["out"], "weight": state["weight_out"]} if weights else {"out": state["out"]}
    k, v = _values(state)
    B = k.shape[0]
    unseen = (torch.arange(k.shape[2], device=k.device)[None] >= state["kv_len"].long()[:, None])[:, None, None]
    x = torch.matmul(state["q_rot"].float().view(B, KV, GROUP, D), k.transpose(-1, -2)) * MULT
    x = (CAP * torch.tanh(x / CAP)).masked_fill_(unseen, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = v.masked_fill(unseen[:, :, 0, :, None], 0.0)
    out = torch.matmul(p, v).view(B, HEADS, D).bfloat16()
    if not weights:
        return {"out": out}
    return {"out": out, "weight": state["weight"] + p.unflatten(-1, (-1, BLOCK)).sum((2, 4))}


def _prefill(state):
    if own:
        G, cache = _cache(state)
        G.kv8_prefill(cache, state["q_rot"], state["cache_len"], state["valid_len"], state["out"], state["ws"])
        return state["out"]
    k, v = _values(state)
    B, T = state["q_rot"].shape[:2]
    length, valid = state["cache_len"].long(), state["valid_len"].long()
    j = torch.arange(k.shape[2], device=k.device)
    row = length[:, None] + torch.arange(T, device=k.device)
    unseen = (j > row[:, :, None]) | (j >= (length + valid)[:, None, None])  # [B, T, J]
    q = state["q_rot"].float().view(B, T, KV, GROUP, D).permute(0, 2, 3, 1, 4).reshape(B, KV, GROUP * T, D)
    x = torch.matmul(q, k.transpose(-1, -2)).view(B, KV, GROUP, T, -1)
    x = x.mul_(MULT / CAP).tanh_().mul_(CAP).masked_fill_(unseen[:, None, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, KV, GROUP * T, -1), v).view(B, KV, GROUP, T, D) / total
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, HEADS, D).bfloat16()


def _evict(state):
    case = state["case"]
    keep, sink, recent = case["keep"], case["sink"], case["recent"]
    if own:
        import grok_gqa_attention_gb300 as G
        G.kv8_evict(state["table"], state["weight"], state["kv_len"], keep, sink, recent, state["table_out"],
                    state["weight_out"], state["kv_len_out"])
        return {"table": state["table_out"], "weight": state["weight_out"], "kv_len": state["kv_len_out"]}
    table, weight, length = state["table"], state["weight"], state["kv_len"].long()
    n = table.shape[2]
    i = torch.arange(n, device=table.device).expand_as(table)
    closed = (length // BLOCK)[:, None, None]
    # 0: always kept, 1: by weight, 2: not a closed block
    group = torch.where((i < sink) | (i >= closed - recent), 0, 1).masked_fill(i >= closed, 2)
    score = torch.nan_to_num(weight, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    by_score = torch.sort(score, dim=-1, descending=True, stable=True).indices
    order = by_score.gather(-1, torch.sort(group.gather(-1, by_score), dim=-1, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, i.contiguous())
    # the row's new order: kept blocks, the open one, evicted ones, the rest
    place = torch.where(i < closed, torch.where(rank < keep, 0, 2), torch.where(i == closed, 1, 3))
    place = torch.where(closed > keep, place, 0)
    new = torch.sort(place, dim=-1, stable=True).indices
    left = torch.where(length // BLOCK > keep, keep * BLOCK + length % BLOCK, length)
    gone = (place == 2).gather(-1, new)
    return {"table": table.gather(-1, new), "weight": weight.gather(-1, new).masked_fill(gone, 0.0),
            "kv_len": left.to(torch.int32)}


# ------------------------------------------------------------------------------------------------- the least work
def work(case):
    op, B = case["op"], case["B"]
    if op == "evict":
        return {"bytes": B * KV * case["blocks"] * 16 + B * 8, "flops": 0}
    # the mean over the seeds, where lengths are drawn
    rows = case["rows"] * (0.5 if case["spread"] else 1.0)
    per_row = KV * (2 * D + 8 / BLOCK)  # codes and scales of a token
    if op == "decode":
        bytes_ = B * (rows * per_row + 2 * HEADS * D * 2 + 4)
        if case["weights"]:
            bytes_ += B * KV * 8 * rows / BLOCK
        return {"bytes": bytes_, "flops": 4.0 * D * HEADS * B * rows}
    T = case["T"]
    new = (case["valid_min"] + T) / 2 if case["valid_min"] else T
    if op == "append":
        per_new = 2 * KV * D * 2 + per_row
        if T < BLOCK:
            per_new += 2 * KV * D * 2  # the new rows of the open block in bf16
        return {"bytes": B * (T * 2 * HEADS * D * 2 + new * per_new + T * 512 + 12), "flops": 6.0 * B * T * (HEADS + KV) * D / 2}
    seen = B * (new * (rows + (new + 1) / 2) + (T - new) * (rows + new))
    return {"bytes": B * (T * 2 * HEADS * D * 2 + (rows + new) * per_row + 8), "flops": 4.0 * D * HEADS * seen}


# ------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        return _exact_evict(state)
    if op == "append":
        return _exact_append(state)
    if op == "prefill":
        return _exact_prefill(state)
    return _exact_decode(state)


def _exact_head(state, b, h, rows):
    """Keys and values [rows, 128] of one head, and the scales' product done in 64 bits."""
    ids = state["table"][b, h, :-(-rows // BLOCK)].long()
    k = state["k_pool"].view(torch.uint8)[ids].view(state["k_pool"].dtype).to(torch.float32).double()
    v = state["v_pool"].view(torch.uint8)[ids].view(state["v_pool"].dtype).to(torch.float32).double()
    k = torch.cat((k[:, 0], k[:, 1]), -1) * state["k_scale"][ids].double()[:, None, None]
    v = v.permute(0, 2, 1) * state["v_scale"][ids].double()[:, None, None]
    return k.reshape(-1, D)[:rows], v.reshape(-1, D)[:rows]


def _exact_decode(state):
    case = state["case"]
    out = torch.zeros(case["B"], HEADS, D, dtype=torch.float64, device="cuda")
    weight = state["weight"].double() if case["weights"] else None
    for b, rows in enumerate(state["kv_len"].tolist()):
        for h in range(KV):
            k, v = _exact_head(state, b, h, rows)
            q = state["q_rot"][b, h * GROUP:(h + 1) * GROUP].double()
            c = CAP * torch.tanh(q @ k.T / math.sqrt(D) / CAP)
            p = torch.softmax(c, -1)
            out[b, h * GROUP:(h + 1) * GROUP] = p @ v
            if weight is not None:
                each = p.sum(0)
                each = torch.cat((each, each.new_zeros(-rows % BLOCK))).view(-1, BLOCK).sum(1)
                weight[b, h, :each.numel()] += each
    return {"out": out} if weight is None else {"out": out, "weight": weight}


def _exact_prefill(state):
    B, T = state["q_rot"].shape[:2]
    out = torch.zeros(B, T, HEADS, D, dtype=torch.float64, device="cuda")
    lens, valid = state["cache_len"].tolist(), state["valid_len"].tolist()
    for b in range(B):
        rows = lens[b] + valid[b]
        last = (torch.arange(T, device="cuda") + lens[b]).clamp(max=rows - 1)
        hidden = torch.arange(rows, device="cuda")[None, :] > last[:, None]
        for h in range(HEADS):
            if h % GROUP == 0:
                k, v = _exact_head(state, b, h // GROUP, rows)
            c = state["q_rot"][b, :, h].double() @ k.T
            c = c.div_(math.sqrt(D) * CAP).tanh_().mul_(CAP).masked_fill_(hidden, -math.inf)
            out[b, :, h] = torch.softmax(c, -1) @ v
    return out


def _exact_append(state):
    """The rotation in real numbers; the codes by their definition, whose roundings are part of it."""
    case = state["case"]
    top = 127.0 if case["kind"] == "int8" else 448.0
    single = lambda x: x.float().double()  # noqa: E731
    lens, valid, starts = (state[n].tolist() for n in ("cache_len", "valid_len", "start_pos"))
    T = case["T"]
    out = {n: state[n].float().double() for n in ("k_scale", "v_scale", "open_k", "open_v")}
    out["q_rot"] = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    pools = {n: state[n + "_pool"].float().double() for n in ("k", "v")}
    for b in range(case["B"]):
        c = state["cos"][starts[b]:starts[b] + T].double()[:, None]
        s = state["sin"][starts[b]:starts[b] + T].double()[:, None]
        lo, hi = state["q"][b, ..., :64].double(), state["q"][b, ..., 64:].double()
        out["q_rot"][b] = torch.cat((lo * c - hi * s, hi * c + lo * s), -1)
        lo, hi = state["k"][b, ..., :64].double(), state["k"][b, ..., 64:].double()
        rotated = torch.cat((single(lo * c) - single(hi * s), single(hi * c) + single(lo * s)), -1)
        rotated = rotated.float().bfloat16().double()
        n, used = valid[b], lens[b] % BLOCK
        for name, x in (("k", rotated), ("v", state["v"][b].double())):
            rows = torch.cat((state["open_" + name][b, :, :used].double(), x[:n].transpose(0, 1)), 1)  # [8, used + n, 128]
            whole = -(-rows.shape[1] // BLOCK)
            for i in range(whole):
                part = rows[:, i * BLOCK:(i + 1) * BLOCK]
                scale = (part.abs().amax((1, 2)) / top)
                inv = single(1.0 / single(scale))
                y = single(part * inv[:, None, None])
                code = torch.round(y) if case["kind"] == "int8" else y.float().to(torch.float8_e4m3fn).float().double()
                ids = state["table"][b, :, lens[b] // BLOCK + i].long()
                out[name + "_scale"][ids] = scale
                m = part.shape[1]
                if name == "k":
                    pools["k"][ids, 0, :m], pools["k"][ids, 1, :m] = code[..., :64], code[..., 64:]
                else:
                    pools["v"][ids, :, :m] = code.transpose(1, 2)
            left = rows.shape[1] % BLOCK
            if left:
                keep = used if rows.shape[1] < BLOCK else 0  # rows that were there before
                out["open_" + name][b, :, keep:left] = rows[:, rows.shape[1] - left + keep:]
    floating = case["kind"] != "int8"
    return {"q_rot": out["q_rot"], "k_scale": out["k_scale"], "v_scale": out["v_scale"], "open_k": out["open_k"],
            "open_v": out["open_v"], "k_pool": pools["k"] if floating else pools["k"].to(torch.int8),
            "v_pool": pools["v"] if floating else pools["v"].to(torch.int8)}


def _exact_evict(state):
    case = state["case"]
    weight, B = state["weight"].double().cpu(), case["B"]
    lens, out = state["kv_len"].tolist(), weight.clone()
    for b in range(B):
        closed = lens[b] // BLOCK
        if closed <= case["keep"]:
            continue
        for h in range(KV):
            w = weight[b, h].tolist()
            must = [i for i in range(closed) if i < case["sink"] or i >= closed - case["recent"]]
            free = range(case["sink"], closed - case["recent"])
            rest = sorted(free, key=lambda i: (-w[i], i))
            kept = sorted(must + rest[:case["keep"] - len(must)])
            gone = [0.0] * (closed - len(kept))
            fresh = [w[i] for i in kept] + w[closed:closed + 1] + gone + w[closed + 1:]
            out[b, h] = torch.tensor(fresh, dtype=torch.float64)
    return {"table": None, "kv_len": None, "weight": out}
