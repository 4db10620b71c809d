"""Serving from a paged cache that is cut down by accumulated attention weight.

The operators of one model layer (or, for the eviction, of all layers) whose keys and
values lie in the pages of a pool, found through a table of page numbers per sequence:

  store   bkv_store_paged: rotary positions (half or interleaved pairs, part of the head,
          scaled for long contexts) of packed queries and keys, keys and values to their
          pages;
  attend  bkv_attend_paged: attention of one new token per sequence over its pages, with
          the attention weight that every slot received added to the slot's account;
  weigh   bkv_weigh_prompt: the attention weight that a prompt's (or a chunk's) queries
          give to every slot, summed per KV head, from the log-sum-exps that the prompt's
          attention has left;
  evict   bkv_evict_weight: keeps the prefix, the recent window and the slots with the
          most accumulated weight, in every layer, and moves keys, values and weights.

A pool is [pages][kv_heads][page_size][d], weights [pages][kv_heads][page_size]; page_size
0 in a case stands for the dense caches of the other calls, [batch][kv_heads][max_cache][d].
Head shapes, budgets and batches are those of synth/workloads.py, and generic ones (one
query head per KV head, 16, 24). With `own` false, run() computes the same in elementary
torch operations.
"""

import math
import random

import numpy as np
import torch

own = False

D = 128
# query heads, KV heads: the head shapes of the workloads, and one, 16 and 24 query heads per KV head
SHAPES = [(4, 1), (32, 8), (40, 8), (28, 4), (8, 8), (32, 2), (24, 1)]
PAGES = [0, 16, 32, 48, 64, 128, 256]


def listed():
    return [
        # the new token of each of 192 sequences, far behind, frequencies stretched fourfold
        {"name": "store_decode", "op": "store", "heads": 32, "kv_heads": 8, "batch": 192, "tokens": 1, "spread": 0.0, "context": 2063,
         "position": 32767, "theta": 1e6, "rotary": 128, "interleaved": False, "scaling": "yarn", "factor": 4.0, "page": 64},
        # ragged prompts, interleaved pairs in the first half of the head
        {"name": "store_prompt", "op": "store", "heads": 40, "kv_heads": 8, "batch": 8, "tokens": 4100, "spread": 0.4, "context": 0,
         "position": 0, "theta": 1e4, "rotary": 64, "interleaved": True, "scaling": "none", "factor": 1.0, "page": 16},
        # a single sequence's decode step at the 2K budget: latency
        {"name": "attend_b1", "op": "attend", "heads": 32, "kv_heads": 8, "batch": 1, "length": 2063, "spread": 0.0, "empty": False,
         "page": 16, "weighed": True, "decay": 1.0},
        # 192 sequences at the 2K budget, every slot's weight kept up to date
        {"name": "attend_b192", "op": "attend", "heads": 32, "kv_heads": 8, "batch": 192, "length": 2063, "spread": 0.1, "empty": False,
         "page": 64, "weighed": True, "decay": 1.0},
        # ragged lengths in the dense caches, slots left empty by finished sequences, GQA 7
        {"name": "attend_ragged", "op": "attend", "heads": 28, "kv_heads": 4, "batch": 64, "length": 4112, "spread": 0.9, "empty": True,
         "page": 0, "weighed": True, "decay": 0.95},
        # long answers of 32K tokens before any eviction, GQA 5, no account
        {"name": "attend_long", "op": "attend", "heads": 40, "kv_heads": 8, "batch": 3, "length": 32767, "spread": 0.5, "empty": False,
         "page": 256, "weighed": False, "decay": 1.0},
        # four chat turns of a few dozen tokens: latency
        {"name": "weigh_short", "op": "weigh", "heads": 32, "kv_heads": 8, "batch": 4, "tokens": 45, "spread": 0.9, "context": 0, "empty": True,
         "page": 16, "decay": 0.0},
        # prompts around the 2K budget, ragged
        {"name": "weigh_2k", "op": "weigh", "heads": 32, "kv_heads": 8, "batch": 8, "tokens": 2064, "spread": 0.4, "context": 0, "empty": False,
         "page": 64, "decay": 0.0},
        # two long prompts, GQA 7, in the caches that prompt attention reads: the largest work
        {"name": "weigh_8k", "op": "weigh", "heads": 28, "kv_heads": 4, "batch": 2, "tokens": 8190, "spread": 0.02, "context": 0, "empty": False,
         "page": 0, "decay": 0.0},
        # one sequence, all layers, 16 slots over the 2K budget
        {"name": "evict_b1", "op": "evict", "layers": 36, "heads": 32, "kv_heads": 8, "batch": 1, "length": 2064, "spread": 0.0, "budget": 2048,
         "prefix": 4, "recent": 16, "order_free": False, "page": 16},
        # a batch's sequences cut from 2048 to 1792 slots in a group of four layers
        {"name": "evict_b192", "op": "evict", "layers": 4, "heads": 32, "kv_heads": 8, "batch": 192, "length": 2048, "spread": 0.05, "budget": 1792,
         "prefix": 4, "recent": 16, "order_free": False, "page": 64},
        # the 1K budget in the dense caches, only the dropped slots filled
        {"name": "evict_order_free", "op": "evict", "layers": 8, "heads": 40, "kv_heads": 8, "batch": 64, "length": 1040, "spread": 0.0, "budget": 1024,
         "prefix": 4, "recent": 16, "order_free": True, "page": 0},
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b + 0.49)))))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "weigh", "weigh", "evict", "evict"])
    heads, kv_heads = rng.choice(SHAPES)
    page = rng.choice(PAGES)
    spread = round(rng.uniform(0.0, 0.9), 2)
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "page": page, "spread": spread}
    if op == "store":
        case["batch"] = _log(rng, 1, 192)
        case["tokens"] = rng.choice([1, _log(rng, 1, 26000 // case["batch"])])
        case |= {"context": _log(rng, 1, 2063), "position": _log(rng, 1, 131072), "theta": rng.choice([1e4, 1e6]),
                 "rotary": rng.choice([16, 32, 64, 96, 128]), "interleaved": rng.random() < 0.5}
        case["scaling"] = rng.choice(["none", "linear", "ntk", "yarn"])
        case["factor"] = 1.0 if case["scaling"] == "none" else rng.choice([2.0, 4.0, 8.0, 5.5])
        return case
    if op == "attend":
        case["batch"] = _log(rng, 1, 192)
        case["length"] = _log(rng, 1, min(32768, 192 * 2063 * 8 // (kv_heads * case["batch"])))
        weighed = rng.random() < 0.6
        return case | {"empty": case["batch"] > 1 and rng.random() < 0.3, "weighed": weighed,
                       "decay": rng.choice([1.0, 1.0, 0.95, 0.0]) if weighed else 1.0}
    if op == "weigh":
        batch = _log(rng, 1, 16)
        tokens = _log(rng, 1, min(8000, 4000000 // (40 * batch)))
        context = rng.choice([0, 0, _log(rng, 1, 2048)])
        while heads * batch * tokens * (tokens + context) > 28 * 2 * 8000 * 8000:
            tokens = tokens * 3 // 4
        return case | {"batch": batch, "tokens": tokens, "context": context, "empty": batch > 1 and rng.random() < 0.3,
                       "decay": rng.choice([0.0, 1.0, 0.95])}
    budget = _log(rng, 8, 4096)
    over = _log(rng, 1, 512)
    recent = rng.choice([0, min(16, budget // 4)])
    order_free = rng.random() < 0.3
    if order_free:
        over = max(over, recent + 1)
        case["spread"] = 0.0  # shorter than budget + recent is refused in this mode
    layers = rng.randint(1, 36)
    batch = _log(rng, 1, max(1, min(192, 4 * 192 * 8 * 2048 // (layers * kv_heads * (budget + over)))))
    return case | {"layers": layers, "batch": batch, "length": budget + over, "budget": budget, "prefix": rng.choice([0, min(4, budget // 4)]),
                   "recent": recent, "order_free": order_free}


def _lengths(most, spread, batch, least=1):
    """Lengths in (most * (1 - spread), most], the same for every seed; the first is `most`."""
    return [max(least, int(round(most * (1.0 - spread * ((b * 0.6180339887) % 1.0))))) for b in range(batch)]


def _shape(case):
    """The lengths that a case's numbers stand for, and its pool."""
    batch, page = case["batch"], case["page"]
    s = {}
    if case["op"] in ("store", "weigh"):
        s["lens"] = _lengths(case["tokens"], case["spread"], batch)
        if case.get("empty"):
            s["lens"][1] = 0
        s["first"] = _lengths(case["context"], case["spread"], batch, 0) if case["context"] else [0] * batch
        s["total"] = sum(s["lens"])
        s["slots"] = [a + b for a, b in zip(s["lens"], s["first"])]
    else:
        s["lens"] = _lengths(case["length"], case["spread"], batch)
        if case.get("empty"):  # sequences that have ended keep their place in the batch
            for b in range(1, batch, 7):
                s["lens"][b] = 0
        s["slots"] = s["lens"]
    most = max(s["slots"]) + 16
    s["page_size"] = page or max(most, case.get("budget", 0) + 1)
    s["per_seq"] = -(-most // page) if page else 1
    s["used"] = [-(-(n + 1) // page) for n in s["slots"]] if page else [1] * batch  # room for the next token too
    s["pages"] = sum(s["used"]) + 7 if page else batch
    return s


def _normal(shape, gen):
    return torch.randn(shape, device="cuda", generator=gen, dtype=torch.float32)


def _pool(shape, gen):
    return torch.empty(shape, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)


def _centres():
    c = torch.from_numpy(np.random.RandomState(6).standard_normal((6, D)).astype(np.float32)).cuda()
    return c / c.norm(dim=1, keepdim=True) * math.sqrt(D) * 0.5


def _queries(tokens, heads, gen):
    """Nine in ten of unit variance with log-normal norms, one in ten aligned to one of six centres (as some keys are)."""
    q = _normal((tokens, heads, D), gen) * torch.exp(0.25 * _normal((tokens, heads, 1), gen))
    far = torch.rand((tokens, heads, 1), device="cuda", generator=gen) < 0.1
    which = torch.randint(0, 6, (tokens, heads), device="cuda", generator=gen)
    return torch.where(far, _centres()[which], q).to(torch.bfloat16)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(s, batch, rs):
    """Pages of the pool in random order; entries behind a sequence's last page are -1."""
    order, at = rs.permutation(s["pages"]), 0
    table = np.full((batch, s["per_seq"]), -1, np.int32)
    for b in range(batch):
        table[b, :s["used"][b]] = order[at:at + s["used"][b]]
        at += s["used"][b]
    return torch.from_numpy(table).cuda()


def _view(pool, s, table, batch, length):
    """The first `length` slots of every sequence, [batch][kv_heads][length][...], from the pool's pages."""
    if table is None:
        return pool[:, :, :length]
    n = -(-length // s["page_size"])
    x = pool[table[:, :n].clamp(min=0).long()].transpose(1, 2)
    return x.reshape((batch, pool.shape[1], n * s["page_size"]) + tuple(pool.shape[3:]))[:, :, :length]


def _rows(s, table, b, slot):
    """Page and place in it of slots `slot` of sequences `b`."""
    if table is None:
        return b, slot
    page = slot // s["page_size"]
    return table[b, page].long(), slot - page * s["page_size"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    s, op, batch, heads, kv = _shape(case), case["op"], case["batch"], case["heads"], case["kv_heads"]
    state = {"case": case, "shape": s, "stream": torch.cuda.current_stream()}
    state["table"] = table = _table(s, batch, rs) if case["page"] else None
    pool = (s["pages"], kv, s["page_size"], D)
    if op == "evict":
        pool = (case["layers"],) + pool
    state["K"] = K = _pool(pool, gen)
    if op != "weigh":
        state["V"] = _pool(pool, gen)
    if op in ("attend", "weigh"):  # one key in 32 near a centre that some queries seek
        near = torch.randint(0, 32 * 6, pool[:3], device="cuda", generator=gen)
        K[near < 6] = (2.0 * _centres()[near[near < 6]] + 0.1 * K[near < 6].float()).to(torch.bfloat16)
    if op in ("store", "weigh"):
        state["cu"] = _int32(np.concatenate([[0], np.cumsum(s["lens"])]).tolist())
        state["first"] = _int32(s["first"])
    else:
        state["lens"] = _int32(s["lens"])
    if op == "store":
        # a fused projection's output: queries, keys and values of a token side by side
        qkv = _normal((s["total"], heads + 2 * kv, D), gen).to(torch.bfloat16)
        state["q"], state["k"], state["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        state["pos"] = _int32([case["position"] + 3 * b for b in range(batch)])
        state["q_rot"] = torch.empty((s["total"], heads, D), dtype=torch.bfloat16, device="cuda")
    elif op == "attend":
        state["q"] = _queries(batch, heads, gen)
        state["out"] = torch.empty_like(state["q"])
        state["lse"] = torch.empty((batch, heads), dtype=torch.float32, device="cuda")
        # what earlier steps have added up
        state["weights"] = torch.exp(2.0 * _normal(pool[:3], gen) - 4.0) if case["weighed"] else None
    elif op == "weigh":
        state["q"] = _queries(s["total"], heads, gen)
        state["weights"] = torch.exp(2.0 * _normal(pool[:3], gen) - 4.0)
        state["lse"] = torch.cat([_row_lse(state, b) for b in range(batch)])
    else:
        # heavy-tailed, as accumulated weights are; one slot in twenty never received any
        w = torch.exp(2.0 * _normal(pool[:4], gen) - 4.0)
        state["weights"] = torch.where(torch.rand(pool[:4], device="cuda", generator=gen) < 0.05, torch.zeros_like(w), w)
        state["kept"] = torch.empty((case["layers"], batch, kv, case["budget"]), dtype=torch.int32, device="cuda")
        state["left"] = torch.empty(batch, dtype=torch.int32, device="cuda")
        state["layers"] = [list(state[x]) for x in ("K", "V", "weights")]
    if own:
        from kv_cache_eviction_head_gb300 import bkv
        flags = bkv.BKV_FLAG_ORDER_FREE if case.get("order_free") else 0
        budget, prefix, recent = (case.get(x, d) for x, d in (("budget", 1), ("prefix", 0), ("recent", 0)))
        state["cfg"] = bkv.make_config(heads=heads, kv_heads=kv, d=D, budget=budget, period=16, prefix=prefix, recent=recent,
                                       layers=case.get("layers", 1), batch=batch, max_cache=max(s["page_size"] * s["per_seq"], budget + 1),
                                       rope_theta=case.get("theta", 1e6), flags=flags)
        if op == "store":
            state["rope"] = bkv.make_rope(theta=case["theta"], rotary_dim=case["rotary"], interleaved=case["interleaved"],
                                          scaling=case["scaling"], factor=case["factor"], original_len=8192)
        if op == "attend":
            n = bkv.bkv_attend_paged_bytes(state["cfg"], state["K"], table, weighed=case["weighed"])
            state["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return state


def _visible_logits(state, b):
    """Scaled logits of sequence b's rows, [H][n][slots] in 32 bits, -inf where a row cannot see a slot."""
    case, s = state["case"], state["shape"]
    n, f, H, kv = s["lens"][b], s["first"][b], case["heads"], case["kv_heads"]
    at = sum(s["lens"][:b])
    table = None if state["table"] is None else state["table"][b:b + 1]
    K = _view(state["K"] if table is not None else state["K"][b:b + 1], s, table, 1, f + n)[0].float()
    q = state["q"][at:at + n].float().permute(1, 0, 2).reshape(kv, H // kv * n, D)
    w = torch.matmul(q, K.transpose(1, 2)).mul_(1.0 / math.sqrt(D)).view(H, n, f + n)
    see = torch.arange(f + n, device="cuda")[None] <= f + torch.arange(n, device="cuda")[:, None]
    return w.masked_fill_(~see, -math.inf)


def _row_lse(state, b):
    """ln of every row's sum of exponentials, [n][H], as the prompt's attention leaves it."""
    if not state["shape"]["lens"][b]:
        return torch.empty((0, state["case"]["heads"]), device="cuda")
    w = _visible_logits(state, b)
    m = w.amax(dim=2, keepdim=True)
    return (m[..., 0] + torch.log(w.sub_(m).exp_().sum(dim=2))).t()


def _frequencies(case):
    """Radians per position of every pair, and what cosines and sines are multiplied by, in 64 bits."""
    r, theta, f = case["rotary"], case["theta"], case["factor"]
    i = torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r
    if case["scaling"] == "ntk":
        theta = theta * f ** (r / (r - 2))
    freq = torch.pow(torch.tensor(theta, dtype=torch.float64, device="cuda"), -i)
    if case["scaling"] == "linear":
        freq = freq / f
    if case["scaling"] != "yarn":
        return freq, 1.0
    keep = ((8192 * freq / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)  # 1: turns often enough in 8192 tokens to stay as it is
    return freq * (keep + (1.0 - keep) / f), 0.1 * math.log(f) + 1.0


def _run_store(state):
    case, s = state["case"], state["shape"]
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(state["cu"][1:], t, right=True)
    i = t - state["cu"][b]
    freq, scale = _frequencies(case)
    angle = (state["pos"][b].long() + i).double()[:, None] * freq  # in 64 bits: far positions
    cos, sin = (torch.cos(angle) * scale).float()[:, None], (torch.sin(angle) * scale).float()[:, None]
    r = case["rotary"]

    def rotate(x):
        x, rest = x[..., :r].float(), x[..., r:]
        if case["interleaved"]:
            a, c = x[..., 0::2], x[..., 1::2]
            y = torch.stack([a * cos - c * sin, c * cos + a * sin], dim=-1).flatten(-2)
        else:
            a, c = x[..., :r // 2], x[..., r // 2:]
            y = torch.cat([a * cos - c * sin, c * cos + a * sin], dim=-1)
        return torch.cat([y.to(torch.bfloat16), rest], dim=-1)

    state["q_rot"].copy_(rotate(state["q"]))
    page, at = _rows(s, state["table"], b, state["first"][b].long() + i)
    state["K"][page, :, at] = rotate(state["k"])
    state["V"][page, :, at] = state["v"]
    return state["q_rot"], state["K"], state["V"]


def _run_attend(state):
    case, s = state["case"], state["shape"]
    B, H, kv, L = case["batch"], case["heads"], case["kv_heads"], max(s["lens"])
    K, V = (_view(state[x], s, state["table"], B, L).float() for x in ("K", "V"))
    seen = torch.arange(L, device="cuda") < state["lens"][:, None]
    V = V.masked_fill(~seen[:, None, :, None], 0.0)
    w = torch.matmul(state["q"].float().view(B, kv, H // kv, D), K.transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    w.masked_fill_(~seen[:, None, None], -math.inf)
    m = w.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    w.sub_(m).exp_()
    total = w.sum(dim=-1, keepdim=True)
    w = w / torch.where(total == 0, torch.ones_like(total), total)
    state["out"].copy_(torch.matmul(w, V).reshape(B, H, D))
    state["lse"].copy_((m + torch.log(total)).reshape(B, H))
    if not case["weighed"]:
        return state["out"], state["lse"]
    b, j = torch.nonzero(seen, as_tuple=True)
    page, at = _rows(s, state["table"], b, j)
    old = state["weights"][page, :, at] * case["decay"]
    old[j == state["lens"][b] - 1] = 0.0  # the new token's slot has no account yet
    state["weights"][page, :, at] = old + w.sum(dim=2)[b, :, j]
    return state["out"], state["lse"], state["weights"]


def _run_weigh(state):
    case, s = state["case"], state["shape"]
    kv, G = case["kv_heads"], case["heads"] // case["kv_heads"]
    cu = np.concatenate([[0], np.cumsum(s["lens"])]).tolist()
    for b in range(case["batch"]):
        n, f = s["lens"][b], s["first"][b]
        if not n:
            continue
        w = _visible_logits(state, b).sub_(state["lse"][cu[b]:cu[b + 1]].t()[:, :, None]).exp_()
        j = torch.arange(f + n, device="cuda")
        page, at = _rows(s, state["table"], torch.full_like(j, b), j)
        old = state["weights"][page, :, at] * case["decay"]
        old[f:] = 0.0  # these slots' tokens are the call's own
        state["weights"][page, :, at] = old + w.view(kv, G * n, f + n).sum(dim=1).t()
    return state["weights"]


def _run_evict(state):
    case, s = state["case"], state["shape"]
    layers, B, kv, budget = case["layers"], case["batch"], case["kv_heads"], case["budget"]
    L = max(max(s["lens"]), budget)
    lens = state["lens"].long()
    slot = torch.arange(L, device="cuda")
    table = state["table"]
    if table is None:
        w = state["weights"][..., :L]
    else:
        n = -(-L // s["page_size"])
        idx = table[:, torch.arange(n, device="cuda").clamp(max=table.shape[1] - 1)].clamp(min=0).long()
        w = state["weights"][:, idx].transpose(2, 3).reshape(layers, B, kv, n * s["page_size"])[..., :L]
    forced = (slot < case["prefix"]) | ((slot >= lens[:, None] - case["recent"]) & (slot < lens[:, None]))
    key = torch.where(forced[:, None], torch.full_like(w, math.inf), w)
    key = torch.where((slot < lens[:, None])[:, None], key, torch.full_like(w, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices  # ties: the lowest slot first
    keep = torch.zeros(key.shape, dtype=torch.bool, device="cuda").scatter_(-1, order[..., :budget], True)
    if case["order_free"]:  # kept slots below the budget stay, the holes take the kept slots behind it
        hole = ~keep[..., :budget]
        tail = torch.sort(torch.where(keep[..., budget:], slot[budget:], L), dim=-1).values
        tail = torch.cat([tail, torch.zeros_like(tail[..., :1])], dim=-1)
        rank = (torch.cumsum(hole, dim=-1) - 1).clamp(0, tail.shape[-1] - 1)
        kept = torch.where(hole, torch.gather(tail, -1, rank), slot[:budget])
    else:
        kept = torch.sort(order[..., :budget], dim=-1).values
    live = slot[:budget] < lens[:, None]  # sequences within the budget keep all they have
    state["kept"].copy_(torch.where(live[:, None], kept, -1))
    l, b, h, i = torch.nonzero((live[:, None] & (kept != slot[:budget])), as_tuple=True)
    page, at = _rows(s, table, b, kept[l, b, h, i])
    to_page, to = _rows(s, table, b, i)
    for pool in (state["K"], state["V"], state["weights"]):
        pool[l, to_page, h, to] = pool[l, page, h, at]
    state["left"].copy_(torch.clamp(state["lens"], max=budget))
    return state["K"], state["V"], state["weights"], state["kept"], state["left"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"store": _run_store, "attend": _run_attend, "weigh": _run_weigh, "evict": _run_evict}[op](s)
    from kv_cache_eviction_head_gb300 import bkv
    if op == "store":
        bkv.bkv_store_paged(s["cfg"], s["rope"], s["q"], s["k"], s["v"], s["cu"], s["first"], s["pos"], s["q_rot"], s["K"], s["V"],
                            table=s["table"], stream=s["stream"])
        return s["q_rot"], s["K"], s["V"]
    if op == "attend":
        bkv.bkv_attend_paged(s["cfg"], s["q"], s["K"], s["V"], s["lens"], s["out"], s["workspace"], table=s["table"], lse=s["lse"],
                             weights=s["weights"], decay=s["case"]["decay"], stream=s["stream"])
        return (s["out"], s["lse"]) if s["weights"] is None else (s["out"], s["lse"], s["weights"])
    if op == "weigh":
        bkv.bkv_weigh_prompt(s["cfg"], s["q"], s["lse"], s["K"], s["cu"], s["first"], s["weights"], table=s["table"],
                             decay=s["case"]["decay"], stream=s["stream"])
        return s["weights"]
    K, V, weights = s["layers"]
    bkv.bkv_evict_weight(s["cfg"], K, V, weights, s["lens"], s["kept"], table=s["table"], new_lens=s["left"], stream=s["stream"])
    return s["K"], s["V"], s["weights"], s["kept"], s["left"]


def work(case):
    s, heads, kv = _shape(case), case["heads"], case["kv_heads"]
    row = D * 2
    if case["op"] == "store":
        return {"bytes": 2 * s["total"] * (heads + 2 * kv) * row, "flops": 3 * case["rotary"] * s["total"] * (heads + kv)}
    if case["op"] == "attend":
        slots = sum(s["lens"])
        account = (8 if case["decay"] else 4) if case["weighed"] else 0  # read (unless it starts anew) and written
        return {"bytes": slots * kv * (2 * row + account) + case["batch"] * heads * (2 * row + 4), "flops": 4 * D * heads * slots}
    if case["op"] == "weigh":
        pairs = sum(n * f + n * (n + 1) // 2 for n, f in zip(s["lens"], s["first"]))
        slots = sum(n + f for n, f in zip(s["lens"], s["first"]) if n)
        return {"bytes": s["total"] * heads * (row + 4) + slots * kv * (row + 4), "flops": 2 * D * heads * pairs}
    # dropped slots lie anywhere between prefix and recent window: in slot order all behind the first of them move,
    # order-free the dropped ones below the budget are filled
    units, moved, read = case["layers"] * kv, 0.0, 0
    for n in s["lens"]:
        drop, among = n - case["budget"], n - case["prefix"] - case["recent"]
        read += n
        if drop > 0:
            if case["order_free"]:
                moved += drop * max(0, case["budget"] - case["prefix"]) / max(1, among)
            else:
                moved += max(0.0, case["budget"] - case["prefix"] - among / (drop + 1))
    return {"bytes": units * (4 * read + 4 * case["budget"] * case["batch"] + moved * (2 * 2 * row + 8)), "flops": 0}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence."""
    state = prepare(case, seed)
    s, B, H, kv = state["shape"], case["batch"], case["heads"], case["kv_heads"]
    G, op, ps, table = H // kv, case["op"], s["page_size"], state["table"]

    def rows_of(b, n):
        """Pages and places of the first n slots of sequence b."""
        j = np.arange(n)
        if table is None:
            return torch.full((n,), b, device="cuda"), torch.from_numpy(j).cuda()
        return torch.from_numpy(table[b].cpu().numpy()[j // ps].astype(np.int64)).cuda(), torch.from_numpy(j % ps).cuda()

    if op == "store":
        r = case["rotary"]
        theta, f = case["theta"], case["factor"]
        freq, scale = [], 1.0
        for i in range(r // 2):
            w = theta ** (-2.0 * i / r)
            if case["scaling"] == "linear":
                w /= f
            elif case["scaling"] == "ntk":
                w = (theta * f ** (r / (r - 2.0))) ** (-2.0 * i / r)
            elif case["scaling"] == "yarn":
                g = min(1.0, max(0.0, (8192 * w / (2 * math.pi) - 1.0) / (32.0 - 1.0)))
                w, scale = (1.0 - g) * w / f + g * w, 1.0 + 0.1 * math.log(f)
            freq.append(w)
        freq = torch.tensor(freq, dtype=torch.float64, device="cuda")
        K, V = state["K"].double(), state["V"].double()
        Q = state["q"].double()
        at = 0
        for b, n in enumerate(s["lens"]):
            first = s["first"][b]
            pos = torch.arange(n, dtype=torch.float64, device="cuda") + float(state["pos"][b])
            z = torch.polar(torch.full((), scale, dtype=torch.float64, device="cuda"), pos[:, None, None] * freq)
            page, place = (x[first:] for x in rows_of(b, first + n))
            for x, key in ((state["q"], False), (state["k"], True)):
                y = x[at:at + n].double().contiguous()
                if case["interleaved"]:
                    t = torch.view_as_complex(y[..., :r].reshape(n, -1, r // 2, 2).contiguous()) * z
                    y[..., :r] = torch.view_as_real(t).reshape(n, -1, r)
                else:
                    t = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * z
                    y[..., :r // 2], y[..., r // 2:r] = t.real, t.imag
                if key:
                    K[page, :, place] = y
                else:
                    Q[at:at + n] = y
            V[page, :, place] = state["v"][at:at + n].double()
            at += n
        return Q, K, V
    if op == "attend":
        out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
        weights = state["weights"].double() if case["weighed"] else None
        for b, n in enumerate(s["lens"]):
            if not n:
                continue
            page, place = rows_of(b, n)
            k, v = state["K"][page, :, place].double(), state["V"][page, :, place].double()  # [n][kv][d]
            logits = torch.einsum("hgd,nhd->hgn", state["q"][b].double().view(kv, G, D), k) / math.sqrt(D)
            lse[b] = torch.logsumexp(logits, dim=-1).view(H)
            p = torch.softmax(logits, dim=-1)
            out[b] = torch.einsum("hgn,nhd->hgd", p, v).reshape(H, D)
            if weights is not None:
                before = weights[page, :, place] * case["decay"]
                before[n - 1] = 0
                weights[page, :, place] = before + p.sum(dim=1).t()
        return (out, lse) if weights is None else (out, lse, weights)
    if op == "weigh":
        weights = state["weights"].double()
        at = 0
        for b, n in enumerate(s["lens"]):
            f = s["first"][b]
            if not n:
                continue
            page, place = rows_of(b, f + n)
            hidden = torch.ones((n, f + n), dtype=torch.bool, device="cuda").triu(f + 1)
            total = torch.zeros((kv, f + n), dtype=torch.float64, device="cuda")
            for h in range(H):
                k = state["K"][page, h // G, place].double()
                logits = state["q"][at:at + n, h].double() @ k.t() / math.sqrt(D) - state["lse"][at:at + n, h].double()[:, None]
                total[h // G] += torch.exp(logits.masked_fill_(hidden, -math.inf)).sum(dim=0)
            before = weights[page, :, place] * case["decay"]
            before[f:] = 0
            weights[page, :, place] = before + total.t()
            at += n
        return weights
    layers, budget, prefix, recent = case["layers"], case["budget"], case["prefix"], case["recent"]
    kept = np.full((layers, B, kv, budget), -1, np.int64)
    for b, n in enumerate(s["lens"]):
        page, place = rows_of(b, n)
        w = state["weights"][:, page, :, place].permute(1, 2, 0).cpu().numpy()  # [layers][kv][n]
        for l in range(layers):
            for h in range(kv):
                if n <= budget:
                    kept[l, b, h, :n] = np.arange(n)
                    continue
                middle = np.arange(prefix, n - recent)
                best = middle[np.lexsort((middle, -w[l, h, middle].astype(np.float64)))][:budget - prefix - recent]
                chosen = np.sort(np.concatenate([np.arange(prefix), best, np.arange(n - recent, n)]))
                if case["order_free"]:
                    layout = np.arange(budget)
                    layout[np.setdiff1d(layout, chosen)] = chosen[chosen >= budget]
                    chosen = layout
                kept[l, b, h] = chosen
    K, V, W = (state[x].clone() for x in ("K", "V", "weights"))
    for l in range(layers):
        for b, n in enumerate(s["lens"]):
            if n > budget:
                page, place = rows_of(b, n)
                i = torch.from_numpy(kept[l, b]).cuda()  # [kv][budget]
                h = torch.arange(kv, device="cuda")[:, None]
                for new, old in ((K, state["K"]), (V, state["V"]), (W, state["weights"])):
                    new[l, page[:budget], h, place[:budget]] = old[l, page[i], h, place[i]]
    return K.double(), V.double(), W.double(), torch.from_numpy(kept.astype(np.int32)).cuda(), _int32([min(n, budget) for n in s["lens"]])
