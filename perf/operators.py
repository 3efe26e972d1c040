"""Operators around the verify step, as they are measured: the selection of
beams over the vocabulary, the reordering of the beams' states, the block
tables and slot maps of a paged cache, and the move of an accepted path's
states into that cache.

Where `own` is false `run` computes the plain forms (elementary torch
operations, 64 bits where values are compared); where it is true it makes the
calls a user's program makes.  `exact` states the same results from their
definitions.
"""
import numpy as np
import torch

own = False

DEV = "cuda"
_kept = {}  # the verifier a user's program keeps between calls


def listed():
    return [
        # One step of beam search or draft-tree expansion over the tiny vocabulary of the first verify
        # configuration: latency is all that counts.
        {"name": "beams tiny f32", "op": "beams", "B": 4, "W": 4, "K": 4, "V": 1000, "dtype": "f32", "pad": 0,
         "masked": False, "finished": False, "first": False},
        # A level of a draft tree for a small batch (8 branches kept of 4 beams), Llama-3 vocabulary.
        {"name": "beams draft level bf16", "op": "beams", "B": 16, "W": 4, "K": 8, "V": 128256, "dtype": "bf16", "pad": 0,
         "masked": False, "finished": False, "first": False},
        # Beam search of a large batch, 8 beams each, Llama-3 vocabulary: one long read.
        {"name": "beams large bf16", "op": "beams", "B": 64, "W": 8, "K": 8, "V": 128256, "dtype": "bf16", "pad": 0,
         "masked": False, "finished": False, "first": False},
        # Beam search with grammar masks and finished hypotheses, twice as many candidates as beams, Qwen
        # vocabulary with rows of odd length (unaligned rows).
        {"name": "beams masked f32 odd", "op": "beams", "B": 8, "W": 5, "K": 10, "V": 151935, "dtype": "f32", "pad": 0,
         "masked": True, "finished": True, "first": False},
        # Beam states of a short sequence: 4 layers' keys and values, out of place.
        {"name": "reorder short", "op": "reorder", "G": 8, "B": 4, "W": 4, "T": 64, "D": 256, "dtype": "bf16",
         "heads": 0, "inplace": False},
        # Beam states of long ragged sequences, out of place: a long copy.
        {"name": "reorder long", "op": "reorder", "G": 16, "B": 8, "W": 8, "T": 1024, "D": 512, "dtype": "bf16",
         "heads": 0, "inplace": False},
        # Heads before positions, odd sizes, fp32, in place (survivors keep their beam, the others are overwritten).
        {"name": "reorder heads in place", "op": "reorder", "G": 6, "B": 5, "W": 5, "T": 333, "D": 80, "dtype": "f32",
         "heads": 7, "inplace": True},
        # A decode step of the Llama-3 verify batch: 64 requests, 5 drafts, pages of 16.
        {"name": "slots decode", "op": "slots", "B": 64, "k": 5, "ragged": False, "block": 16, "max_len": 4000},
        # Thousands of requests with draft counts of their own.
        {"name": "slots ragged", "op": "slots", "B": 4096, "k": 8, "ragged": True, "block": 16, "max_len": 2000},
        # The accepted paths of the 64-node draft trees of 16 requests, 16 layers' keys and values.
        {"name": "path tree", "op": "path", "G": 32, "B": 16, "N": 64, "depth": 6, "D": 1024, "dtype": "bf16",
         "slots": 4096},
        # A large batch of small trees, fp32 rows of odd length.
        {"name": "path large f32", "op": "path", "G": 8, "B": 256, "N": 24, "depth": 8, "D": 250, "dtype": "f32",
         "slots": 20000},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["beams", "beams", "reorder", "slots", "path"])
    if op == "beams":
        while True:
            c = {"op": op, "B": _log_int(rng, 1, 64), "W": _log_int(rng, 1, 16), "K": _log_int(rng, 1, 32),
                 "V": _log_int(rng, 60, 152000), "dtype": rng.choice(["bf16", "f32"]), "pad": rng.choice([0, 0, 1, 8]),
                 "masked": rng.random() < 0.3, "finished": rng.random() < 0.3, "first": rng.random() < 0.15}
            if c["B"] * c["W"] * c["V"] * _size(c["dtype"]) <= 120e6:
                return c
    if op == "reorder":
        while True:
            heads = rng.choice([0, 0, 2, 7])
            c = {"op": op, "G": _log_int(rng, 1, 32), "B": _log_int(rng, 1, 16), "W": _log_int(rng, 1, 16),
                 "T": _log_int(rng, 1, 1500), "D": _log_int(rng, 16, 1024), "dtype": rng.choice(["bf16", "f32"]),
                 "heads": heads, "inplace": rng.random() < 0.4}
            if c["G"] * max(1, heads) * c["B"] * c["W"] * c["T"] * c["D"] * _size(c["dtype"]) <= 0.9e9:
                return c
    if op == "slots":
        return {"op": op, "B": _log_int(rng, 1, 4096), "k": _log_int(rng, 1, 32), "ragged": rng.random() < 0.5,
                "block": rng.choice([1, 8, 16, 32, 48, 64]), "max_len": _log_int(rng, 10, 2000)}
    c = {"op": op, "G": _log_int(rng, 1, 32), "B": _log_int(rng, 1, 128), "N": _log_int(rng, 2, 80),
         "depth": rng.randint(1, 10), "D": _log_int(rng, 16, 1024), "dtype": rng.choice(["bf16", "f32"])}
    c["slots"] = c["B"] * (c["depth"] + 1) + _log_int(rng, 100, 2000)
    return c


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _type(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(int(seed))
    return {"beams": _beams_state, "reorder": _reorder_state, "slots": _slots_state, "path": _path_state}[case["op"]](
        case, g)


def _rand(shape, g):
    return torch.rand(shape, generator=g, device=DEV)


def _ints(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _beams_state(c, g):
    """Logits N(0, 2^2) with one planted token a row (+8), cumulative log probabilities in descending order."""
    B, W, V = c["B"], c["W"], c["V"]
    x = torch.randn((B, W, V), generator=g, device=DEV).mul_(2.0)
    x.scatter_add_(2, torch.randint(0, V, (B, W, 1), generator=g, device=DEV), torch.full((B, W, 1), 8.0, device=DEV))
    if c["masked"]:  # a grammar allows 70 % of the tokens
        x.masked_fill_(_rand((B, 1, V), g) < 0.3, float("-inf"))
    rows = torch.zeros((B, W, V + c["pad"]), device=DEV, dtype=_type(c["dtype"]))
    rows[..., :V] = x.to(rows.dtype)
    scores = -torch.cumsum(_rand((B, W), g) * 1.5, 1)
    if c["first"]:  # the first step of a search: only beam 0 holds a hypothesis
        scores[:, 1:] = float("-inf")
    done = (_rand((B, W), g) < 0.3).to(torch.int32) if c["finished"] else None
    K = c["K"]
    out = (torch.empty(B, K, device=DEV), torch.empty(B, K, device=DEV, dtype=torch.int32),
           torch.empty(B, K, device=DEV, dtype=torch.int32))
    return {"op": "beams", "logits": rows[..., :V], "scores": scores, "K": K, "finished": done, "eos": 2, "out": out}


def _reorder_state(c, g):
    G, B, W, T, D, H = c["G"], c["B"], c["W"], c["T"], c["D"], c["heads"]
    dt = _type(c["dtype"])
    shape = (G, B, W, H, T, D) if H else (G, B, W, T, D)  # heads before positions, or positions first
    states = torch.randn(shape, generator=g, device=DEV, dtype=dt)
    parents = _ints(0, W, (B, W), g)
    if c["inplace"]:  # the parent of a parent is itself: survivors keep their beam
        for _ in range(5):
            parents = torch.gather(parents, 1, parents.long())
        fixed = torch.zeros_like(parents).scatter_(1, parents.long(), 1)
        ids = torch.arange(W, device=DEV, dtype=torch.int32).expand(B, W)
        parents = torch.where(fixed.bool(), ids, parents)
    lengths = (T * (0.25 + 0.75 * _rand((B,), g))).ceil().clamp(1, T).to(torch.int32)
    return {"op": "reorder", "states": states, "parents": parents, "lengths": lengths,
            "time_dim": 4 if H else 3,
            "out": None if c["inplace"] else torch.randn(shape, generator=g, device=DEV, dtype=dt)}


def _slots_state(c, g):
    B, k, bs = c["B"], c["k"], c["block"]
    lens = _ints(1, c["max_len"] + 1, (B,), g)
    accept = _ints(0, k + 1, (B,), g)
    release = (_rand((B,), g) < 0.02).to(torch.int32)
    held = (lens + bs - 1) // bs
    cols = (c["max_len"] + 2 * (k + 1) + bs - 1) // bs + 1
    blocks = B * cols
    perm = torch.randperm(blocks, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    start = torch.cumsum(held, 0) - held
    col = torch.arange(cols, device=DEV, dtype=torch.int32)
    mine = col[None, :] < held[:, None]
    tables = torch.where(mine, perm[(start[:, None] + col).clamp(max=blocks - 1).long()], torch.full_like(col, -1))
    used = int(held.sum())
    head = int(torch.randint(0, blocks, (1,), generator=g, device=DEV))
    ring = torch.full((blocks,), -1, device=DEV, dtype=torch.int32)
    ring[(head + torch.arange(blocks - used, device=DEV)) % blocks] = perm[used:]
    if c["ragged"]:  # every count from 0 to k, in an order of the seed's
        counts = torch.arange(B, device=DEV) % (k + 1)
        total = int(counts.sum())
        offsets = torch.zeros(B + 1, device=DEV, dtype=torch.int32)
        offsets[1:] = torch.cumsum(counts[torch.randperm(B, generator=g, device=DEV)], 0)
    else:
        offsets, total = None, B * k
    rows = B + total
    i32 = dict(device=DEV, dtype=torch.int32)
    out = (torch.empty(B, **i32), torch.empty(B, **i32), torch.empty(2, **i32),
           torch.empty(rows, device=DEV, dtype=torch.int64), torch.empty(rows, device=DEV, dtype=torch.int64))
    return {"op": "slots", "lens": lens, "accept": accept, "release": release, "held": held.to(torch.int32),
            "tables": tables.contiguous(), "ring": ring, "ring_state": torch.tensor([head, blocks - used], **i32),
            "block": bs, "k": k, "offsets": offsets, "total": total, "out": out}


def _path_state(c, g):
    G, B, N, depth, D = c["G"], c["B"], c["N"], c["depth"], c["D"]
    dt = _type(c["dtype"])
    src = torch.randn((G, B, N + 1, D), generator=g, device=DEV, dtype=dt)
    cache = torch.randn((G, c["slots"], D), generator=g, device=DEV, dtype=dt)
    most = min(depth, N)
    al = _ints(0, most + 1, (B,), g)
    order = torch.argsort(_rand((B, N), g), 1)[:, :most].sort(1).values.to(torch.int32) + 1  # ascending node indices
    nodes = torch.full((B, depth), -1, device=DEV, dtype=torch.int32)
    nodes[:, :most] = order
    nodes = torch.where(torch.arange(depth, device=DEV) < al[:, None], nodes, torch.full_like(nodes, -1))
    slots = torch.randperm(c["slots"], generator=g, device=DEV)[:B * (depth + 1)].reshape(B, depth + 1)
    return {"op": "path", "src": src, "cache": cache, "accept_len": al, "nodes": nodes.contiguous(),
            "slots": slots.contiguous()}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"beams": _beams_plain, "reorder": _reorder_plain, "slots": _slots_plain, "path": _path_plain}[state["op"]](
        state)


def _run_own(s):
    import speculative_decoding_draft_decode_b200 as sd
    if s["op"] == "beams":
        ver = _kept.get("verifier")
        if ver is None:
            ver = _kept["verifier"] = sd.Verifier(torch.device("cuda", torch.cuda.current_device()))
        return ver.beam_select(s["logits"], s["scores"], s["K"], finished=s["finished"], eos_token=s["eos"], out=s["out"])
    if s["op"] == "reorder":
        return sd.reorder_states(s["states"], s["parents"], lengths=s["lengths"], time_dim=s["time_dim"], out=s["out"])
    if s["op"] == "slots":
        got = sd.plan_slots(s["lens"], s["tables"], s["held"], s["ring"], s["ring_state"], s["block"], k=s["k"],
                            draft_offsets=s["offsets"], total_drafts=s["total"], accept_len=s["accept"],
                            release=s["release"], out=s["out"])
        return (*got, s["tables"], s["ring"])
    return sd.commit_path(s["src"], s["accept_len"], s["nodes"], s["cache"], s["slots"])


def _beams_plain(s):
    """log softmax + score in 64 bits; a row's K best by (value, lowest index), then the K best of the rows'."""
    x, K, done = s["logits"], s["K"], s["finished"]
    B, W, V = x.shape
    d = x.double()
    m = d.amax(2, keepdim=True)
    lse = (m + torch.log(torch.exp(d - m).sum(2, keepdim=True))).squeeze(2)
    bits = (x.float() + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    order = (order << 32) | (0xFFFFFFFF - torch.arange(V, device=x.device))
    best = torch.topk(order, min(K, V), dim=2).values
    token = 0xFFFFFFFF - (best & 0xFFFFFFFF)
    cand = (s["scores"].double() - lse)[..., None] + torch.gather(d, 2, token)
    if done is not None:  # a finished beam goes on as itself, with the end token
        is_done = done.bool()[..., None]
        firsts = torch.arange(cand.shape[2], device=x.device) == 0
        only = torch.where(firsts, s["scores"].double()[..., None], float("-inf"))
        cand = torch.where(is_done, only, cand)
        token = torch.where(is_done, s["eos"], token)
    cand = torch.where(s["scores"][..., None] == float("-inf"), float("-inf"), cand)
    flat = cand.flatten(1)
    if flat.shape[1] < K:
        flat = torch.cat([flat, flat.new_full((B, K - flat.shape[1]), float("-inf"))], 1)
    value, at = torch.sort(flat, dim=1, descending=True, stable=True)
    value, at = value[:, :K], at[:, :K]
    real = value > float("-inf")
    parent = torch.where(real, at // cand.shape[2], -1).to(torch.int32)
    token = torch.gather(token.flatten(1), 1, at.clamp(max=token[0].numel() - 1))
    return value.float(), parent, torch.where(real, token, -1).to(torch.int32)


def _reorder_plain(s):
    x, parents, lengths = s["states"], s["parents"], s["lengths"]
    to = x if s["out"] is None else s["out"]
    moved = x[:, torch.arange(x.shape[1], device=x.device)[:, None], parents.long()]
    valid = torch.arange(x.shape[-2], device=x.device) < lengths[:, None]
    valid = valid[None, :, None, :, None] if x.dim() == 5 else valid[None, :, None, None, :, None]
    return to.copy_(torch.where(valid, moved, to))


def _slots_plain(s):
    bs, ring, tables = s["block"], s["ring"], s["tables"]
    dev, (B, cols), cap = ring.device, tables.shape, ring.numel()
    gone = s["release"] != 0
    if s["offsets"] is None:
        n = torch.full((B,), s["k"] + 1, device=dev)
    else:
        n = (s["offsets"][1:] - s["offsets"][:-1] + 1).long()
    lens = torch.where(gone, 0, s["lens"].long() + s["accept"] + 1)
    held = s["held"].long()
    need = (lens + n + bs - 1) // bs
    grow = torch.where(gone | (need > cols), 0, (need - held).clamp(min=0))
    upto = torch.cumsum(grow, 0)
    head, count = s["ring_state"][0].long(), s["ring_state"][1].long()
    got = torch.where(upto <= count, grow, 0)
    first = upto - grow
    col = torch.arange(cols, device=dev)
    new = col[None, :] - held[:, None]
    fresh = (new >= 0) & (new < got[:, None])
    new_tables = torch.where(fresh, ring[(head + first[:, None] + new) % cap], tables)
    back = torch.where(gone, held, 0)
    at = torch.cumsum(back, 0) - back
    ret = (col[None, :] < back[:, None])
    place = torch.where(ret, (head + count + at[:, None] + col) % cap, cap)
    new_ring = torch.cat([ring, ring[:1]]).scatter(0, place.flatten(), tables.flatten())[:cap]
    held2 = torch.where(gone, 0, held + got)
    taken = got.sum()
    state = torch.stack([(head + taken) % cap, count - taken + back.sum()]).to(torch.int32)
    rows = B + s["total"]
    req = torch.repeat_interleave(torch.arange(B, device=dev), n, output_size=rows)
    j = torch.arange(rows, device=dev) - (torch.cumsum(n, 0) - n)[req]
    pos = lens[req] + j
    page = pos // bs
    block = new_tables[req, page.clamp(max=cols - 1)].long()
    ok = (page < held2[req]) & (block >= 0) & ~gone[req]
    slots = torch.where(ok, block * bs + pos % bs, -1)
    pos = torch.where(gone[req], -1, pos)
    return lens.to(torch.int32), held2.to(torch.int32), state, pos, slots, new_tables, new_ring


def _path_plain(s):
    src, cache, nodes, slots = s["src"], s["cache"], s["nodes"], s["slots"]
    B, depth = nodes.shape
    path = torch.cat([torch.zeros_like(nodes[:, :1]), nodes], 1).long()
    kept = torch.arange(depth + 1, device=src.device) <= s["accept_len"][:, None]
    rows = src[:, torch.arange(B, device=src.device)[:, None], path.clamp(min=0)]
    cache[:, slots] = torch.where(kept[None, :, :, None], rows, cache[:, slots])
    return cache


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "beams":
        live = c["B"] * (1 if c["first"] else c["W"]) * (0.7 if c["finished"] else 1.0)
        n = live * c["V"]
        return {"bytes": n * _size(c["dtype"]) + 4.0 * c["B"] * (c["W"] * (2 if c["finished"] else 1) + 3 * c["K"]),
                "flops": 4.0 * n}
    if c["op"] == "reorder":
        row = c["G"] * max(1, c["heads"]) * c["B"] * 0.625 * c["T"] * c["D"] * _size(c["dtype"])
        W = c["W"]
        read = W * (1.0 - (1.0 - 1.0 / W) ** W)  # distinct parents of a random map
        if c["inplace"]:  # rows that move are written, their parents read
            moved = W - max(1.0, 0.4 * W) if W > 1 else 0.0
            return {"bytes": max(8.0 * c["B"] * W, row * (min(read, moved) + moved)), "flops": 0.0}
        return {"bytes": row * (read + W) + 4.0 * c["B"] * (W + 1), "flops": 0.0}
    if c["op"] == "slots":
        rows = c["B"] * (1 + (c["k"] / 2 if c["ragged"] else c["k"]))
        pages = c["B"] * (1 + (c["k"] + c["block"]) / c["block"])
        return {"bytes": 4.0 * c["B"] * 7 + 16.0 * rows + 8.0 * pages, "flops": 10.0 * rows}
    rows = c["B"] * (1 + min(c["depth"], c["N"]) / 2.0)
    return {"bytes": 2.0 * rows * c["G"] * c["D"] * _size(c["dtype"]) + 12.0 * rows, "flops": 0.0}


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"beams": _beams_exact, "reorder": _reorder_exact, "slots": _slots_exact, "path": _path_exact}[case["op"]](s)


def _beams_exact(s):
    x, K = s["logits"], s["K"]
    B, W, V = x.shape
    value = torch.full((B, K), float("-inf"), dtype=torch.float64, device=x.device)
    parent = torch.full((B, K), -1, dtype=torch.int32, device=x.device)
    token = torch.full((B, K), -1, dtype=torch.int32, device=x.device)
    for b in range(B):
        c = torch.log_softmax(x[b].to(torch.float64), 1) + s["scores"][b].to(torch.float64)[:, None]
        for w in range(W):
            if float(s["scores"][b, w]) == float("-inf"):
                c[w] = float("-inf")
            elif s["finished"] is not None and int(s["finished"][b, w]):
                c[w] = float("-inf")
                c[w, s["eos"]] = float(s["scores"][b, w])
        v, i = torch.sort(c.flatten(), descending=True, stable=True)
        n = min(K, int((v[:K] > float("-inf")).sum()))
        value[b, :n], parent[b, :n], token[b, :n] = v[:n], (i[:n] // V).int(), (i[:n] % V).int()
    return value, parent, token


def _reorder_exact(s):
    src = s["states"]
    to = (src if s["out"] is None else s["out"]).clone()
    parents, lengths = s["parents"].tolist(), s["lengths"].tolist()
    for b, row in enumerate(parents):
        for i, p in enumerate(row):
            to[:, b, i, ..., :lengths[b], :] = src[:, b, p, ..., :lengths[b], :]
    return to


def _slots_exact(s):
    lens, held = s["lens"].tolist(), s["held"].tolist()
    accept, release = s["accept"].tolist(), s["release"].tolist()
    tables, ring = s["tables"].cpu().numpy().copy(), s["ring"].cpu().numpy().copy()
    head, count = s["ring_state"].tolist()
    bs, cap, cols = s["block"], len(ring), tables.shape[1]
    B = len(lens)
    n = [s["k"] + 1] * B if s["offsets"] is None else (np.diff(s["offsets"].cpu().numpy()) + 1).tolist()
    free = [int(ring[(head + i) % cap]) for i in range(count)]
    asked = taken = returned = 0
    pos, slots, new_lens, new_held = [], [], [], []
    for b in range(B):
        if release[b]:
            for i in range(held[b]):
                ring[(head + count + returned) % cap] = tables[b, i]
                returned += 1
            new_lens.append(0)
            new_held.append(0)
            pos += [-1] * n[b]
            slots += [-1] * n[b]
            continue
        length = lens[b] + accept[b] + 1
        need = -(-(length + n[b]) // bs)
        grow = max(0, need - held[b]) if need <= cols else 0
        asked += grow
        if asked <= count:
            tables[b, held[b]:held[b] + grow] = free[taken:taken + grow]
            taken += grow
        else:
            grow = 0
        h = held[b] + grow
        for p in range(length, length + n[b]):
            pos.append(p)
            slots.append(int(tables[b, p // bs]) * bs + p % bs if p // bs < h else -1)
        new_lens.append(length)
        new_held.append(h)
    i32 = lambda v: torch.tensor(np.asarray(v, dtype=np.int32))  # noqa: E731
    return (i32(new_lens), i32(new_held), i32([(head + taken) % cap, count - taken + returned]),
            torch.tensor(pos), torch.tensor(slots), i32(tables), i32(ring))


def _path_exact(s):
    to = s["cache"].clone()
    al, nodes, slots = s["accept_len"].tolist(), s["nodes"].tolist(), s["slots"].tolist()
    for b, h in enumerate(al):
        for j in range(h + 1):
            to[:, slots[b][j]] = s["src"][:, b, 0 if j == 0 else nodes[b][j - 1]]
    return to
