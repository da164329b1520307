"""What is measured of softmax attention, its paged cache and the pages' upkeep.

Operators (see include/kda_attn.h and include/kda_pages.h):

  prompt      o_i = sum_j P_ij v_j, P = softmax_j(scale q_i . k_j) over a sequence's tokens j <= i, H heads on G heads of k and v
  prompt_bwd  its gradients
  paged       new tokens of requests: their k and v into the pages of a cache, then their attention over all of the request
  turn        pages of a serving turn: requests forked into branches, all of them grown for drafts, the drafts rolled back
  compact     the pages in use moved to the lowest numbers

`own` picks the framework's kernels; otherwise the operators run in their plain form in 32 bits.
"""
import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one long prompt of a layer with four heads per head of k and v
        {"name": "prompt long", "op": "prompt", "dtype": "bf16", "n": 1, "T": 8192, "H": 32, "G": 8, "D": 128, "packed": False},
        # a few short ragged prompts of a small layer in 32 bits, where latency counts
        {"name": "prompt ragged f32", "op": "prompt", "dtype": "f32", "n": 5, "T": 333, "H": 6, "G": 2, "D": 64, "packed": True},
        # training of the first layer: two sequences of 4096
        {"name": "prompt_bwd train", "op": "prompt_bwd", "dtype": "bf16", "n": 2, "T": 4096, "H": 32, "G": 8, "D": 128, "packed": False},
        # a small ragged training batch in 32 bits
        {"name": "prompt_bwd ragged f32", "op": "prompt_bwd", "dtype": "f32", "n": 3, "T": 517, "H": 6, "G": 2, "D": 64, "packed": True},
        # one request, one token: pure latency
        {"name": "paged one", "op": "paged", "dtype": "bf16", "n": 1, "T": 1, "ctx": 500, "H": 16, "G": 2, "D": 128, "page": 16, "packed": False},
        # a serving batch, one token each, contexts of a quarter of ctx up to all of it
        {"name": "paged batch", "op": "paged", "dtype": "bf16", "n": 64, "T": 1, "ctx": 8192, "H": 32, "G": 8, "D": 128, "page": 64, "packed": False},
        # four drafts and the token before them
        {"name": "paged drafts", "op": "paged", "dtype": "bf16", "n": 32, "T": 5, "ctx": 2001, "H": 64, "G": 8, "D": 64, "page": 32, "packed": False},
        # chunks of two long prompts, of different lengths, packed
        {"name": "paged chunk", "op": "paged", "dtype": "bf16", "n": 2, "T": 1024, "ctx": 32768, "H": 32, "G": 8, "D": 128, "page": 16, "packed": True},
        # one prompt sampled four times
        {"name": "turn one", "op": "turn", "dtype": "bf16", "n": 1, "branches": 4, "ctx": 500, "layers": 1, "G": 2, "D": 128, "page": 16, "drafts": 4},
        # a batch of prompts sampled seven times each, a pool of four layers
        {"name": "turn batch", "op": "turn", "dtype": "bf16", "n": 32, "branches": 7, "ctx": 4096, "layers": 4, "G": 8, "D": 128, "page": 32, "drafts": 5},
        # a small pool of one layer in 32 bits
        {"name": "compact small", "op": "compact", "dtype": "f32", "n": 4, "ctx": 300, "layers": 1, "G": 2, "D": 64, "page": 16, "live": 0.6},
        # a pool of four layers after many requests have left
        {"name": "compact pool", "op": "compact", "dtype": "bf16", "n": 64, "ctx": 2048, "layers": 4, "G": 8, "D": 128, "page": 32, "live": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt_bwd", "paged", "paged", "turn", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D, G = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 16, 32, 64, 128])
    if op == "turn":
        return {"op": op, "dtype": dtype, "n": _log(rng, 1, 32), "branches": rng.randint(1, 7), "ctx": _log(rng, 40, 4096), "layers": rng.randint(1, 2),
                "G": G, "D": D, "page": page, "drafts": rng.randint(1, 8)}
    if op == "compact":
        return {"op": op, "dtype": dtype, "n": _log(rng, 1, 64), "ctx": _log(rng, 40, 2048), "layers": rng.randint(1, 2),
                "G": G, "D": D, "page": page, "live": rng.choice([0.3, 0.5, 0.8])}
    H = G * rng.randint(1, 32 // G)
    while True:
        if op == "paged":
            T = rng.choice([1, 1, 2, 5, 8, _log(rng, 9, 1024)])
            case = {"op": op, "dtype": dtype, "n": _log(rng, 1, 64), "T": T, "ctx": T + _log(rng, 16, 16384), "H": H, "G": G, "D": D, "page": page,
                    "packed": T > 8 and rng.random() < 0.5}
            many = case["n"] * case["ctx"] * G * D > (1 << 28)
        else:
            packed = rng.random() < 0.5
            n = _log(rng, 1, 12)
            most = 8192 if op == "prompt" else 4096
            T = _log(rng, 64, most) if packed else max(1, _log(rng, 64, most) // n)
            case = {"op": op, "dtype": dtype, "n": n, "T": T, "H": H, "G": G, "D": D, "packed": packed}
            many = False
        if not many and work(case)["flops"] * (16 if dtype == "f32" else 1) < 4e11:
            return case


def _es(case):
    return 2 if case["dtype"] == "bf16" else 4


def _shape(case):
    """A page of the pool: all layers' k and v."""
    return (case["layers"], 2, case["G"], case["page"], case["D"])


def work(case):
    op, es = case["op"], _es(case)
    G, D = case["G"], case["D"]
    if op in ("turn", "compact"):
        per = math.prod(_shape(case)) * es
        held = 0.625 * case["ctx"] / case["page"] + 0.5       # pages of a request, on average
        if op == "turn":
            made = case["n"] * case["branches"]
            return {"bytes": made * (2 * per + 24 * held), "flops": 4 * made * held}
        live = case["n"] * held
        return {"bytes": live * (1 - case["live"]) * 2 * per + live * (8 + 8 / case["live"]), "flops": live / case["live"]}
    H = case["H"]
    if op == "paged":
        rows, keys = case["n"] * case["T"], case["n"] * (case["T"] + 0.625 * (case["ctx"] - case["T"]))   # on average
        if case["packed"]:
            rows = case["T"]
        return {"bytes": 2 * keys * G * D * es + rows * ((2 * H + 4 * G) * D * es + 4 * H), "flops": 4 * D * H * rows * (keys / case["n"] - rows / case["n"] / 2)}
    rows = case["T"] if case["packed"] else case["n"] * case["T"]
    pairs = H * rows * (rows / case["n"] + 1) / 2
    if op == "prompt":
        return {"bytes": rows * ((2 * H + 2 * G) * D * es + 4 * H), "flops": 4 * D * pairs}
    return {"bytes": rows * ((4 * H + 4 * G) * D * es + 4 * H), "flops": 10 * D * pairs}


# ----------------------------------------------------------------- inputs

def _lens(r, n, T):
    """n lengths that add up to T, some far shorter than others."""
    w = [r.uniform(0.1, 1.0) for _ in range(n)]
    lens = [int(T * x / sum(w)) for x in w]
    lens[-1] += T - sum(lens)
    return lens


def _contexts(r, n, ctx):
    """Lengths of n requests, spread over a quarter of ctx up to all of it, in any order, and the most that they can be."""
    part = 0.75 * ctx / n
    held = [int(ctx / 4 + (i + r.random()) * part) for i in range(n)]
    r.shuffle(held)
    return [max(1, h) for h in held], [int(ctx / 4 + (i + 1) * part) + 1 for i in range(n)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed * 7919 + case["n"])
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    op, n, G, D = case["op"], case["n"], case["G"], case["D"]
    s = {"op": op, "n": n, "G": G, "D": D}
    if op in ("turn", "compact"):
        return _prepare_pages(case, s, r, normal, ints)
    H = s["H"] = case["H"]
    if case["packed"]:
        lens = _lens(r, n, case["T"])
        rows = (case["T"],)
        s["cu"], s["longest"] = ints([0] + list(np.cumsum(lens))), max(lens)
    else:
        lens = [case["T"]] * n
        rows = (n, case["T"])
        s["cu"], s["longest"] = None, case["T"]
    # q, k and v are the columns of one projection's output
    s["qkv"] = normal(*rows, (H + 2 * G) * D)
    s["qkv"][..., :H * D] *= 1.5
    if op == "paged":
        page = case["page"]
        held, at_most = _contexts(r, n, case["ctx"])
        held = [max(m, h) for m, h in zip(lens, held)]
        s["lengths"], s["page"] = ints(held), page
        most = -(-case["ctx"] // page)
        count = [-(-h // page) for h in held]
        total = sum(-(-max(case["T"], h) // page) for h in at_most) + 1
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((n, most), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, c in enumerate(count):
            table[b, :c] = order[at:at + c]
            at += c
        s["table"] = table
        s["k_pages"], s["v_pages"] = normal(total, G, page, D), normal(total, G, page, D)
        return s
    if op == "prompt_bwd":
        s["gy"] = normal(*rows, H, D)
        with torch.no_grad():   # what the forward pass of the step has left
            P, lse = _softmax(s, *_operands(s))
            o = (P @ _heads(s, _padded(s, _split(s)[2]))).transpose(1, 2)
        s["o"], s["lse"] = _unpadded(s, o).to(dt).contiguous(), _unpadded(s, lse.transpose(1, 2)).contiguous()
    return s


def _prepare_pages(case, s, r, normal, ints):
    """A pool of pages that requests hold in no order."""
    page, n = case["page"], case["n"]
    s["page"] = page
    if case["op"] == "turn":
        own_len, at_most = _contexts(r, n, case["ctx"])
        slots = n * (1 + case["branches"])
        held = own_len + [0] * (slots - n)
        s["src"] = ints([i for i in range(n) for _ in range(case["branches"])])
        s["dst"] = ints(list(range(n, slots)))
        back = own_len + [own_len[i] for i in range(n) for _ in range(case["branches"])]
        s["up"], s["back"] = ints([h + case["drafts"] for h in back]), ints(back)
        most = -(-(case["ctx"] + case["drafts"]) // page)
        total = sum(-(-h // page) for h in at_most) + slots * (3 + case["drafts"] // page)
        shared = 0
    else:
        held, at_most = _contexts(r, n, case["ctx"])
        most = -(-case["ctx"] // page)
        total = int(sum(-(-h // page) for h in at_most) / case["live"]) + 1
        shared = 1
    free = list(range(total))
    r.shuffle(free)
    table = [[-1] * most for _ in held]
    refs = [0] * total
    for b, h in enumerate(held):
        for c in range(-(-h // page)):
            # every fourth request of the compacted pool is a branch of the one before it
            if shared and b % 4 == 3 and c < min(h, held[b - 1]) // page // 2:
                table[b][c] = table[b - 1][c]
            else:
                table[b][c] = free.pop()
            refs[table[b][c]] += 1
    s["table"], s["lengths"], s["refs"] = ints(table), ints(held), ints(refs)
    s["pages"] = normal(total, *_shape(case))
    return s


def _split(s):
    """q, k and v as the columns of the projection's output."""
    HD, GD = s["H"] * s["D"], s["G"] * s["D"]
    q, k, v = s["qkv"][..., :HD], s["qkv"][..., HD:HD + GD], s["qkv"][..., HD + GD:]
    return q.unflatten(-1, (s["H"], s["D"])), k.unflatten(-1, (s["G"], s["D"])), v.unflatten(-1, (s["G"], s["D"]))


# -------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


# --- the framework's calls

def _own_prompt(s):
    import gated_delta_rule_amd as kda
    q, k, v = _split(s)
    return kda.attn_fwd(q, k, v, s["cu"])


def _own_prompt_bwd(s):
    import gated_delta_rule_amd as kda
    q, k, v = _split(s)
    g = torch.empty_like(s["qkv"])
    gq, gk, gv = _split({**s, "qkv": g})
    kda.attn_bwd(q, k, v, s["o"], s["lse"], s["gy"], s["cu"], grad_q=gq, grad_k=gk, grad_v=gv)
    return g


def _own_paged(s):
    import gated_delta_rule_amd as kda
    q, k, v = _split(s)
    kda.kv_append(k, v, s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["cu"])
    o, lse = kda.attn_paged_fwd(q, s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["cu"])
    return o, lse, s["k_pages"], s["v_pages"]


def _own_turn(s):
    import gated_delta_rule_amd as kda
    forked = kda.kv_fork(s["table"], s["lengths"], s["refs"], s["src"], s["dst"], s["pages"], s["page"])
    grown = kda.kv_resize(s["table"], s["lengths"], s["refs"], s["up"], s["page"])
    kda.kv_resize(s["table"], s["lengths"], s["refs"], s["back"], s["page"])
    return forked, grown, s["table"], s["lengths"], s["refs"], s["pages"]


def _own_compact(s):
    import gated_delta_rule_amd as kda
    table, refs, n_live = kda.kv_compact(s["table"], s["lengths"], s["refs"], s["pages"], s["page"])
    return table, refs, n_live, s["pages"]


_run_own = {"prompt": _own_prompt, "prompt_bwd": _own_prompt_bwd, "paged": _own_paged, "turn": _own_turn, "compact": _own_compact}


# --- the plain forms

def _padded(s, t):
    """A packed batch as equal lengths [n, longest, ...] in 32 bits, rows past a sequence's end zero."""
    t = t.float()
    if s["cu"] is None:
        return t
    start, end = s["cu"].long()[:-1, None], s["cu"].long()[1:, None]
    at = start + torch.arange(s["longest"], device=t.device)
    kept = (at < end).view(at.shape + (1,) * (t.dim() - 1))
    return t[at.clamp(max=t.shape[0] - 1)] * kept


def _unpadded(s, t):
    if s["cu"] is None:
        return t
    cu = s["cu"].long()
    rows = torch.arange(s["qkv"].shape[0], device=t.device)
    seq = torch.searchsorted(cu, rows, right=True) - 1
    return t[seq, rows - cu[seq]]


def _heads(s, t):
    """[n, T, G, D] as [n, H, T, D]."""
    return t.repeat_interleave(s["H"] // s["G"], 2).transpose(1, 2).contiguous()


def _operands(s):
    """q and k^T of every head, and which keys a query sees."""
    q, k, _ = _split(s)
    q, k = _padded(s, q).transpose(1, 2).contiguous(), _heads(s, _padded(s, k))
    T = q.shape[2]
    seen = torch.tril(torch.ones(T, T, dtype=torch.bool, device=q.device))
    return q, k.transpose(-1, -2).contiguous(), seen


def _softmax(s, q, kT, seen):
    """P and the logarithm of its rows' sums."""
    x = torch.where(seen, (q @ kT) * s["D"] ** -0.5, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    return x / total, (top + torch.log(total))[..., 0]


def _plain_prompt(s):
    P, lse = _softmax(s, *_operands(s))
    o = P @ _heads(s, _padded(s, _split(s)[2]))
    return _unpadded(s, o.transpose(1, 2)).to(s["qkv"].dtype), _unpadded(s, lse.transpose(1, 2))


def _plain_prompt_bwd(s):
    q, kT, seen = _operands(s)
    P, _ = _softmax(s, q, kT, seen)
    vT = _heads(s, _padded(s, _split(s)[2])).transpose(-1, -2).contiguous()
    gy = _padded(s, s["gy"]).transpose(1, 2).contiguous()
    gv = P.transpose(-1, -2).contiguous() @ gy
    gP = gy @ vT
    gS = P * (gP - (P * gP).sum(-1, keepdim=True)) * s["D"] ** -0.5
    gq = gS @ kT.transpose(-1, -2).contiguous()
    gk = gS.transpose(-1, -2).contiguous() @ q

    def fold(t):   # the sum over the heads of a group
        return t.unflatten(1, (s["G"], s["H"] // s["G"])).sum(2)

    every = torch.cat([gq, fold(gk), fold(gv)], 1).transpose(1, 2)
    return _unpadded(s, every).flatten(-2).to(s["qkv"].dtype)


def _positions(s):
    """Request and position of every new row, as [n, longest]; rows past a request's chunk are not there."""
    dev = s["qkv"].device
    if s["cu"] is None:
        count = torch.full((s["n"],), s["longest"], device=dev)
    else:
        count = (s["cu"][1:] - s["cu"][:-1]).long()
    t = torch.arange(s["longest"], device=dev)
    return (s["lengths"].long() - count)[:, None] + t, t < count[:, None]


def _plain_paged(s):
    q, k, v = _split(s)
    page, n, G, D, H = s["page"], s["n"], s["G"], s["D"], s["H"]
    pos, there = _positions(s)
    b = torch.arange(n, device=pos.device)[:, None].expand_as(pos)[there]
    x = pos[there]
    at = s["table"].long()[b, x // page]
    s["k_pages"][at, :, x % page] = k.reshape(-1, G, D)
    s["v_pages"][at, :, x % page] = v.reshape(-1, G, D)

    def all_of(pages):   # [n, H, L, D]
        t = pages[s["table"].long().clamp(min=0)].float()
        return t.transpose(2, 3).reshape(n, -1, G, D)

    L = s["table"].shape[1] * page
    j = torch.arange(L, device=pos.device)
    used = (j < s["lengths"].long()[:, None])[..., None, None]
    K, V = torch.where(used, all_of(s["k_pages"]), 0.0), torch.where(used, all_of(s["v_pages"]), 0.0)
    # the heads of a group beside each other: [n, G, H / G * T, D]
    per = H // G
    qs = _padded(s, q).unflatten(2, (G, per)).permute(0, 2, 3, 1, 4).reshape(n, G, -1, D)
    seen = (j <= pos[..., None]).repeat(1, per, 1)[:, None]
    P, lse = _softmax(s, qs, K.permute(0, 2, 3, 1).contiguous(), seen)
    o = (P @ V.transpose(1, 2).contiguous()).view(n, H, -1, D).transpose(1, 2)
    lse = lse.reshape(n, H, -1).transpose(1, 2)
    return _unpadded(s, o).to(s["qkv"].dtype), _unpadded(s, lse), s["k_pages"], s["v_pages"]


def _used(s):
    return (s["lengths"].long() + s["page"] - 1) // s["page"]


def _free_pages(refs):
    """The free pages' numbers, lowest first, and how many they are."""
    free = refs == 0
    rank = torch.cumsum(free.long(), 0) - 1
    found = torch.zeros(refs.numel() + 1, dtype=torch.long, device=refs.device)
    found[torch.where(free, rank, refs.numel())] = torch.arange(refs.numel(), device=refs.device)
    return found, free.sum()


def _plain_resize(s, want):
    table, refs = s["table"], s["refs"]
    col = torch.arange(table.shape[1], device=table.device)
    before = _used(s)
    after = (want.long() + s["page"] - 1) // s["page"]
    gone = (col >= after[:, None]) & (col < before[:, None])
    refs.index_add_(0, table.long().clamp(min=0).flatten(), -gone.flatten().to(refs.dtype))
    need = (after - before).clamp(min=0)
    upto = torch.cumsum(need, 0)
    found, n_free = _free_pages(refs)
    ok = (need == 0) | (upto <= n_free)
    new = (col >= before[:, None]) & (col < after[:, None]) & ok[:, None]
    pick = found[((upto - need)[:, None] + col - before[:, None]).clamp(0, refs.numel())]
    refs.index_add_(0, torch.where(new, pick, 0).flatten(), new.flatten().to(refs.dtype))
    table.copy_(torch.where(new, pick.to(table.dtype), torch.where(gone, -1, table)))
    s["lengths"].copy_(torch.where(ok, want, s["lengths"]))
    return ok.to(torch.int32)


def _plain_fork(s):
    table, refs, src, dst, page = s["table"], s["refs"], s["src"].long(), s["dst"].long(), s["page"]
    col = torch.arange(table.shape[1], device=table.device)
    used, length = _used(s), s["lengths"]
    open_ = (length[src] % page != 0).long()
    upto = torch.cumsum(open_, 0)
    found, n_free = _free_pages(refs)
    ok = upto <= n_free
    pick = found[(upto - 1).clamp(0, refs.numel())]
    rows, old = table[src], table[dst]
    last = (col == used[src][:, None] - 1) & (open_ > 0)[:, None]
    held = (col < used[src][:, None]) & ok[:, None]
    left = (col < used[dst][:, None]) & ok[:, None]
    tail = rows.long()[torch.arange(src.numel(), device=src.device), (used[src] - 1).clamp(min=0)]
    copied = torch.nonzero(ok & (open_ > 0))[:, 0]
    s["pages"][pick[copied]] = s["pages"][tail[copied]]
    new = torch.where(last, pick[:, None].to(table.dtype), rows)
    refs.index_add_(0, new.long().clamp(min=0).flatten(), held.flatten().to(refs.dtype))
    refs.index_add_(0, old.long().clamp(min=0).flatten(), -left.flatten().to(refs.dtype))
    table[dst] = torch.where(ok[:, None], torch.where(held, new, -1), old)
    length[dst] = torch.where(ok, length[src], length[dst])
    return ok.to(torch.int32)


def _plain_turn(s):
    forked = _plain_fork(s)
    grown = _plain_resize(s, s["up"])
    _plain_resize(s, s["back"])
    return forked, grown, s["table"], s["lengths"], s["refs"], s["pages"]


def _plain_compact(s):
    table, refs = s["table"].long(), s["refs"]
    N = refs.numel()
    live = refs > 0
    n_live = live.sum()
    p = torch.arange(N, device=refs.device)
    moves, hole = live & (p >= n_live), ~live & (p < n_live)
    rank_of = torch.cumsum(moves.long(), 0) - 1
    holes = torch.zeros(N + 1, dtype=torch.long, device=refs.device)
    holes[torch.where(hole, torch.cumsum(hole.long(), 0) - 1, N)] = p
    to = torch.where(moves, holes[rank_of.clamp(min=0)], p)
    at = torch.nonzero(moves)[:, 0]
    s["pages"][to[at]] = s["pages"][at]
    used = torch.arange(table.shape[1], device=table.device) < _used(s)[:, None]
    refs_after = torch.where(p < n_live, refs, 0)
    refs_after[to[at]] = refs[at]
    return torch.where(used, to[table.clamp(min=0)], -1).to(torch.int32), refs_after, n_live.to(torch.int32).view(1), s["pages"]


_run_plain = {"prompt": _plain_prompt, "prompt_bwd": _plain_prompt_bwd, "paged": _plain_paged, "turn": _plain_turn, "compact": _plain_compact}


# ------------------------------------------------------------------ exact

def _exact_head(q, K, V, first, scale, gy=None):
    """One head of one sequence in 64 bits: queries at positions first, first + 1, ... over all keys up to their own."""
    x = (q @ K.t()) * scale
    late = torch.arange(K.shape[0], device=x.device) > first + torch.arange(q.shape[0], device=x.device)[:, None]
    x.masked_fill_(late, -math.inf)
    lse = torch.logsumexp(x, -1)
    P = torch.exp(x - lse[:, None])
    o = P @ V
    if gy is None:
        return o, lse
    gS = P * (gy @ V.t() - (gy * o).sum(-1, keepdim=True))
    return scale * (gS @ K), scale * (gS.t() @ q), P.t() @ gy


def exact(case, seed):
    """The definitions, head by head in 64 bits."""
    if case["op"] in ("turn", "compact"):
        return None   # whole numbers, and pages whose bits move
    s = prepare(case, seed)
    n, H, G, D = case["n"], case["H"], case["G"], case["D"]
    q, k, v = (t.reshape(-1, t.shape[-2], D).double() for t in _split(s))
    cu = s["cu"].tolist() if s["cu"] is not None else [i * case["T"] for i in range(n + 1)]
    lead = s["qkv"].shape[:-1]
    scale, per = 1.0 / math.sqrt(D), H // G
    if case["op"] == "prompt_bwd":
        gy = s["gy"].reshape(-1, H, D).double()
        gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for a, e in zip(cu, cu[1:]):
            for h in range(H):
                g = h // per
                x, y, z = _exact_head(q[a:e, h], k[a:e, g], v[a:e, g], 0, scale, gy[a:e, h])
                gq[a:e, h] = x
                gk[a:e, g] += y
                gv[a:e, g] += z
        return torch.cat([t.flatten(-2) for t in (gq, gk, gv)], -1).view(*lead, -1)
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    if case["op"] == "paged":
        held, table, page = s["lengths"].tolist(), s["table"].tolist(), case["page"]
    for i, (a, e) in enumerate(zip(cu, cu[1:])):
        if case["op"] == "prompt":
            K, V, first = k[a:e], v[a:e], 0
        else:   # the request's earlier tokens from its pages, then the new ones
            first = held[i] - (e - a)
            mine = torch.tensor(table[i][:-(-held[i] // page)], device=q.device)
            old = [s[name][mine].transpose(1, 2).reshape(-1, G, D)[:first].double() for name in ("k_pages", "v_pages")]
            K, V = torch.cat([old[0], k[a:e]]), torch.cat([old[1], v[a:e]])
        for h in range(H):
            o[a:e, h], lse[a:e, h] = _exact_head(q[a:e, h], K[:, h // per], V[:, h // per], first, scale)
    o, lse = o.view(*lead, H, D), lse.view(*lead, H)
    return (o, lse) if case["op"] == "prompt" else (o, lse, None, None)
