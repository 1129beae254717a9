"""Workloads of a serving and training step around the paged K/V cache: norms of queries and keys with
their rotary positions (forward, gradient, and written to the cache), the pages and slots of new tokens,
and attention of one new token over a cache whose first keys the whole batch shares.

Each case has a plain form (elementary torch operations in 32 bits, angles and long sums in 64) and the
calls of this package (``own``).  Caches are [pages, page_size, Hkv, d] with the pages of a sequence in a
shuffled order; lengths are ragged.
"""
import math

import torch

own = False


def listed():
    return [
        # queries and keys of the video self-attention's blocks: (time, height, width) axes
        {"name": "norm_rope_video", "op": "norm", "backward": False, "B": 1, "S": 32760, "H": 12, "Hkv": 12, "d": 128,
         "layout": "bshd", "axis_dims": "44,42,42", "pairing": "adjacent", "fused": True, "far": 0, "weight": "fp32"},
        # a short prompt: the call's own latency; half of each head is rotated
        {"name": "norm_rope_short_d64", "op": "norm", "backward": False, "B": 3, "S": 37, "H": 4, "Hkv": 2, "d": 64,
         "layout": "bhsd", "axis_dims": "32", "pairing": "halves", "fused": False, "far": 0, "weight": "bf16"},
        # training step of the decoder-style prefill: gradients of q, k and of both weights
        {"name": "norm_rope_bwd_gqa", "op": "norm", "backward": True, "B": 2, "S": 8192, "H": 32, "Hkv": 8, "d": 128,
         "layout": "bshd", "axis_dims": "128", "pairing": "halves", "fused": True, "far": 0, "weight": "bf16"},
        # the same of a small model's short sequences
        {"name": "norm_rope_bwd_d64", "op": "norm", "backward": True, "B": 3, "S": 333, "H": 6, "Hkv": 2, "d": 64,
         "layout": "bhsd", "axis_dims": "20,22,22", "pairing": "adjacent", "fused": False, "far": 1000000, "weight": "fp32"},
        # one decoding step of a batch: the new tokens' q, k, v out of one projection
        {"name": "norm_append_step", "op": "append", "B": 64, "new": 1, "H": 32, "Hkv": 8, "d": 128, "page": 256,
         "longest": 4096, "axis_dims": "128", "pairing": "halves", "far": 0, "weight": "bf16"},
        # a ragged chunk of a prefill, written to the cache before it is attended to
        {"name": "norm_append_chunk", "op": "append", "B": 16, "new": 512, "H": 32, "Hkv": 8, "d": 128, "page": 128,
         "longest": 4096, "axis_dims": "32,48,48", "pairing": "adjacent", "far": 0, "weight": "fp32"},
        # pages and slots of a decoding step: one token each, a few sequences reach a new page, some have ended
        {"name": "reserve_step", "op": "reserve", "B": 256, "new": 1, "page": 16, "longest": 4096, "ended": 0.05, "shared": 0},
        # of a prefill's chunks beside them, behind a shared prefix of 8 pages
        {"name": "reserve_prefill", "op": "reserve", "B": 64, "new": 1024, "page": 64, "longest": 8192, "ended": 0.2,
         "shared": 8},
        # a few samples of one short prompt: the call's own latency
        {"name": "prefix_few_d64", "op": "prefix", "B": 4, "H": 8, "Hkv": 2, "d": 64, "page": 16, "prefix": 600, "shortest": 1,
         "longest": 64},
        # a serving batch behind one long instruction
        {"name": "prefix_batch", "op": "prefix", "B": 64, "H": 32, "Hkv": 8, "d": 128, "page": 256, "prefix": 16384,
         "shortest": 256, "longest": 1024},
        # questions about one long document
        {"name": "prefix_long", "op": "prefix", "B": 24, "H": 32, "Hkv": 8, "d": 128, "page": 128, "prefix": 65500,
         "shortest": 1, "longest": 300},
        # a large batch with an odd group of query heads and small odd pages: the prefix is bound by its products
        {"name": "prefix_wide", "op": "prefix", "B": 512, "H": 40, "Hkv": 8, "d": 128, "page": 24, "prefix": 4133,
         "shortest": 1, "longest": 200},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, pairs, axes):
    """`pairs` pairs over `axes` axes, one at least for each, as the axes' rotated dimensions."""
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return ",".join(str(2 * (b - a)) for a, b in zip([0] + cuts, cuts + [pairs]))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "reserve", "prefix", "prefix"])
    if op == "reserve":
        B, page = _log(rng, 1, 1024), rng.choice([1, 16, 24, 64, 128, 256])
        new = _log(rng, 1, max(1, 65536 // B))
        longest = new + _log(rng, 64, 8192)
        return {"op": op, "B": B, "new": new, "page": page, "longest": longest, "ended": rng.choice([0.0, 0.05, 0.3]),
                "shared": rng.choice([0, 0, rng.randint(1, 64)])}
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8])
    H = Hkv * rng.choice([1, 2, 4, 4, 5, 8])
    page = rng.choice([1, 16, 24, 64, 100, 128, 256])
    if op == "prefix":
        B = _log(rng, 1, 256)
        # products, keys and values of the prefix, and those of the rest, within the largest listed ones'
        prefix = _log(rng, 16, max(17, min(65500, 8000000 // (B * H) * 10, 65500 * 8 * 128 // (Hkv * d))))
        longest = _log(rng, 1, max(2, min(4096, 512 * 200 * 8 // (B * Hkv))))
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "page": page, "prefix": prefix,
                "shortest": rng.randint(1, longest), "longest": longest}
    pairing = rng.choice(["adjacent", "halves"])
    pairs = rng.choice([d // 2, d // 2, d // 4])
    axis_dims = _split(rng, pairs, rng.choice([1, 1, 2, 3]))
    far = rng.choice([0, 0, 100000, 1000000])
    weight = rng.choice(["fp32", "bf16"])
    if op == "append":
        return {"op": op, "B": _log(rng, 1, 64), "new": _log(rng, 1, 128), "H": H, "Hkv": Hkv, "d": d, "page": page,
                "longest": _log(rng, 600, 4096), "axis_dims": axis_dims, "pairing": pairing, "far": far, "weight": weight}
    B = rng.choice([1, 1, 2, 3])
    S = _log(rng, 1, max(2, 640000 // (B * (H + Hkv))))
    return {"op": op, "backward": rng.random() < 0.5, "B": B, "S": S, "H": H, "Hkv": Hkv, "d": d,
            "layout": rng.choice(["bshd", "bhsd"]), "axis_dims": axis_dims, "pairing": pairing,
            "fused": rng.random() < 0.5, "far": far, "weight": weight}


# ------------------------------------------------------------------------------------- inputs
EPS = 1e-6


def _frequencies(axis_dims):
    """Radians per unit of position of each rotated pair, and the axis whose position it takes."""
    dims = [int(n) for n in axis_dims.split(",")]
    freqs = [10000.0 ** (-2.0 * i / n) for n in dims for i in range(n // 2)]
    axes = [a for a, n in enumerate(dims) for _ in range(n // 2)]
    return freqs, axes, len(dims)


def _randint(g, lo, hi, n):
    """n whole numbers from lo to hi."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    s = dict(case)
    B = case["B"]
    if case["op"] == "reserve":
        page, new, shared = case["page"], case["new"], case["shared"]
        longest = case["longest"] + shared * page
        # each sequence's pages before the step; those that have ended give theirs back
        news = _randint(g, max(1, new // 2), new, B)
        old = _randint(g, 0, longest - shared * page - new, B) + shared * page
        ended = torch.rand(B, generator=g, device="cuda") < case["ended"]
        held = (old + page - 1) // page
        most = -(-longest // page)
        pages = shared + B * most                                       # enough for every sequence at its longest
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        at = torch.arange(most, device="cuda")
        own_page = (at >= shared) & (at < held[:, None])
        rank = torch.cumsum(own_page.flatten(), 0).view(B, most) - 1 + shared
        table = torch.where(own_page, order[rank.clamp(min=0)], -1)
        if shared:
            table[:, :shared] = order[:shared]
        used = shared + int(own_page.sum())
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        s["free"][:pages - used] = order[used:]
        s["count"] = torch.tensor([pages - used], dtype=torch.int32, device="cuda")
        s["table"], s["held"] = table, held
        news = torch.where(ended, 0, news)
        s["lens"] = torch.where(ended, 0, old + news).to(torch.int32)
        s["cu"] = torch.cat([news.new_zeros(1), news.cumsum(0)]).to(torch.int32)
        s["shared_pages"] = torch.full((B,), shared, dtype=torch.int32, device="cuda") if shared else None
        total = B * new                                                 # the step's token budget
        s["held_out"], s["count_out"] = torch.zeros_like(held), torch.zeros_like(s["count"])
        s["slots"] = torch.zeros(total, dtype=torch.int64, device="cuda")
        s["positions"] = torch.zeros(total, dtype=torch.int32, device="cuda")
        return s
    Hkv, d = case["Hkv"], case["d"]
    normal = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    if case["op"] == "prefix":
        page, prefix = case["page"], case["prefix"]
        own_keys = _randint(g, case["shortest"], case["longest"], B)
        own_keys[0] = case["longest"]
        s["lens"] = own_keys + prefix
        # pages wholly inside the prefix are shared; of the one that it ends in every sequence has a copy
        shared, most = prefix // page, -(-(prefix + case["longest"]) // page)
        pages = shared + B * (most - shared)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["table"] = torch.cat([order[:shared].expand(B, shared), order[shared:].view(B, most - shared)], 1).contiguous()
        s["k_cache"], s["v_cache"] = normal(pages, page, Hkv, d), normal(pages, page, Hkv, d)
        rest = prefix - shared * page
        if rest:
            ends = s["table"][:, shared].long()
            for c in (s["k_cache"], s["v_cache"]):
                c[ends, :rest] = c[ends[0], :rest]
        s["q"] = normal(B, case["H"], d) * 2                            # logits of deviation 2: some keys stand out
        return s
    freqs, axes, n = _frequencies(case["axis_dims"])
    H = case["H"]
    s["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
    s["axes"] = torch.tensor(axes, dtype=torch.int32, device="cuda")
    wt = torch.bfloat16 if case["weight"] == "bf16" else torch.float32
    s["qw"], s["kw"] = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(wt) for _ in range(2))
    if case["op"] == "append":
        page = case["page"]
        new = _randint(g, max(1, case["new"] // 2), case["new"], B).long()
        new[0] = case["new"]
        total = B * case["new"]     # the program's token budget; rows past the last sequence's are not used
        cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
        lens = new + torch.randint(0, case["longest"] - case["new"] + 1, (B,), generator=g, device="cuda")
        most = -(-case["longest"] // page)
        table = torch.randperm(B * most, generator=g, device="cuda").view(B, most)
        token = torch.arange(total, device="cuda")
        b = (torch.searchsorted(cu, token, right=True) - 1).clamp(max=B - 1)
        at = lens[b] - cu[b + 1] + token
        used = token < cu[B]
        s["slots"] = torch.where(used, table[b, torch.where(used, at, 0) // page] * page + at % page, -1)
        x = normal(total, H + 2 * Hkv, d) * 3
        s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        s["q_out"] = torch.zeros((total, H, d), dtype=torch.bfloat16, device="cuda")
        s["k_cache"], s["v_cache"] = normal(B * most, page, Hkv, d), normal(B * most, page, Hkv, d)
        s["positions"] = (torch.randint(0, 4096, (n, total), generator=g, device="cuda") + case["far"]).to(torch.int32)
        return s
    S = case["S"]
    # the grid's positions (or a text's), the same for every sequence of the batch
    at = torch.arange(S, device="cuda")
    side = max(1, math.isqrt(S))
    s["positions"] = torch.stack([at // (side ** (n - 1 - a)) % (side if a else S) + case["far"] for a in range(n)]).to(torch.int32)
    for names in (("q", "k"), ("dq", "dk"))[:2 if case["backward"] else 1]:
        # projections' outputs have heads of different sizes
        if case["fused"]:   # views of one projection's output
            x = normal(B, S, H + 2 * Hkv, d) * 3
            pair = x[:, :, :H], x[:, :, H:H + Hkv]
        else:
            pair = normal(B, S, H, d) * 3, normal(B, S, Hkv, d) * 0.3
        if case["layout"] == "bhsd":
            pair = [t.transpose(1, 2) if case["fused"] else t.transpose(1, 2).contiguous() for t in pair]
        s[names[0]], s[names[1]] = pair
    return s


# ------------------------------------------------------------------------------------- plain forms
def _turn(x, cos, sin, pairing):
    """x [..., d] (fp32) rotated by angles whose cosines and sines are [..., pairs]."""
    n = cos.shape[-1]
    if pairing == "adjacent":
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _angles(s, head_dim):
    """Cosines and sines of the positions, from angles in 64 bits, to be broadcast over the heads."""
    angle = s["positions"][s["axes"].long()].double().T * s["freqs"]
    return angle.cos().float().unsqueeze(head_dim), angle.sin().float().unsqueeze(head_dim)


def _norm_turn(x, w, cos, sin, pairing):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _turn(y, cos, sin, pairing).to(torch.bfloat16)


def _norm_turn_bwd(dy, x, w, cos, sin, pairing):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    g = _turn(dy.float(), cos, -sin, pairing)
    dw = (g * n).sum((0, 1, 2), dtype=torch.float64).float()
    g = g * w.float()
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dw


def _plain_norm(s):
    cos, sin = _angles(s, 1 if s["layout"] == "bshd" else 0)
    if not s["backward"]:
        return [_norm_turn(s["q"], s["qw"], cos, sin, s["pairing"]), _norm_turn(s["k"], s["kw"], cos, sin, s["pairing"])]
    dq, dqw = _norm_turn_bwd(s["dq"], s["q"], s["qw"], cos, sin, s["pairing"])
    dk, dkw = _norm_turn_bwd(s["dk"], s["k"], s["kw"], cos, sin, s["pairing"])
    return [dq, dk, dqw, dkw]


def _plain_append(s):
    cos, sin = _angles(s, 1)
    used = s["slots"] >= 0
    # a token without a slot writes what the first one does
    slot = torch.where(used, s["slots"], s["slots"][0])
    row = torch.where(used, torch.arange(slot.numel(), device="cuda"), 0)
    k = _norm_turn(s["k"], s["kw"], cos, sin, s["pairing"])
    s["k_cache"].view(-1, s["Hkv"], s["d"])[slot] = k[row]
    s["v_cache"].view(-1, s["Hkv"], s["d"])[slot] = s["v"][row]
    q = _norm_turn(s["q"], s["qw"], cos, sin, s["pairing"])
    s["q_out"].copy_(torch.where(used[:, None, None], q, s["q_out"]))
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _plain_reserve(s):
    page, table, free = s["page"], s["table"], s["free"]
    B, most = table.shape
    held, lens, cu = s["held"].long(), s["lens"].long(), s["cu"].long()
    want = (lens + page - 1) // page
    if s["shared_pages"] is not None:
        want = torch.maximum(want, s["shared_pages"].long())
    at = torch.arange(most, device="cuda")
    back = (at >= want[:, None]) & (at < held[:, None])
    take = (at >= held[:, None]) & (at < want[:, None])
    returned = torch.cumsum(back.flatten(), 0).view(B, most)
    taken = torch.cumsum(take.flatten(), 0).view(B, most)
    count = s["count"].long()
    # returned pages go on top of the stack, taken ones come from its top; positions that
    # no page goes to lie behind the stack's end
    end = free.numel()
    stack = torch.cat([free, free.new_zeros(1)])
    stack.scatter_(0, torch.where(back, count + returned - 1, end).flatten(), table.flatten())
    top = count + returned[-1, -1]
    pages = stack[torch.where(take, top - taken, 0).clamp(min=0)]
    table.copy_(torch.where(take, pages, table))
    free.copy_(stack[:end])
    s["held_out"].copy_(want)
    s["count_out"].copy_(top - taken[-1, -1])
    token = torch.arange(s["slots"].numel(), device="cuda")
    b = (torch.searchsorted(cu, token, right=True) - 1).clamp(max=B - 1)
    used = token < cu[B]
    position = torch.where(used, lens[b] - cu[b + 1] + token, 0)
    s["positions"].copy_(position)
    s["slots"].copy_(torch.where(used, table[b, position // page].long() * page + position % page, -1))
    return _reserved(s)


def _reserved(s):
    return [s["table"], s["held_out"], s["free"], s["count_out"], s["slots"], s["positions"]]


def _plain_prefix(s):
    B, Hkv, d, page, prefix = s["B"], s["Hkv"], s["d"], s["page"], s["prefix"]
    table = s["table"].long()
    whole, cut = -(-prefix // page), prefix // page
    q = s["q"].float().view(B, Hkv, -1, d)
    G = q.shape[2]
    # the prefix once for all sequences
    k, v = (s[c][table[0, :whole]].flatten(0, 1)[:prefix].float().transpose(0, 1) for c in ("k_cache", "v_cache"))
    rows = q.transpose(0, 1).reshape(Hkv, B * G, d)
    x = torch.matmul(rows, k.transpose(1, 2)).view(Hkv, B, G, prefix) / math.sqrt(d)
    # each sequence's own keys
    ko, vo = (s[c][table[:, cut:]].flatten(1, 2).float() for c in ("k_cache", "v_cache"))
    xo = torch.matmul(q, ko.permute(0, 2, 3, 1)).transpose(0, 1) / math.sqrt(d)
    at = torch.arange(ko.shape[1], device="cuda") + cut * page
    seen = (at >= prefix) & (at < s["lens"][:, None])
    xo = torch.where(seen[:, None], xo, -math.inf)
    top = torch.maximum(x.amax(-1, keepdim=True), xo.amax(-1, keepdim=True))
    e, eo = torch.exp(x - top), torch.exp(xo - top)
    total = e.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True)
    o = torch.matmul(e.view(Hkv, B * G, prefix), v).view(Hkv, B, G, d)
    vo = torch.where(seen[..., None, None], vo, 0.0)
    o = (o + torch.matmul(eo, vo.permute(2, 0, 1, 3))) / total
    lse = (top + torch.log(total)).squeeze(-1)
    return [o.transpose(0, 1).reshape(B, -1, d).to(torch.bfloat16), lse.transpose(0, 1).reshape(B, -1)]


def run(s):
    if own:
        import bf16_attention_forward_gb300 as attn
        if s["op"] == "norm":
            where = dict(eps=EPS, layout=s["layout"], pairing=s["pairing"])
            if s["backward"]:
                return list(attn.attn_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["positions"],
                                                    s["freqs"], s["axes"], **where))
            return list(attn.attn_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["positions"], s["freqs"], s["axes"], **where))
        if s["op"] == "append":
            attn.attn_norm_rope_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"], q_out=s["q_out"],
                                       q_weight=s["qw"], k_weight=s["kw"], positions=s["positions"], freqs=s["freqs"],
                                       axes=s["axes"], eps=EPS, pairing=s["pairing"])
            return [s["q_out"], s["k_cache"], s["v_cache"]]
        if s["op"] == "reserve":
            attn.attn_paged_reserve(s["lens"], s["cu"], s["table"], s["held"], s["free"], s["count"], s["page"],
                                    shared_pages=s["shared_pages"], held_out=s["held_out"], count_out=s["count_out"],
                                    slots=s["slots"], positions=s["positions"])
            return _reserved(s)
        return list(attn.attn_paged_prefix_decode(s["q"], s["k_cache"], s["v_cache"], s["lens"], s["table"], s["prefix"],
                                                  return_lse=True))
    return {"norm": _plain_norm, "append": _plain_append, "reserve": _plain_reserve, "prefix": _plain_prefix}[s["op"]](s)


# ------------------------------------------------------------------------------------- work
def work(case):
    """Each input read once and each output written once.  Numbers drawn between two bounds count with their
    mean.  Of a table, a list of free pages and the cache only what a step reads or changes counts."""
    B = case["B"]
    if case["op"] == "reserve":
        new = (max(1, case["new"] // 2) + case["new"]) / 2 * (1 - case["ended"])
        room = case["longest"] - case["new"]
        moved = new / case["page"] + case["ended"] * room / 2 / case["page"]     # pages taken and returned
        # lengths, offsets, pages held before and after; a page's entry read and written; a slot and a position
        return {"bytes": B * (16 + 8 * moved + 12 * case["new"]), "flops": B * case["new"]}
    Hkv, d = case["Hkv"], case["d"]
    row = 2 * d
    if case["op"] == "prefix":
        n, mean = case["prefix"], (case["shortest"] + case["longest"]) / 2
        return {"bytes": 2 * (n + B * mean) * Hkv * row + 2 * B * case["H"] * row + 4 * B * case["H"],
                "flops": 4 * B * case["H"] * d * (n + mean)}
    axes = case["axis_dims"].count(",") + 1
    if case["op"] == "append":
        n = B * (max(1, case["new"] // 2) + case["new"]) / 2
        return {"bytes": n * (2 * (case["H"] + 2 * Hkv) * row + 4 * axes + 8), "flops": 7 * n * (case["H"] + Hkv) * d}
    n = B * case["S"] * (case["H"] + Hkv)
    return {"bytes": (3 if case["backward"] else 2) * n * row + 4 * axes * case["S"],
            "flops": (15 if case["backward"] else 7) * n * d}


# ------------------------------------------------------------------------------------- 64 bits
def _exact_turn(y, positions, case, sign):
    """[tokens, heads, d] in 64 bits, rotated pair by pair."""
    freqs, axes, _ = _frequencies(case["axis_dims"])
    y = y.clone()
    n = len(freqs)
    for p, (f, a) in enumerate(zip(freqs, axes)):
        i, j = (2 * p, 2 * p + 1) if case["pairing"] == "adjacent" else (p, p + n)
        z = torch.polar(torch.ones_like(positions[a], dtype=torch.float64), sign * f * positions[a].double())[:, None]
        turned = torch.complex(y[..., i], y[..., j]) * z
        y[..., i], y[..., j] = turned.real, turned.imag
    return y


def _exact_norm(x, w, positions, case):
    x = x.double()
    size = torch.sqrt(torch.einsum("thd,thd->th", x, x) / case["d"] + EPS)
    return _exact_turn(x / size[..., None] * w.double(), positions, case, 1.0)


def _exact_norm_bwd(dy, x, w, positions, case):
    """dx through the matrix of first derivatives, (I - n n^T / d) / size, with n = x / size."""
    x = x.double()
    size = torch.sqrt(torch.einsum("thd,thd->th", x, x) / case["d"] + EPS)[..., None]
    g = _exact_turn(dy.double(), positions, case, -1.0)
    n = x / size
    dw = torch.einsum("thd,thd->d", g, n)
    g = g * w.double()
    return (g - n * torch.einsum("thd,thd->th", g, n)[..., None] / case["d"]) / size, dw


def exact(case, seed):
    s = prepare(case, seed)
    B = case["B"]
    if case["op"] == "reserve":
        page, shared = case["page"], case["shared"]
        table, held, lens, cu = s["table"].tolist(), s["held"].tolist(), s["lens"].tolist(), s["cu"].tolist()
        free, count = s["free"].tolist(), int(s["count"])
        want = [max(-(-n // page), shared) for n in lens]
        for b in range(B):
            for i in range(want[b], held[b]):
                free[count] = table[b][i]
                count += 1
        for b in range(B):
            for i in range(held[b], want[b]):
                count -= 1
                table[b][i] = free[count]
        slots, positions = [-1] * s["slots"].numel(), [0] * s["slots"].numel()
        for b in range(B):
            for t in range(cu[b], cu[b + 1]):
                j = positions[t] = lens[b] - cu[b + 1] + t
                slots[t] = table[b][j // page] * page + j % page
        return [torch.tensor(x, dtype=torch.float64, device="cuda") for x in (table, want, free, [count], slots, positions)]
    Hkv, d = case["Hkv"], case["d"]
    if case["op"] == "norm":
        dx, dw = [], []
        for x, dy, w in ((s["q"], s.get("dq"), s["qw"]), (s["k"], s.get("dk"), s["kw"])):
            x, dy = (t if t is None or case["layout"] == "bshd" else t.transpose(1, 2) for t in (x, dy))
            if case["backward"]:
                parts = [_exact_norm_bwd(dy[b], x[b], w, s["positions"], case) for b in range(B)]
                y = torch.stack([p[0] for p in parts])
                dw.append(sum(p[1] for p in parts))
            else:
                y = torch.stack([_exact_norm(x[b], w, s["positions"], case) for b in range(B)])
            dx.append(y if case["layout"] == "bshd" else y.transpose(1, 2))
        return dx + dw
    if case["op"] == "append":
        q, k = (_exact_norm(s[x], s[x + "w"], s["positions"], case) for x in ("q", "k"))
        out = [s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()]
        rows = [(t, slot) for t, slot in enumerate(s["slots"].tolist()) if slot >= 0]
        token, slot = (torch.tensor(x, device="cuda") for x in zip(*rows))
        out[0].index_copy_(0, token, q[token])
        out[1].view(-1, Hkv, d).index_copy_(0, slot, k[token])
        out[2].view(-1, Hkv, d).index_copy_(0, slot, s["v"][token].double())
        return out
    page, prefix = case["page"], case["prefix"]
    G = case["H"] // Hkv
    o = torch.empty((B, case["H"], d), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, case["H"]), dtype=torch.float64, device="cuda")

    def keys(b, first, end, h):
        ids = s["table"][b, first // page:-(-end // page)].long()
        at = slice(first % page, first % page + end - first)
        return [s[c][..., h, :].index_select(0, ids).flatten(0, 1)[at].double() for c in ("k_cache", "v_cache")]

    lens = s["lens"].tolist()
    for h in range(Hkv):
        q = s["q"][:, h * G:(h + 1) * G].double()
        shared_k, shared_v = keys(0, 0, prefix, h)
        x = (q.reshape(B * G, d) @ shared_k.T * d ** -0.5).view(B, G, prefix)
        for b in range(B):
            k, v = keys(b, prefix, lens[b], h)
            y = q[b] @ k.T * d ** -0.5
            z = torch.logaddexp(torch.logsumexp(x[b], 1), torch.logsumexp(y, 1))[:, None]
            o[b, h * G:(h + 1) * G] = (x[b] - z).exp() @ shared_v + (y - z).exp() @ v
            lse[b, h * G:(h + 1) * G] = z[:, 0]
    return [o, lse]
