"""Workloads of the operators around the paged K/V cache: rotary positions with several axes
(forward and backward), appending to the cache, attention of one new token, and eviction by
accumulated attention weight.

Each case has a plain form (elementary torch operations in 32 bits, angles in 64) and the calls
of this package (``own``).  Caches are [pages, page_size, Hkv, d] with the pages of a sequence
in a shuffled order; sequence lengths are ragged.
"""
import math

import torch

own = False


def listed():
    return [
        # rotary positions of the video self-attention's q and k: (time, height, width) axes
        {"name": "rope_video", "op": "rope", "B": 1, "S": 32760, "H": 12, "Hkv": 12, "d": 128, "layout": "bshd",
         "axis_dims": "44,42,42", "pairing": "adjacent", "backward": False, "fused": False, "far": 0},
        # gradients of the decoder-style prefill's rotated q and k, one axis, far positions
        {"name": "rope_gqa_backward", "op": "rope", "B": 2, "S": 8192, "H": 32, "Hkv": 8, "d": 128, "layout": "bshd",
         "axis_dims": "128", "pairing": "halves", "backward": True, "fused": False, "far": 1000000},
        # a short prompt: the call's own latency; part of each head is rotated
        {"name": "rope_short_d64", "op": "rope", "B": 3, "S": 37, "H": 4, "Hkv": 2, "d": 64, "layout": "bhsd",
         "axis_dims": "32,16", "pairing": "adjacent", "backward": False, "fused": False, "far": 0},
        # one decoding step of a batch: the new token's q, k, v out of one projection
        {"name": "append_step", "op": "append", "B": 64, "new": 1, "H": 32, "Hkv": 8, "d": 128, "page": 256,
         "longest": 4096, "axis_dims": "128", "pairing": "halves", "far": 0},
        # a ragged chunk of a prefill with image positions, written to the cache before it is attended to
        {"name": "append_chunk", "op": "append", "B": 16, "new": 512, "H": 32, "Hkv": 8, "d": 128, "page": 128,
         "longest": 4096, "axis_dims": "32,48,48", "pairing": "halves", "far": 0},
        # one user's first tokens: a short cache, small pages
        {"name": "decode_one_short", "op": "decode", "B": 1, "H": 8, "Hkv": 2, "d": 64, "page": 16, "shortest": 513,
         "longest": 513, "weights": False},
        # a few long sequences
        {"name": "decode_few_long", "op": "decode", "B": 4, "H": 32, "Hkv": 8, "d": 128, "page": 256, "shortest": 4096,
         "longest": 16384, "weights": False},
        # the serving batch of the decoding benchmark
        {"name": "decode_batch", "op": "decode", "B": 64, "H": 32, "Hkv": 8, "d": 128, "page": 256, "shortest": 4096,
         "longest": 16384, "weights": False},
        # very ragged lengths, small pages, an odd group of query heads, weights kept for eviction
        {"name": "decode_ragged_weights", "op": "decode", "B": 24, "H": 40, "Hkv": 8, "d": 128, "page": 16, "shortest": 1,
         "longest": 20000, "weights": True},
        # eviction while decoding: each cache is a few keys over its budget
        {"name": "evict_step", "op": "evict", "B": 32, "Hkv": 8, "d": 128, "page": 16, "shortest": 1000, "longest": 1040,
         "budget": 1024, "sinks": 4, "recent": 128},
        # after a prefill: long caches cut to a budget
        {"name": "evict_prefill", "op": "evict", "B": 16, "Hkv": 8, "d": 128, "page": 256, "shortest": 2048,
         "longest": 16384, "budget": 4096, "sinks": 4, "recent": 512},
        # one very long cache
        {"name": "evict_one_long", "op": "evict", "B": 1, "Hkv": 8, "d": 128, "page": 128, "shortest": 131072,
         "longest": 131072, "budget": 16384, "sinks": 16, "recent": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, pairs, axes):
    """`pairs` pairs over `axes` axes, one at least for each, as the axes' rotated dimensions."""
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return ",".join(str(2 * (b - a)) for a, b in zip([0] + cuts, cuts + [pairs]))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "evict"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8])
    H = Hkv * rng.choice([1, 2, 4, 4, 5, 8])
    pairing = rng.choice(["adjacent", "halves"])
    pairs = rng.choice([d // 2, d // 2, d // 4])
    axis_dims = _split(rng, pairs, rng.choice([1, 1, 2, 3]))
    far = rng.choice([0, 0, 100000, 1000000])
    if op == "rope":
        B = rng.choice([1, 1, 2, 3])
        S = _log(rng, 1, max(2, 786240 // (B * (H + Hkv))))
        return {"op": op, "B": B, "S": S, "H": H, "Hkv": Hkv, "d": d, "layout": rng.choice(["bshd", "bhsd"]),
                "axis_dims": axis_dims, "pairing": pairing, "backward": rng.random() < 0.5,
                "fused": rng.random() < 0.3, "far": far}
    page = rng.choice([16, 24, 64, 128, 256])
    if op == "append":
        return {"op": op, "B": _log(rng, 1, 64), "new": _log(rng, 1, 128), "H": H, "Hkv": Hkv, "d": d, "page": page,
                "longest": _log(rng, 600, 4096), "axis_dims": axis_dims, "pairing": pairing, "far": far}
    if op == "decode":
        B = _log(rng, 1, 64)
        longest = _log(rng, 8, 16384)
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "page": page, "shortest": rng.randint(1, longest),
                "longest": longest, "weights": rng.random() < 0.5}
    B = _log(rng, 1, 16)
    longest = _log(rng, 64, 16384)
    budget = rng.randint(max(8, longest // 8), longest)
    return {"op": op, "B": B, "Hkv": Hkv, "d": d, "page": page, "shortest": max(1, longest // 2), "longest": longest,
            "budget": budget, "sinks": rng.randint(0, budget // 8), "recent": rng.randint(0, budget // 2)}


# ------------------------------------------------------------------------------------- inputs
def _frequencies(axis_dims):
    """Radians per unit of position of each rotated pair, and the axis whose position it takes."""
    dims = [int(n) for n in axis_dims.split(",")]
    freqs = [10000.0 ** (-2.0 * i / n) for n in dims for i in range(n // 2)]
    axes = [a for a, n in enumerate(dims) for _ in range(n // 2)]
    return freqs, axes, len(dims)


def _lengths(case, g):
    n = torch.randint(case["shortest"], case["longest"] + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)
    n[0] = case["longest"]
    return n


def _cache(case, g, longest):
    """Keys, values and the block table: every table entry is a page of its own, in a shuffled order."""
    most = -(-longest // case["page"])
    pages = case["B"] * most
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(case["B"], most)
    shape = (pages, case["page"], case["Hkv"], case["d"])
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    return k, v, table


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    normal = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    s = dict(case)
    if case["op"] in ("rope", "append"):
        freqs, axes, n = _frequencies(case["axis_dims"])
        s["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
        s["axes"] = torch.tensor(axes, dtype=torch.int32, device="cuda")
    if case["op"] == "rope":
        H, S = case["H"], case["S"]
        # the grid's positions (or a text's), the same for every sequence of the batch
        at = torch.arange(S, device="cuda")
        side = max(1, math.isqrt(S))
        s["positions"] = torch.stack([at // (side ** (n - 1 - a)) % (side if a else S) + case["far"]
                                      for a in range(n)]).to(torch.int32)
        if case["fused"]:   # views of one projection's output
            x = normal(B, S, H + 2 * Hkv, d)
            q, k = x[:, :, :H], x[:, :, H:H + Hkv]
        else:
            q, k = normal(B, S, H, d), normal(B, S, Hkv, d)
        if case["layout"] == "bhsd":
            q, k = q.transpose(1, 2), k.transpose(1, 2)
            if not case["fused"]:
                q, k = q.contiguous(), k.contiguous()
        s["q"], s["k"] = q, k
    elif case["op"] == "append":
        H = case["H"]
        new = torch.randint(max(1, case["new"] // 2), case["new"] + 1, (B,), generator=g, device="cuda")
        new[0] = case["new"]
        total = B * case["new"]     # the program's token budget; rows past the last sequence's are not used
        s["cu"] = torch.cat([new.new_zeros(1), new.cumsum(0)]).to(torch.int32)
        s["lens"] = (new + torch.randint(0, case["longest"] - case["new"] + 1, (B,), generator=g, device="cuda")).to(torch.int32)
        x = normal(total, H + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        s["q_out"] = torch.zeros((total, H, d), dtype=torch.bfloat16, device="cuda")
        s["k_cache"], s["v_cache"], s["table"] = _cache(case, g, case["longest"])
        s["positions"] = (torch.randint(0, 4096, (n, total), generator=g, device="cuda") + case["far"]).to(torch.int32)
    else:
        s["lens"] = _lengths(case, g)
        s["k_cache"], s["v_cache"], s["table"] = _cache(case, g, case["longest"])
        room = s["table"].shape[1] * case["page"]
        held = torch.arange(room, device="cuda") < s["lens"][:, None, None]
        if case["op"] == "decode":
            s["q"] = normal(B, case["H"], d) * 2      # logits of deviation 2: some keys stand out
            # weights that earlier tokens left
            s["weights"] = torch.rand((B, Hkv, room), generator=g, device="cuda") * held if case["weights"] else None
        else:
            # a few keys hold most of the weight, and many have none yet
            w = torch.empty((B, Hkv, room), device="cuda").exponential_(generator=g) ** 3
            s["weights"] = w * (torch.rand((B, Hkv, room), generator=g, device="cuda") < 0.9) * held
            s["weights_out"] = torch.zeros_like(w)
            s["lens_out"] = torch.zeros_like(s["lens"])
    return s


# ------------------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, pairing):
    """x [..., d] rotated by angles whose cosines and sines are [..., pairs]."""
    x = x.float()
    n = cos.shape[-1]
    if pairing == "adjacent":
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * n:]], -1).to(torch.bfloat16)


def _angles(s):
    """Cosines and sines [tokens, pairs] of the positions, from angles in 64 bits."""
    angle = s["positions"][s["axes"].long()].double().T * s["freqs"]
    return angle.cos().float(), angle.sin().float()


def _plain_rope(s):
    cos, sin = _angles(s)
    if s["backward"]:
        sin = -sin
    if s["layout"] == "bshd":
        cos, sin = cos[:, None], sin[:, None]
    return [_rotate(s["q"], cos, sin, s["pairing"]), _rotate(s["k"], cos, sin, s["pairing"])]


def _plain_append(s):
    cos, sin = (t[:, None] for t in _angles(s))
    total = s["q"].shape[0]
    token = torch.arange(total, device="cuda")
    cu = s["cu"].long()
    b = torch.searchsorted(cu, token, right=True) - 1
    used = b < s["B"]
    b = b.clamp(max=s["B"] - 1)
    at = s["lens"].long()[b] - cu[b + 1] + token
    slot = s["table"].long()[b, torch.where(used, at, 0) // s["page"]] * s["page"] + at % s["page"]
    # a token past the last sequence writes what the first one does
    slot = torch.where(used, slot, slot[0])
    row = torch.where(used, token, 0)
    k = _rotate(s["k"], cos, sin, s["pairing"])
    s["k_cache"].view(-1, s["Hkv"], s["d"])[slot] = k[row]
    s["v_cache"].view(-1, s["Hkv"], s["d"])[slot] = s["v"][row]
    s["q_out"].copy_(torch.where(used[:, None, None], _rotate(s["q"], cos, sin, s["pairing"]), s["q_out"]))
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _plain_decode(s):
    B, Hkv, d = s["B"], s["Hkv"], s["d"]
    table = s["table"].long()
    k = s["k_cache"][table].flatten(1, 2).float()
    v = s["v_cache"][table].flatten(1, 2).float()
    q = s["q"].float().view(B, Hkv, -1, d)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(d)
    seen = torch.arange(k.shape[1], device="cuda") < s["lens"][:, None, None, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    p = e / total
    o = torch.matmul(p, v.transpose(1, 2)).view(B, -1, d).to(torch.bfloat16)
    lse = (top + torch.log(total)).view(B, -1)
    if s["weights"] is None:
        return [o, lse]
    s["weights"] += p.sum(2)
    return [o, lse, s["weights"]]


def _plain_evict(s):
    B, Hkv, room, budget, sinks, recent = s["B"], s["Hkv"], s["weights"].shape[2], s["budget"], s["sinks"], s["recent"]
    n = s["lens"].long()[:, None, None]
    at = torch.arange(room, device="cuda").expand(B, Hkv, room)
    over = n > budget
    old = (at >= sinks) & (at < n - recent)
    order = torch.sort(torch.where(old, s["weights"], -1.0), dim=2, descending=True, stable=True).indices
    best = torch.zeros((B, Hkv, room), dtype=torch.bool, device="cuda")
    best.scatter_(2, order[:, :, :budget - sinks - recent], True)
    kept = (at < sinks) | (best & old)
    end = budget - recent
    hole = ~kept & (at < end)
    late = kept & (at >= end) & (at < n - recent)
    # the i-th survivor past the end goes to the i-th hole; the recent keys follow in order
    survivors = torch.sort(torch.where(late, at, room), dim=2).values
    rank = torch.cumsum(hole, 2) - 1
    source = torch.where(hole, survivors.gather(2, rank.clamp(min=0)), at)
    source = torch.where((at >= end) & (at < budget), n - budget + at, source)
    source = torch.where(over, source, at).clamp(max=room - 1)
    upto = min(budget, room)
    slots = (s["table"].long()[:, :, None] * s["page"] + torch.arange(s["page"], device="cuda")).flatten(1)
    rows = slots[:, None].expand(B, Hkv, room).gather(2, source)[:, :, :upto]
    heads = torch.arange(Hkv, device="cuda")[None, :, None]
    to = slots[:, None, :upto].expand(B, Hkv, upto)
    k, v = s["k_cache"].view(-1, Hkv, s["d"]), s["v_cache"].view(-1, Hkv, s["d"])
    k[to, heads] = k[rows, heads]
    v[to, heads] = v[rows, heads]
    s["lens_out"].copy_(s["lens"].clamp(max=budget))
    w = torch.where(at < s["lens_out"][:, None, None], s["weights"].gather(2, source), 0.0)
    s["weights_out"].copy_(w)
    return [s["lens_out"], s["weights_out"], s["k_cache"], s["v_cache"]]


def run(s):
    if own:
        import bf16_attention_forward_gb300 as attn
        if s["op"] == "rope":
            call = attn.attn_rope_bwd if s["backward"] else attn.attn_rope
            return list(call(s["q"], s["k"], s["positions"], s["freqs"], s["axes"], layout=s["layout"],
                             pairing=s["pairing"]))
        if s["op"] == "append":
            attn.attn_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["cu"], s["lens"], s["table"],
                                   q=s["q"], q_out=s["q_out"], positions=s["positions"], freqs=s["freqs"],
                                   axes=s["axes"], pairing=s["pairing"])
            return [s["q_out"], s["k_cache"], s["v_cache"]]
        if s["op"] == "decode":
            o, lse = attn.attn_paged_decode(s["q"], s["k_cache"], s["v_cache"], s["lens"], s["table"],
                                            weights=s["weights"], return_lse=True)
            return [o, lse] if s["weights"] is None else [o, lse, s["weights"]]
        attn.attn_paged_evict(s["k_cache"], s["v_cache"], s["weights"], s["lens"], s["table"], s["budget"],
                              sinks=s["sinks"], recent=s["recent"], seqlens_out=s["lens_out"],
                              weights_out=s["weights_out"])
        return [s["lens_out"], s["weights_out"], s["k_cache"], s["v_cache"]]
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}[s["op"]](s)


# ------------------------------------------------------------------------------------- work
def work(case):
    """Each input read once and each output written once.  Lengths are drawn between `shortest` and
    `longest`, new tokens between half and all of `new`: their means stand for them.  Of an eviction's keys
    the recent ones of every cache that is over its budget have to move; the others' moves depend on the
    weights, and of the survivors the share that lies past the new end is counted."""
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    row = 2 * d
    if case["op"] == "rope":
        n = B * case["S"] * (case["H"] + Hkv)
        axes = case["axis_dims"].count(",") + 1
        return {"bytes": 2 * n * row + 4 * axes * case["S"], "flops": 3 * n * d}
    if case["op"] == "append":
        n = B * (max(1, case["new"] // 2) + case["new"]) / 2
        axes = case["axis_dims"].count(",") + 1
        return {"bytes": n * (2 * (case["H"] + 2 * Hkv) * row + 4 * axes), "flops": 3 * n * (case["H"] + Hkv) * d}
    lo, hi = case["shortest"], case["longest"]
    if case["op"] == "decode":
        n = B * (lo + hi) / 2
        return {"bytes": 2 * n * Hkv * row + 2 * B * case["H"] * row + (8 * n * Hkv if case["weights"] else 0),
                "flops": 4 * n * case["H"] * d}
    budget, sinks, recent = case["budget"], case["sinks"], case["recent"]
    moved = held = 0.0
    for i in range(101):
        n = lo + (hi - lo) * i / 100
        held += min(n, budget) / 101
        if n > budget:
            kept, old = budget - sinks - recent, n - sinks - recent
            moved += (recent + kept * (1 - kept / old if old > 0 else 0)) / 101
    return {"bytes": B * Hkv * (4 * (lo + hi) / 2 + 4 * held + moved * 4 * row), "flops": B * Hkv * (lo + hi) / 2}


# ------------------------------------------------------------------------------------- 64 bits
def _exact_rotate(x, positions, case):
    """[tokens, heads, d] in 64 bits, pair by pair."""
    freqs, axes, _ = _frequencies(case["axis_dims"])
    sign = -1.0 if case.get("backward") else 1.0
    y = x.double().clone()
    n = len(freqs)
    for p, (f, a) in enumerate(zip(freqs, axes)):
        i, j = (2 * p, 2 * p + 1) if case["pairing"] == "adjacent" else (p, p + n)
        z = torch.polar(torch.ones_like(positions[a], dtype=torch.float64), sign * f * positions[a].double())[:, None]
        turned = torch.complex(x[..., i].double(), x[..., j].double()) * z
        y[..., i], y[..., j] = turned.real, turned.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        out = []
        for x in (s["q"], s["k"]):
            x = x if case["layout"] == "bshd" else x.transpose(1, 2)
            y = torch.stack([_exact_rotate(x[b], s["positions"], case) for b in range(B)])
            out.append(y if case["layout"] == "bshd" else y.transpose(1, 2))
        return out
    lens = s["lens"].tolist()
    page = case["page"]
    if case["op"] == "append":
        cu, table = s["cu"].tolist(), s["table"].tolist()
        q, k = (_exact_rotate(s[x], s["positions"], case) for x in ("q", "k"))
        out = [s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()]
        out[0][:cu[B]] = q[:cu[B]]
        for b in range(B):
            done = cu[b]
            while done < cu[b + 1]:     # page by page
                at = lens[b] - cu[b + 1] + done
                n = min(page - at % page, cu[b + 1] - done)
                to = (table[b][at // page], slice(at % page, at % page + n))
                out[1][to], out[2][to] = k[done:done + n], s["v"][done:done + n].double()
                done += n
        return out
    if case["op"] == "decode":
        G = case["H"] // Hkv
        o = torch.empty((B, case["H"], d), dtype=torch.float64, device="cuda")
        lse = torch.empty((B, case["H"]), dtype=torch.float64, device="cuda")
        weights = None if s["weights"] is None else s["weights"].double()
        for b, n in enumerate(lens):
            ids = s["table"][b, :-(-n // page)].long()
            k, v = (s[c].index_select(0, ids).flatten(0, 1)[:n].double() for c in ("k_cache", "v_cache"))
            for h in range(Hkv):
                heads = slice(h * G, (h + 1) * G)
                x = (k[:, h] @ s["q"][b, heads].double().T) * d ** -0.5
                lse[b, heads] = torch.logsumexp(x, 0)
                p = (x - lse[b, heads]).exp()
                o[b, heads] = p.T @ v[:, h]
                if weights is not None:
                    weights[b, h, :n] += p.sum(1)
        return [o, lse] if weights is None else [o, lse, weights]
    budget, sinks, recent = case["budget"], case["sinks"], case["recent"]
    w_in, w_out = s["weights"].cpu(), torch.zeros(s["weights"].shape, dtype=torch.float64)
    k, v, table = s["k_cache"], s["v_cache"], s["table"].cpu()
    at = torch.arange(table.shape[1] * page)
    for b, n in enumerate(lens):
        slots = table[b].long()[at // page] * page + at % page
        for h in range(Hkv):
            source = list(range(min(n, budget)))
            if n > budget:
                w = w_in[b, h].tolist()
                ranked = sorted(range(sinks, n - recent), key=lambda j: (-w[j], j))
                survivors = set(range(sinks)) | set(ranked[:budget - sinks - recent])
                late = iter(sorted(j for j in survivors if j >= budget - recent))
                source = [j if j in survivors else next(late) for j in range(budget - recent)] + list(range(n - recent, n))
                to, rows = slots[:budget].cuda(), slots[torch.tensor(source)].cuda()
                for c in (k, v):
                    flat = c.view(-1, Hkv, d)
                    flat[to, h] = flat[rows, h]
            w_out[b, h, :len(source)] = w_in[b, h][torch.tensor(source)].double()
    return [None, w_out, k.double(), v.double()]
