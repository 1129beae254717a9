"""Pages and slots of a step's tokens (attn_paged_reserve) against a plain loop (needs a GB300)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SITE = 25


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import bf16_attention_forward_gb300 as a
    a.load()
    return a


def plain(lens, cu, table, held, free, count, page, total, shared=None):
    """The step on copies of numpy arrays: (table, held, free, count, slots, positions)."""
    table, free, held = table.copy(), free.copy(), held.copy()
    B = len(lens)
    want = [max(-(-int(lens[b]) // page), 0 if shared is None else int(shared[b])) for b in range(B)]
    for b in range(B):
        for i in range(want[b], held[b]):
            free[count] = table[b, i]
            count += 1
    for b in range(B):
        for i in range(held[b], want[b]):
            count -= 1
            table[b, i] = free[count]
    slots, positions = np.full(total, -1, np.int64), np.zeros(total, np.int32)
    for b in range(B):
        for t in range(cu[b], cu[b + 1]):
            j = int(lens[b]) - int(cu[b + 1]) + t
            positions[t] = j
            slots[t] = int(table[b, j // page]) * page + j % page
    return table, np.array(want, np.int32), free, count, slots, positions


def make(seed, B, page, longest, new, ended=0.0, spare=0, shared=0, start=0, capacity=None):
    """A state: sequences of up to `longest` keys, some with pages to spare, some that have ended."""
    g = np.random.default_rng(seed)
    old = g.integers(0, longest + 1, B)
    old = np.where(g.random(B) < 0.2, 0, old)
    news = g.integers(0, new + 1, B)
    end = g.random(B) < ended
    room = shared + -(-(longest + new) // page) + spare
    held = np.minimum(shared + -(-old // page) + g.integers(0, spare + 1, B), room)
    ids = g.permutation(B * room + shared + 8)
    table = np.full((B, room), -5, np.int32)
    table[:, :shared] = ids[:shared]
    at = shared
    for b in range(B):
        n = held[b] - shared
        table[b, shared:held[b]] = ids[at:at + n]
        at += n
    left = ids[at:]
    free = np.full(len(ids) if capacity is None else capacity, -9, np.int32)
    free[:len(left)] = left
    news = np.where(end, 0, news)
    lens = np.where(end, 0, old + shared * page + news)
    cu = np.concatenate([[start], start + np.cumsum(news)]).astype(np.int32)
    return dict(lens=lens.astype(np.int32), cu=cu, table=table, held=held.astype(np.int32), free=free, count=len(left),
                page=page, total=int(cu[-1]) + 5, shared=np.full(B, shared, np.int32) if shared else None)


def call(attn, s, out_of_place=False):
    t = {n: torch.as_tensor(s[n]).cuda() for n in ("lens", "cu", "table", "held", "free")}
    count = torch.tensor([s["count"]], dtype=torch.int32, device="cuda")
    shared = None if s["shared"] is None else torch.as_tensor(s["shared"]).cuda()
    kw = {}
    if out_of_place:
        kw = dict(held_out=torch.full_like(t["held"], 77), count_out=torch.full_like(count, 77))
    slots, positions = attn.attn_paged_reserve(t["lens"], t["cu"], t["table"], t["held"], t["free"], count, s["page"],
                                               total=s["total"], shared_pages=shared, **kw)
    held, n = kw.get("held_out", t["held"]), kw.get("count_out", count)
    if out_of_place:
        assert np.array_equal(t["held"].cpu(), s["held"]) and int(count) == s["count"]
    return t["table"].cpu().numpy(), held.cpu().numpy(), t["free"].cpu().numpy(), int(n), slots.cpu().numpy(), positions.cpu().numpy()


def same(got, want):
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


CASES = [  # B, page size, longest, new, ended, spare, shared, start
    (1, 16, 0, 1, 0.0, 0, 0, 0),
    (1, 1, 5, 3, 0.0, 0, 0, 2),
    (7, 16, 100, 1, 0.0, 0, 0, 0),
    (33, 24, 300, 5, 0.2, 3, 0, 7),
    (64, 128, 2000, 40, 0.5, 2, 3, 0),
    (256, 16, 500, 1, 0.1, 0, 0, 0),
    (1000, 7, 60, 2, 0.3, 4, 1, 0),
    (1023, 3, 20, 3, 0.3, 1, 0, 0),
    (1025, 16, 90, 2, 0.1, 1, 2, 0),
    (4095, 5, 30, 2, 0.2, 1, 0, 0),
    (5000, 5, 30, 2, 0.2, 1, 1, 3),
    (3, 256, 4000, 9000, 0.0, 0, 0, 0),
    (50, 1, 10, 700, 0.1, 50, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_a_plain_loop(attn, case):
    for seed in range(3):
        s = make(seed, *case)
        want = plain(s["lens"], s["cu"], s["table"], s["held"], s["free"], s["count"], s["page"], s["total"], s["shared"])
        same(call(attn, s, out_of_place=seed == 1), want)
    assert attn.cache_device_status() == (0, 0)


def test_all_come_back_and_the_same_pages_go_out(attn):
    """Every free page is taken, returned ones among them, in the stack's order."""
    s = make(5, 40, 8, 200, 0, spare=4)
    s["lens"] = s["lens"][::-1].copy()               # other sequences' lengths: some shrink, some grow
    missing = sum(max(-(-int(n) // 8) - int(h), 0) for n, h in zip(s["lens"], s["held"]))
    back = sum(max(int(h) - -(-int(n) // 8), 0) for n, h in zip(s["lens"], s["held"]))
    assert missing > 0 and back > 0
    s["count"] = max(missing - back, 0)
    want = plain(s["lens"], s["cu"], s["table"], s["held"], s["free"], s["count"], 8, s["total"])
    same(call(attn, s), want)
    s["count"] = missing - back - 1 if missing > back else 0
    if missing > back:
        got = call(attn, s)
        assert attn.cache_device_status() == (1, SITE)
        same(got[:4], (s["table"], s["held"], s["free"], s["count"]))


def broken(kind):
    s = make(3, 20, 16, 200, 40, ended=0.2, spare=2, shared=1)
    if kind == "negative length":
        s["lens"][4] = -1
    elif kind == "length past the table":
        s["lens"][4] = s["table"].shape[1] * 16 + 1
    elif kind == "more new tokens than length":
        b = int(np.argmax(np.diff(s["cu"])))
        s["lens"][b] = np.diff(s["cu"])[b] - 1
    elif kind == "falling offsets":
        s["cu"][5] = s["cu"][7] + 1
    elif kind == "negative offset":
        s["cu"][0] = -1
    elif kind == "offsets past the tokens":
        s["total"] = int(s["cu"][-1]) - 1
    elif kind == "negative pages":
        s["held"][2] = -1
    elif kind == "too many pages":
        s["held"][2] = s["table"].shape[1] + 1
    elif kind == "shared past held":
        s["shared"][2] = s["held"][2] + 1
    elif kind == "negative shared":
        s["shared"][2] = -1
    elif kind == "count past the stack":
        s["count"] = len(s["free"]) + 1
    elif kind == "negative count":
        s["count"] = -1
    elif kind == "no room for what comes back":
        s["lens"][:] = 0
        s["cu"][:] = 0
        s["free"] = s["free"][:s["count"] + 3].copy()
    elif kind == "too few pages":                    # every sequence to its table's end, one page short
        s["lens"][:] = s["table"].shape[1] * 16
        s["count"] = int((s["table"].shape[1] - s["held"]).sum()) - 1
    return s


@pytest.mark.parametrize("kind", ["negative length", "length past the table", "more new tokens than length", "falling offsets",
                                  "negative offset", "offsets past the tokens", "negative pages", "too many pages",
                                  "shared past held", "negative shared", "count past the stack", "negative count",
                                  "no room for what comes back", "too few pages"])
def test_all_or_nothing(attn, kind):
    s = broken(kind)
    got = call(attn, s, out_of_place=True)
    assert attn.cache_device_status() == (1, SITE)
    same(got, (s["table"], s["held"], s["free"], s["count"], np.full(s["total"], -1), np.zeros(s["total"])))
    got = call(attn, s)                              # in place too
    assert attn.cache_device_status() == (1, SITE)
    same(got[:4], (s["table"], s["held"], s["free"], s["count"]))


def test_long_cache_slots_pass_31_bits(attn):
    """Slots are 64 bits: page numbers are taken as they are."""
    s = make(1, 3, 1000, 5000, 100)
    s["free"][:s["count"]] += 2 ** 24
    s["table"][s["table"] >= 0] += 2 ** 24
    want = plain(s["lens"], s["cu"], s["table"], s["held"], s["free"], s["count"], 1000, s["total"])
    assert want[4].max() > 2 ** 32
    same(call(attn, s), want)


def test_no_tokens_and_a_given_slots_tensor(attn):
    s = make(2, 9, 16, 100, 0, ended=0.5, spare=1)
    s["total"] = 0
    want = plain(s["lens"], s["cu"], s["table"], s["held"], s["free"], s["count"], 16, 0)
    same(call(attn, s)[:4], want[:4])
    s = make(2, 9, 16, 100, 5)
    t = {n: torch.as_tensor(s[n]).cuda() for n in ("lens", "cu", "table", "held", "free")}
    count = torch.tensor([s["count"]], dtype=torch.int32, device="cuda")
    slots = torch.full((s["total"] + 2,), 55, dtype=torch.int64, device="cuda")
    got, positions = attn.attn_paged_reserve(t["lens"], t["cu"], t["table"], t["held"], t["free"], count, 16, slots=slots[1:-1])
    want = plain(s["lens"], s["cu"], s["table"], s["held"], s["free"], s["count"], 16, s["total"])
    assert np.array_equal(got.cpu(), want[4]) and np.array_equal(positions.cpu(), want[5])
    assert int(slots[0]) == 55 and int(slots[-1]) == 55


def test_a_captured_loop(attn):
    """Lengths grow on the GPU; one graph reserves step after step, and never gives one page to two sequences."""
    B, page, most, steps = 17, 4, 12, 40
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    held, free = torch.zeros_like(lens), torch.randperm(B * most, device="cuda").to(torch.int32)
    count = torch.tensor([B * most], dtype=torch.int32, device="cuda")
    slots, positions = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        lens.add_(1)
        attn.attn_paged_reserve(lens, cu, table, held, free, count, page, slots=slots, positions=positions)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = set(slots.tolist())
    for i in range(1, steps):
        graph.replay()
        assert positions.tolist() == [i] * B
        now = slots.tolist()
        assert len(set(now)) == B and not seen & set(now)
        seen |= set(now)
    assert len(seen) == B * steps and int(count) == B * most - B * (steps // page)
    assert attn.cache_device_status() == (0, 0)


@pytest.mark.parametrize("page", [1, 4])
def test_a_negative_page_is_no_padding(attn, page):
    """Tokens on a held page that is not there: no slot of theirs is -1, and the call that writes them reports it."""
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, cu, held = torch.tensor([page], **i32), torch.tensor([0, page], **i32), torch.tensor([1], **i32)
    table, free, count = torch.full((1, 2), -1, **i32), torch.zeros(3, **i32), torch.tensor([0], **i32)
    slots, positions = attn.attn_paged_reserve(lens, cu, table, held, free, count, page, total=page)
    assert attn.cache_device_status() == (0, 0)
    assert slots.tolist() == [-2] * page and positions.tolist() == list(range(page))
    k = torch.ones(page, 1, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(3, page, 1, 64, dtype=torch.bfloat16, device="cuda")
    attn.attn_norm_rope_append(k, k, cache, cache.clone(), slots)
    assert attn.cache_device_status()[1] == 24 and not cache.any()
