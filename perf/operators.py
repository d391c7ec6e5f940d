"""What the paged-cache operators are measured on, with their plain forms.

The operators serve generate() for many requests at once: a key/value cache
cut into pages that requests take from a common ring, the append that fills
it, decode attention that reads it, and decode attention over the pages
that a cheap score selects.

  plan    attn_paged_plan     block tables, slots and positions from lengths
  append  attn_cache_append   new K and V rows into their slots, and the
                              pages' channel bounds
  decode  attn_decode_paged   the newest Tq positions against their pages
  select  attn_page_select    the pages whose bounds promise the largest scores
  sparse  attn_decode_sparse  decode attention over the selected pages
"""

import math
import random

import torch

own = False

BF16 = torch.bfloat16
DEV = "cuda"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch: most requests add a token, a few end
        # and a few begin
        dict(name="plan_step_b64", op="plan", B=64, P=16, longest=1024, tokens=1, width=80),
        # admission of many prompts at once
        dict(name="plan_prompts_b256", op="plan", B=256, P=16, longest=4000, tokens=500, width=512),
        # the new tokens of one decode step of the GPT-2 124M layer
        dict(name="append_step_b16_h12_d64", op="append", B=16, Hkv=12, D=64, P=16, tokens=1,
             start=700, extra=12),
        # prompts, K and V read in place from a fused projection with grouped heads
        dict(name="append_prompts_h8_d128", op="append", B=24, Hkv=8, D=128, P=32, tokens=683,
             start=77, extra=32),
        # one short chat with the char-level model: the latency of a call
        dict(name="decode_b1_h6_l250_d64", op="decode", B=1, Hkv=6, G=1, Tq=1, D=64, P=16,
             shortest=250, longest=250),
        # the GPT-2 124M layer, requests at all stages up to its block size
        dict(name="decode_b16_h12_l1024_d64", op="decode", B=16, Hkv=12, G=1, Tq=1, D=64, P=16,
             shortest=60, longest=1024),
        # a full batch of ragged requests with grouped heads
        dict(name="decode_b64_h32kv8_l8192_d128", op="decode", B=64, Hkv=8, G=4, Tq=1, D=128, P=16,
             shortest=512, longest=8192),
        # one very long document, several new tokens checked in one call
        dict(name="decode_b1_h32kv8_l131071_tq4", op="decode", B=1, Hkv=8, G=4, Tq=4, D=128, P=64,
             shortest=131071, longest=131071),
        # page selection for one long request
        dict(name="select_b1_h16_l8192_d128", op="select", B=1, Hkv=16, G=1, Tq=1, D=128, P=16,
             shortest=8192, longest=8192, K=64),
        # page selection for a batch of long requests
        dict(name="select_b16_h32kv8_l32768", op="select", B=16, Hkv=8, G=4, Tq=1, D=128, P=16,
             shortest=9000, longest=32768, K=128),
        # attention over the selected pages of one request
        dict(name="sparse_b2_h16_k64_d128", op="sparse", B=2, Hkv=16, G=1, Tq=1, D=128, P=16,
             shortest=5000, longest=8192, K=64),
        # and of a batch of long requests
        dict(name="sparse_b16_h32kv8_k128", op="sparse", B=16, Hkv=8, G=4, Tq=1, D=128, P=16,
             shortest=9000, longest=32768, K=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


LARGEST = 7e8  # bytes that a drawn case's caches or new rows may have


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode", "select", "sparse"])
    P = rng.choice([8, 16, 16, 20, 32, 64, 128])
    D = rng.choice([16, 32, 64, 64, 128, 128])
    G = rng.choice([1, 1, 2, 3, 4, 5, 8])
    Hkv = rng.choice([1, 2, 3, 5, 6, 8, 8, 12, 16, 25])
    if op == "plan":
        B = _log(rng, 1, 512)
        longest, tokens = _log(rng, 16, 4000), _log(rng, 1, max(2, min(1000, 120000 // B)))
        return dict(op=op, B=B, P=P, longest=longest, tokens=tokens,
                    width=(longest + 2 * tokens) // P + 2 + rng.randrange(40))
    if op == "append":
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, Hkv=Hkv, D=D, P=P, tokens=_log(rng, 1, max(2, min(2000, 16000 // B))),
                    start=rng.randrange(1500), extra=Hkv * rng.choice([1, 1, 2, 4]))
    if op == "decode":
        B = _log(rng, 1, 256)
        per = Hkv * D * 4
        longest = _log(rng, 1, max(16, min(131072, int(LARGEST / per / B))))
        return dict(op=op, B=B, Hkv=Hkv, G=G, Tq=rng.choice([1, 1, 1, 2, 4, 5, 8]), D=D, P=P,
                    shortest=_log(rng, 1, longest), longest=longest)
    B = _log(rng, 1, 64)
    longest = _log(rng, 4 * P, max(5 * P, min(65536, int(LARGEST / (Hkv * D * 4) / B))))
    return dict(op=op, B=B, Hkv=Hkv, G=G, Tq=rng.choice([1, 1, 1, 2, 4]), D=D, P=P,
                shortest=_log(rng, 1, longest), longest=longest,
                K=max(4, min(256, _log(rng, 4, max(5, longest // P)))))


def _lengths(case):
    """B lengths from shortest to longest, evenly on a logarithmic scale."""
    lo, hi, B = case["shortest"], case["longest"], case["B"]
    if B == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (B - 1)))) for i in range(B)]


def _plan_requests(case):
    """(cached length, new tokens) of B requests: of every eight one ends
    (-1), one begins, and one idles; the others go on."""
    out = []
    for i in range(case["B"]):
        n = case["tokens"] + (i * 7) % (case["tokens"] + 1) if case["tokens"] > 1 else 1
        length = 1 + (i * 977) % case["longest"]
        kind = i % 8
        out.append((length, -1) if kind == 3 else (0, n) if kind == 5 else
                   (length, 0) if kind == 6 else (length, n))
    return out


def _pages(n, P):
    return -(-n // P)


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std)


def _shuffled(values, seed):
    values = list(values)
    random.Random(seed).shuffle(values)
    return values


def _table(g, counts, width, n_pages):
    """A block table whose rows hold disjoint pages in random order, -1 behind."""
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    c = torch.tensor(counts, device=DEV)
    first = torch.cumsum(c, 0) - c
    j = torch.arange(width, device=DEV)[None, :]
    at = (first[:, None] + j).clamp(max=n_pages - 1)
    used = int(sum(counts))
    return torch.where(j < c[:, None], order[at], -1).to(torch.int32).contiguous(), order[used:]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    return globals()["_prepare_" + case["op"]](case, int(seed), g)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _prepare_plan(case, seed, g):
    P, B = case["P"], case["B"]
    req = _shuffled(_plan_requests(case), seed)
    counts = [_pages(length, P) for length, _ in req]
    need = sum(_pages(length + n, P) - _pages(length, P) for length, n in req if n > 0)
    n_pages = sum(counts) + need + 7
    width = max(case["width"], max(_pages(length + max(n, 0), P) for length, n in req))
    table, free = _table(g, counts, width, n_pages)
    head = seed % n_pages  # the ring has been in use: its first free page is anywhere
    ring = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(len(free), device=DEV)) % n_pages] = free
    tokens = sum(n for _, n in req if n > 0)
    slots = tokens + 5
    return dict(op="plan", P=P, new=_i32([n for _, n in req]), lengths=_i32([n for n, _ in req]),
                table=table, ring=ring, n_slots=slots,
                state=torch.tensor([head, head + len(free)], dtype=torch.int64, device=DEV),
                lengths_out=_i32([0] * B), cu=_i32([0] * (B + 1)), status=_i32([0]),
                state_out=torch.zeros(2, dtype=torch.int64, device=DEV),
                slots=torch.zeros(slots, dtype=torch.int64, device=DEV),
                positions=torch.zeros(slots, dtype=torch.int32, device=DEV))


def _prepare_append(case, seed, g):
    B, Hkv, D, P, n = (case[k] for k in ("B", "Hkv", "D", "P", "tokens"))
    starts = _shuffled([case["start"] + i for i in range(B)], seed)
    counts = [_pages(s + n, P) for s in starts]
    n_pages = sum(counts) + 3
    table, _ = _table(g, counts, max(counts), n_pages)
    pos = torch.tensor(starts, device=DEV)[:, None] + torch.arange(n, device=DEV)[None, :]
    slots = table.gather(1, pos // P).long() * P + pos % P
    # rows of a fused projection [q heads | k heads | v heads]
    fused = _randn(g, B * n, (case["extra"] + 2 * Hkv) * D).to(BF16)
    rows = fused.view(B * n, case["extra"] + 2 * Hkv, D)
    caches = [_randn(g, n_pages, P, Hkv, D).to(BF16).transpose(1, 2) for _ in range(2)]
    lo = _randn(g, n_pages, Hkv, 1, D)
    bounds = torch.cat([lo, lo + _randn(g, n_pages, Hkv, 1, D).abs()], 2).to(BF16)
    return dict(op="append", P=P, k_new=rows[:, case["extra"]:case["extra"] + Hkv],
                v_new=rows[:, case["extra"] + Hkv:], k=caches[0], v=caches[1],
                slots=slots.reshape(-1).contiguous(), bounds=bounds)


def _prepare_decode(case, seed, g):
    B, Hkv, G, Tq, D, P = (case[k] for k in ("B", "Hkv", "G", "Tq", "D", "P"))
    lengths = _shuffled(_lengths(case), seed)
    counts = [_pages(n, P) for n in lengths]
    n_pages = sum(counts) + 2
    table, _ = _table(g, counts, max(counts) + 3, n_pages)
    caches = [_randn(g, n_pages, P, Hkv, D).to(BF16).transpose(1, 2) for _ in range(2)]
    q = _randn(g, B, Tq, Hkv * G, D, std=1.5).to(BF16).transpose(1, 2)
    return dict(op="decode", P=P, q=q, k=caches[0], v=caches[1], table=table,
                lengths=_i32(lengths), scale=D ** -0.5, **_outputs(q))


def _outputs(q):
    B, H, Tq, D = q.shape
    return dict(o=torch.empty(B, Tq, H, D, dtype=BF16, device=DEV).transpose(1, 2),
                lse=torch.empty(B, H, Tq, dtype=torch.float32, device=DEV), keep={})


def _prepare_select(case, seed, g):
    B, Hkv, G, Tq, D, P = (case[k] for k in ("B", "Hkv", "G", "Tq", "D", "P"))
    lengths = _shuffled(_lengths(case), seed)
    counts = [_pages(n, P) for n in lengths]
    n_pages = sum(counts) + 2
    table, _ = _table(g, counts, max(counts) + 1, n_pages)
    # neighbouring keys are alike: a page's channels spread around its own centre
    mid, wide = _randn(g, n_pages, Hkv, 1, D), _randn(g, n_pages, Hkv, 2, D, std=0.6).abs()
    bounds = torch.cat([mid - wide[:, :, :1], mid + wide[:, :, 1:]], 2).to(BF16)
    q = _randn(g, B, Tq, Hkv * G, D).to(BF16).transpose(1, 2)
    return dict(op="select", P=P, K=case["K"], q=q, bounds=bounds, table=table,
                lengths=_i32(lengths), keep={},
                pages=torch.empty(B, Hkv, case["K"], dtype=torch.int32, device=DEV))


def _prepare_sparse(case, seed, g):
    s = _prepare_decode(case, seed, g)
    B, Hkv, K = case["B"], case["Hkv"], case["K"]
    count = -(-s["lengths"].long() // case["P"])
    width = s["table"].shape[1]
    # K of each request's pages at random, the last one among them, ascending
    mark = torch.rand(B, Hkv, width, generator=g, device=DEV)
    j = torch.arange(width, device=DEV)
    mark = torch.where(j == (count - 1)[:, None, None], 2.0, mark)
    mark = torch.where(j < count[:, None, None], mark, -1.0)
    top = mark.sort(-1, descending=True).indices[..., :K]
    if top.shape[-1] < K:
        top = torch.nn.functional.pad(top, (0, K - top.shape[-1]), value=width)
    top = torch.where(top < count[:, None, None], top, 1 << 30).sort(-1).values
    s.update(op="sparse", pages=torch.where(top < (1 << 30), top, -1).to(torch.int32))
    return s


# --------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return globals()["_plain_" + state["op"]](state)


def _run_own(s):
    import causal_self_attention_flash_b200 as cattn
    if s["op"] == "plan":
        cattn.attn_paged_plan(s["new"], s["lengths"], s["table"], s["ring"], s["state"], s["P"],
                              s["n_slots"], lengths_out=s["lengths_out"],
                              ring_state_out=s["state_out"], cu_new=s["cu"], slots=s["slots"],
                              positions=s["positions"], status=s["status"])
        return _plan_outputs(s)
    if s["op"] == "append":
        cattn.attn_cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["slots"], s["bounds"])
        return dict(k=s["k"], v=s["v"], bounds=s["bounds"])
    if s["op"] == "select":
        B, Hkv = s["q"].shape[0], s["bounds"].shape[1]
        if "ws" not in s["keep"]:  # a workspace that the program keeps
            n = cattn.attn_page_select_workspace_bytes(B, Hkv, s["table"].shape[1])
            s["keep"]["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        cattn.attn_page_select(s["q"], s["bounds"], s["table"], s["lengths"], s["P"], s["K"],
                               n_first=1, n_last=1, pages=s["pages"], workspace=s["keep"]["ws"])
        return s["pages"]
    B, H, Tq, D = s["q"].shape
    if "ws" not in s["keep"]:
        n = cattn.attn_decode_paged_workspace_bytes(B, H, s["k"].shape[1], Tq, D)
        s["keep"]["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    if s["op"] == "decode":
        cattn.attn_decode_paged(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["scale"],
                                o=s["o"], lse=s["lse"], workspace=s["keep"]["ws"])
    else:
        cattn.attn_decode_sparse(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["pages"],
                                 s["scale"], o=s["o"], lse=s["lse"], workspace=s["keep"]["ws"])
    return dict(o=s["o"], lse=s["lse"])


def _plan_outputs(s):
    return {k: s[k] for k in ("lengths_out", "state_out", "cu", "slots", "positions", "status",
                              "table", "ring")}


def _plain_plan(s):
    P, table, ring = s["P"], s["table"], s["ring"]
    n_pages, B = ring.numel(), table.shape[0]
    length, asked = s["lengths"].long(), s["new"].long()
    n = asked.clamp(min=0)
    have = -(-length // P)
    need = -(-(length + n) // P) - have
    back = torch.where(asked < 0, have, 0)
    head, tail = s["state"][0], s["state"][1]
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    first_need, first_back = need.cumsum(0) - need, back.cumsum(0) - back
    # the pages of the requests that end, behind the ring's tail
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    old = table.clone()
    at = torch.where(j < back[:, None], (tail + first_back[:, None] + j) % n_pages, n_pages)
    more = torch.cat([ring, ring.new_zeros(1)]).scatter_(0, at.reshape(-1), old.reshape(-1))
    # new pages from the ring's head
    mine = (j >= have[:, None]) & (j < (have + need)[:, None])
    taken = ring[(head + first_need[:, None] + j - have[:, None]) % n_pages]
    table.copy_(torch.where(mine, taken, old))
    ring.copy_(more[:n_pages])
    # slots and positions of the new tokens, -1 behind the last
    i = torch.arange(s["n_slots"], device=DEV)
    r = torch.searchsorted(cu[1:], i, right=True)
    live, r = r < B, r.clamp(max=B - 1)
    pos = length[r] + i - cu[r]
    slot = table[r, (pos // P).clamp(0, table.shape[1] - 1)].long() * P + pos % P
    s["slots"].copy_(torch.where(live, slot, -1))
    s["positions"].copy_(torch.where(live, pos, -1))
    s["cu"].copy_(cu)
    s["lengths_out"].copy_(torch.where(asked < 0, 0, length + n))
    s["state_out"].copy_(torch.stack([head + need.sum(), tail + back.sum()]))
    s["status"].zero_()
    return _plan_outputs(s)


def _plain_append(s):
    P, slots = s["P"], s["slots"]
    n_pages, Hkv, D = s["k"].shape[0], s["k"].shape[1], s["k"].shape[3]
    page, off = slots // P, slots % P
    s["k"].transpose(1, 2)[page, off] = s["k_new"]
    s["v"].transpose(1, 2)[page, off] = s["v_new"]
    # a page whose first row is new starts over, another one goes on
    fresh = torch.zeros(n_pages, dtype=torch.bool, device=DEV)
    fresh[page[off == 0]] = True
    old = s["bounds"].float()
    lo = torch.where(fresh[:, None, None], math.inf, old[:, :, 0])
    hi = torch.where(fresh[:, None, None], -math.inf, old[:, :, 1])
    at = page[:, None, None].expand(-1, Hkv, D)
    k = s["k_new"].float()
    lo = lo.scatter_reduce(0, at, k, "amin")
    hi = hi.scatter_reduce(0, at, k, "amax")
    s["bounds"].copy_(torch.stack([lo, hi], 2))
    return dict(k=s["k"], v=s["v"], bounds=s["bounds"])


def _attend(s, k, v, position):
    """k, v (B, Hkv, N, D) and the keys' positions (B, 1 or Hkv, N), negative where none."""
    B, H, Tq, D = s["q"].shape
    Hkv = k.shape[1]
    q = s["q"].float().reshape(B, Hkv, H // Hkv * Tq, D)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    last = (s["lengths"][:, None] - Tq + torch.arange(Tq, device=DEV)[None, :]).repeat(1, H // Hkv)
    seen = (position[:, :, None, :] >= 0) & (position[:, :, None, :] <= last[:, None, :, None])
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total == 0, 1.0, total)
    s["o"].copy_(o.reshape(B, H, Tq, D))
    s["lse"].copy_((m + torch.log(total)).reshape(B, H, Tq))
    return dict(o=s["o"], lse=s["lse"])


def _plain_decode(s):
    P, table = s["P"], s["table"].long()
    n_pages, Hkv, _, D = s["k"].shape
    B, width = table.shape
    held = (table >= 0) & (table < n_pages)
    at = table.clamp(0, n_pages - 1)
    k, v = (c[at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * P, D).float()
            for c in (s["k"], s["v"]))
    j = torch.arange(width * P, device=DEV)[None, :]
    ok = held.repeat_interleave(P, 1) & (j < s["lengths"][:, None])
    return _attend(s, k, torch.where(ok[:, None, :, None], v, 0.0),
                   torch.where(ok, j, -1)[:, None])


def _plain_sparse(s):
    P, table, pages = s["P"], s["table"].long(), s["pages"].long()
    n_pages, Hkv, _, D = s["k"].shape
    B, _, K = pages.shape
    phys = table.gather(1, pages.clamp(0, table.shape[1] - 1).reshape(B, -1)).reshape(B, Hkv, K)
    held = (pages >= 0) & (phys >= 0) & (phys < n_pages)
    at = phys.clamp(0, n_pages - 1)
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    k, v = (c[at, head].reshape(B, Hkv, K * P, D).float() for c in (s["k"], s["v"]))
    pos = (pages[..., None] * P + torch.arange(P, device=DEV)).reshape(B, Hkv, K * P)
    ok = held.repeat_interleave(P, 2) & (pos < s["lengths"][:, None, None])
    return _attend(s, k, torch.where(ok[..., None], v, 0.0), torch.where(ok, pos, -1))


def _plain_select(s):
    P, K, table = s["P"], s["K"], s["table"].long()
    B, H, Tq, D = s["q"].shape
    n_pages, Hkv = s["bounds"].shape[:2]
    width = table.shape[1]
    # 64 bits: two pages' scores may be next to each other
    q = s["q"].double().reshape(B, Hkv, H // Hkv * Tq, D)
    b = s["bounds"][table.clamp(0, n_pages - 1)].permute(0, 2, 3, 4, 1).double()
    x = (torch.matmul(q.clamp(min=0), b[:, :, 1]) + torch.matmul(q.clamp(max=0), b[:, :, 0])).amax(2)
    held = (table >= 0) & (table < n_pages)
    x = torch.where(held[:, None], x, -math.inf)
    count = (-(-s["lengths"].long() // P)).clamp(max=width)[:, None, None]
    j = torch.arange(width, device=DEV)
    # the first and the last page are always taken, none behind the last
    rank = torch.where((j < 1) | (j >= count - 1), 1, 0)
    rank = torch.where(j < count, rank, -1)
    order = x.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, rank.expand(x.shape).gather(-1, order).sort(
        dim=-1, descending=True, stable=True).indices)
    top = torch.nn.functional.pad(order[..., :K], (0, max(0, K - width)), value=width)
    top = torch.where(top < count, top, 1 << 30).sort(-1).values
    s["pages"].copy_(torch.where(top < (1 << 30), top, -1))
    return s["pages"]


# -------------------------------------------------------------- exact, work

def exact(case, seed):
    if case["op"] in ("plan", "select"):  # whole numbers
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    B, H, Tq, D = s["q"].shape
    n_pages, Hkv = s["k"].shape[:2]
    P, G = s["P"], H // s["k"].shape[1]
    o = torch.zeros(B, H, Tq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device=DEV)
    lengths, table = s["lengths"].tolist(), s["table"].tolist()
    chosen = s["pages"].tolist() if case["op"] == "sparse" else None
    for b in range(B):
        for h in range(Hkv):
            logical = chosen[b][h] if chosen else range(_pages(lengths[b], P))
            logical = [p for p in logical if 0 <= p < _pages(lengths[b], P)]
            at = torch.tensor([table[b][p] for p in logical], device=DEV, dtype=torch.long)
            pos = (torch.tensor(logical, device=DEV, dtype=torch.long)[:, None] * P
                   + torch.arange(P, device=DEV)).reshape(-1)
            k = s["k"][at, h].reshape(-1, D)[pos < lengths[b]].double()
            v = s["v"][at, h].reshape(-1, D)[pos < lengths[b]].double()
            pos = pos[pos < lengths[b]]
            for t in range(Tq):
                n = (pos <= lengths[b] - Tq + t)
                if lengths[b] - Tq + t < 0 or not len(pos):
                    continue
                x = s["q"][b, h * G:(h + 1) * G, t].double() @ k[n].T * s["scale"]
                lse[b, h * G:(h + 1) * G, t] = torch.logsumexp(x, -1)
                o[b, h * G:(h + 1) * G, t] = torch.softmax(x, -1) @ v[n]
    return dict(o=o, lse=lse)


def _exact_append(s):
    P, k, v, bounds = s["P"], s["k"].double(), s["v"].double(), s["bounds"].double()
    slots = s["slots"]
    started = torch.unique(slots[slots % P == 0] // P)
    for page in torch.unique(slots // P).tolist():
        rows = ((slots // P) == page).nonzero()[:, 0]
        off = slots[rows] % P
        new = s["k_new"][rows].double()
        k[page][:, off] = new.transpose(0, 1)
        v[page][:, off] = s["v_new"][rows].double().transpose(0, 1)
        lo, hi = new.amin(0), new.amax(0)
        if not bool((started == page).any()):
            lo, hi = torch.minimum(lo, bounds[page, :, 0]), torch.maximum(hi, bounds[page, :, 1])
        bounds[page, :, 0], bounds[page, :, 1] = lo, hi
    return dict(k=k, v=v, bounds=bounds)


def work(case):
    op, P, B = case["op"], case["P"], case["B"]
    if op == "plan":
        req = _plan_requests(case)
        new = [(length, n) for length, n in req if n > 0]
        pages = sum(_pages(length + n, P) - _pages(length, P) for length, n in new)
        back = sum(_pages(length, P) for length, n in req if n < 0)
        tokens = sum(n for _, n in new)
        # lengths and counts in, lengths and offsets out; a page read and
        # written for each taken or given back; a slot and a position a token
        return dict(bytes=16 * B + 8 * (pages + back) + 12 * tokens + 36, flops=0)
    if op == "append":
        n, row = B * case["tokens"], case["Hkv"] * case["D"] * 2
        touched = sum(_pages(case["start"] + i + case["tokens"], P) - (case["start"] + i) // P
                      for i in range(B))
        return dict(bytes=4 * n * row + 8 * n + 2 * touched * row, flops=2 * n * row)
    Hkv, D, rows = case["Hkv"], case["D"], case["G"] * case["Tq"]
    lengths = _lengths(case)
    io = B * Hkv * rows * (4 * D + 4)
    if op == "decode":
        keys = sum(lengths) * Hkv
        return dict(bytes=keys * D * 4 + io + 4 * sum(_pages(n, P) for n in lengths),
                    flops=4 * keys * D * rows)
    if op == "select":
        pages = sum(_pages(n, P) for n in lengths if _pages(n, P) > case["K"]) * Hkv
        return dict(bytes=pages * D * 4 + io // 2 + 4 * B * Hkv * case["K"],
                    flops=4 * pages * D * rows)
    keys = sum(min(n, case["K"] * P) for n in lengths) * Hkv
    return dict(bytes=keys * D * 4 + io + 8 * B * Hkv * case["K"], flops=4 * keys * D * rows)
