"""GPU tests of the paged key/value cache: attn_paged_plan, attn_cache_append,
attn_decode_paged, attn_page_select and attn_decode_sparse against the fp64
oracle, and a run of them together as a server uses them."""

import numpy as np
import pytest
import torch

import oracle.paged as opaged
from paged_util import as64, check_decode, make_table, poison_unread, rows
from test_paged_emu import plan_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x)).to(dtype).to(DEV)


def setup(seed, lengths, Hkv, G, Tq, D, P, spare=0, holes=(), nhd=True):
    """(q, k, v on the CPU, k, v views on the device, table)"""
    width = max(1, max(opaged.n_pages_of(n, P) for n in lengths) + spare)
    n_pages = max(1, sum(min(opaged.n_pages_of(n, P), width) for n in lengths) + 1)
    table = make_table(seed, lengths, P, width, n_pages)
    for (b, i), page in holes:
        table[b, i] = page
    k, v = (rows(seed + s, n_pages, Hkv, P, D) for s in (1, 2))
    poison_unread(k, v, table, lengths, P)
    kd, vd = (x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) if nhd else x.to(DEV)
              for x in (k, v))
    q = rows(seed + 3, len(lengths), Hkv * G, Tq, D, std=1.5)
    return q, k, v, kd, vd, table


def run_case(lib, seed, lengths, Hkv, G, Tq, D, P, spare=0, holes=(), nhd=True, pages=None):
    q, k, v, kd, vd, table = setup(seed, lengths, Hkv, G, Tq, D, P, spare, holes, nhd)
    scale = np.float32(D ** -0.5)
    args = (q.to(DEV), kd, vd, dev(table), dev(lengths))
    # a workspace with garbage in it
    n = lib.attn_decode_paged_workspace_bytes(len(lengths), Hkv * G, Hkv, Tq, D)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV)
    if pages is None:
        o, lse = lib.attn_decode_paged(*args, scale=scale, workspace=ws)
    else:
        o, lse = lib.attn_decode_sparse(*args, dev(pages), scale=scale, workspace=ws)
    torch.cuda.synchronize()
    ref = opaged.decode(as64(q), as64(k), as64(v), table, lengths, scale, pages)
    check_decode(as64(o.cpu()), as64(lse.cpu()), ref, max(1, max(lengths)), D)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("P", [16, 20, 1, 64])
@pytest.mark.parametrize("G,Tq", [(1, 1), (4, 1), (3, 3), (8, 4)])
def test_decode(lib, D, P, G, Tq):
    run_case(lib, D + P, [1, 0, 300, 17, Tq, 64, 129], 2, G, Tq, D, P, spare=1, nhd=P != 20)


@pytest.mark.parametrize("lengths,Hkv,G,Tq,D,P", [
    ([1], 1, 1, 1, 64, 16),                    # one key
    ([9000], 1, 1, 1, 128, 16),                # one item over every warp
    ([4097], 1, 16, 1, 64, 32),                # 16 query heads on one
    ([3000, 5], 1, 5, 8, 64, 48),              # 40 rows: three tiles
    ([700 + 13 * i for i in range(20)], 3, 1, 1, 64, 16),
    ([(i * 53) % 90 for i in range(700)], 2, 2, 1, 32, 16),
    ([(i * 7) % 23 for i in range(5000)], 1, 1, 1, 16, 8),   # 40 requests per thread of the scan
    ([20000, 9001], 2, 5, 4, 64, 16),          # 20 rows: two tiles, cut over many CTAs
    ([12000, 0, 7, 12345], 1, 2, 1, 16, 16),   # one short and one empty item among cut ones
])
def test_decode_shapes(lib, lengths, Hkv, G, Tq, D, P):
    run_case(lib, 5, lengths, Hkv, G, Tq, D, P)


def test_decode_pages_that_are_not_held(lib):
    holes = [((0, 0), -1), ((0, 3), 10 ** 6), ((1, 2), -7), ((2, 0), 1 << 30), ((2, 1), -1)]
    run_case(lib, 6, [200, 90, 20], 2, 4, 1, 64, 16, holes=holes)
    run_case(lib, 6, [200, 90, 20], 2, 4, 5, 128, 16, holes=holes)


@pytest.mark.parametrize("L", [3, 700, 20000])
@pytest.mark.parametrize("D,G,Tq", [(16, 1, 1), (32, 9, 1), (64, 3, 2), (128, 4, 1), (128, 5, 4)])
def test_decode_infinite_values(lib, L, D, G, Tq):
    """an infinite value that a row sees is its result (NaN where both signs
    meet), whatever the key's weight; other channels are as without it"""
    lengths, P = [L, 40], 16
    q, k, v, kd, vd, table = setup(11, lengths, 2, G, Tq, D, P)
    scale = np.float32(D ** -0.5)
    ref = opaged.decode(as64(q), as64(k), as64(v), table, lengths, scale)
    seen = max(1, L - Tq + 1)                      # keys that every row with a key sees
    for d, sign in ((0, 1), (1, -1), (2, 1), (3, -1)):
        pos = d * (seen - 1) // 3
        vd[table[0, pos // P], :, pos % P, d] = sign * float("inf")
    for pos, sign in ((0, 1), (seen - 1, -1)):
        vd[table[0, pos // P], :, pos % P, 7] = sign * float("inf")
    o, lse = lib.attn_decode_paged(q.to(DEV), kd, vd, dev(table), dev(lengths), scale=scale)
    o, lse = as64(o.cpu()), as64(lse.cpu())
    some = o[0][np.isfinite(lse[0])]                # rows with a key
    assert (some[:, [0, 2]] == np.inf).all() and (some[:, [1, 3]] == -np.inf).all()
    assert np.isnan(some[:, 7]).all() or seen == 1
    o[0][..., [0, 1, 2, 3, 7]] = ref[0][0][..., [0, 1, 2, 3, 7]]
    check_decode(o, lse, ref, L, D)


@pytest.mark.parametrize("L", [150, 9000])
@pytest.mark.parametrize("D,G,Tq", [(16, 1, 1), (64, 3, 2), (128, 9, 1)])
def test_decode_large_values(lib, L, D, G, Tq):
    """scores that rise by less than the running maximum follows, with values
    near the largest bf16: finite where the formula is"""
    q, k, v, kd, vd, table = setup(13, [L], 1, G, Tq, D, 16)
    q[..., 0], q[..., 1:] = 1, 0
    kd[..., 0] = 0
    k[..., 0] = 0
    for i, x in enumerate((5.25, 5.5, 5.375)):      # e^5.5 < 2^8
        pos = L - Tq - 2 + i
        for kk, vv in ((k, v), (kd, vd)):
            kk[table[0, pos // 16], 0, pos % 16, 0] = x
            vv[table[0, pos // 16], 0, pos % 16, :] = 3e38 * (-1) ** i
            vv[table[0, pos // 16], 0, pos % 16, 1::2] = 1.5e38
    ref = opaged.decode(as64(q), as64(k), as64(v), table, [L], 1.0)
    o, lse = lib.attn_decode_paged(q.to(DEV), kd, vd, dev(table), dev([L]), scale=1.0)
    check_decode(as64(o.cpu()), as64(lse.cpu()), ref, L, D)


@pytest.mark.parametrize("D,G,Tq", [(64, 1, 1), (128, 4, 1), (128, 2, 3)])
def test_sparse(lib, D, G, Tq):
    rng = np.random.default_rng(D)
    lengths, P, K, Hkv = [1000, 130, 16, 0, 517], 16, 12, 3
    pages = np.full((len(lengths), Hkv, K), -1)
    for b, n in enumerate(lengths):
        for h in range(Hkv):
            count = min(K, opaged.n_pages_of(n, P))
            pages[b, h, :count] = np.sort(rng.permutation(opaged.n_pages_of(n, P))[:count])
    pages[0, 0, 3] = 1000                      # lists nothing
    run_case(lib, 8, lengths, Hkv, G, Tq, D, P, pages=pages)


def test_sparse_long_lists(lib):
    """more listed keys than one cluster takes: the flat kernel"""
    rng = np.random.default_rng(1)
    B, Hkv, P, K = 40, 4, 16, 200
    lengths = [5000 if b % 3 else 100 + b for b in range(B)]
    pages = np.full((B, Hkv, K), -1)
    for b, n in enumerate(lengths):
        count = opaged.n_pages_of(n, P)
        for h in range(Hkv):
            some = np.sort(rng.permutation(count)[:K])
            pages[b, h, :len(some)] = some
    run_case(lib, 12, lengths, Hkv, 2, 1, 64, P, pages=pages)


def test_two_calls_at_once(lib):
    """calls on two streams, each with its own workspace, give the bits of a
    call alone"""
    cases = []
    for seed, lengths, Hkv, G, D in ((1, [30000], 2, 4, 128), (2, [900, 4000, 70], 4, 1, 64)):
        q, _, _, kd, vd, table = setup(seed, lengths, Hkv, G, 1, D, 16)
        args = (q.to(DEV), kd, vd, dev(table), dev(lengths))
        want = [x.clone() for x in lib.attn_decode_paged(*args)]
        ws = torch.empty(lib.attn_decode_paged_workspace_bytes(len(lengths), Hkv * G, Hkv, 1, D),
                         dtype=torch.uint8, device=DEV)
        cases.append((args, want, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        for args, want, ws, stream in cases:
            with torch.cuda.stream(stream):
                got.append((lib.attn_decode_paged(*args, workspace=ws), want))
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in got:
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_decode_matches_the_contiguous_cache(lib):
    """one request, its pages in order: attn_decode on the same cache"""
    H, L, D, P, Tq = 3, 400, 64, 16, 2
    k, v, q = (rows(s, 1, H, n, D).to(DEV) for s, n in ((1, L), (2, L), (3, Tq)))
    pool = [x[0].view(H, L // P, P, D).transpose(0, 1) for x in (k, v)]
    table = torch.arange(L // P, dtype=torch.int32, device=DEV)[None]
    o, lse = lib.attn_decode_paged(q, *pool, table, dev([L]))
    o2, lse2 = lib.attn_decode(q, k, v, L)
    torch.cuda.synchronize()
    assert torch.allclose(lse, lse2, atol=1e-5, rtol=0)
    # both round o; attn_decode rounds its weights to bf16 too (2^-8 of a sum |v| <~ 1)
    assert (o.float() - o2.float()).abs().max().item() < 2 * 2.0 ** -8


def test_strides_outputs_and_repeats(lib):
    """q and o as parts of wider rows, a table that is a part of a wider one,
    pages with gaps between heads; what lies between is left as it was; a
    second call gives the same bits"""
    B, Hkv, G, Tq, D, P = 3, 2, 3, 2, 64, 16
    lengths = [333, 16, 80]
    q, k, v, _, _, table = setup(4, lengths, Hkv, G, Tq, D, P)
    wide = torch.full((B, Tq, Hkv * G + 2, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :, 1:-1] = q.to(DEV).transpose(1, 2)
    pool = torch.full((k.shape[0], P + 1, Hkv, 3, D), float("nan"), dtype=torch.bfloat16,
                      device=DEV)
    pool[:, :P, :, 0] = k.to(DEV).transpose(1, 2)
    pool[:, :P, :, 2] = v.to(DEV).transpose(1, 2)
    tab = torch.full((B, table.shape[1] + 5), 99, dtype=torch.int32, device=DEV)
    tab[:, 2:2 + table.shape[1]] = dev(table)
    out = torch.full((B, Tq, Hkv * G + 2, D), 7.0, dtype=torch.bfloat16, device=DEV)
    args = (wide[:, :, 1:-1].transpose(1, 2), pool[:, :P, :, 0].transpose(1, 2),
            pool[:, :P, :, 2].transpose(1, 2), tab[:, 2:2 + table.shape[1]], dev(lengths))
    o = out[:, :, 1:-1].transpose(1, 2)
    _, lse = lib.attn_decode_paged(*args, o=o)
    ref = opaged.decode(as64(q), as64(k), as64(v), table, lengths, np.float32(D ** -0.5))
    check_decode(as64(o.cpu()), as64(lse.cpu()), ref, max(lengths), D)
    assert (out[:, :, 0] == 7).all() and (out[:, :, -1] == 7).all()
    o2, lse2 = lib.attn_decode_paged(*args)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("lengths,G,Tq,D", [([300, 41], 2, 1, 64), ([9000], 3, 2, 128)])
def test_k_and_v_in_different_layouts(lib, lengths, G, Tq, D):
    q, k, v, kd, vd, table = setup(14, lengths, 2, G, Tq, D, 16)
    gaps = torch.full((k.shape[0], 2, 16 + 3, D + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    gaps[:, :, :16, :D] = v.to(DEV)
    ref = opaged.decode(as64(q), as64(k), as64(v), table, lengths, np.float32(D ** -0.5))
    for kk, vv in ((kd, v.to(DEV)), (k.to(DEV), vd), (kd, gaps[:, :, :16, :D])):
        o, lse = lib.attn_decode_paged(q.to(DEV), kk, vv, dev(table), dev(lengths))
        check_decode(as64(o.cpu()), as64(lse.cpu()), ref, max(lengths), D)


def test_offsets_beyond_32_bits(lib):
    """a pool of more than 2^32 elements, read and written at its far end"""
    P, D, Hkv = 64, 128, 8
    n_pages = (1 << 32) // (P * D * Hkv) + 70
    pool = torch.empty(n_pages, P, Hkv, D, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    bounds = torch.zeros(n_pages, Hkv, 2, D, dtype=torch.bfloat16, device=DEV)
    L = 150
    table = np.array([[n_pages - 1, 0, n_pages - 33]], np.int32)
    kn, q = rows(1, L, Hkv, D), rows(2, 1, Hkv, 1, D)
    slots = [int(table[0, p // P]) * P + p % P for p in range(L)]
    lib.attn_cache_append(kn.to(DEV), kn.to(DEV), pool, pool, dev(slots, torch.int64), bounds)
    o, lse = lib.attn_decode_paged(q.to(DEV), pool, pool, dev(table), dev([L]))
    small = torch.zeros(3, Hkv, P, D, dtype=torch.bfloat16)
    for p in range(L):
        small[p // P, :, p % P] = kn[p]
    ref = opaged.decode(as64(q), as64(small), as64(small), np.array([[0, 1, 2]]), [L],
                        np.float32(D ** -0.5))
    check_decode(as64(o.cpu()), as64(lse.cpu()), ref, L, D)
    assert torch.equal(bounds[n_pages - 33, :, 0].cpu(), kn[2 * P:].amin(0))


# -------------------------------------------------------- plan and append

@pytest.mark.parametrize("B,P,longest,most", [
    (1, 16, 40, 1), (64, 16, 1000, 1), (33, 8, 60, 300), (1000, 16, 64, 3), (7, 1, 9, 4),
    (1, 16, 0, 40000), (8192, 16, 40, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(lib, B, P, longest, most, in_place):
    asked, lengths, table, ring, state = plan_inputs(B + P, B, P, longest, most)
    if B == 1:
        asked[:] = most
    n_slots = int(np.maximum(asked, 0).sum()) + 3
    want = opaged.plan(asked, lengths, table, ring, state, P, n_slots)
    ln, tb, rg, st = dev(lengths), dev(table), dev(ring), dev(state, torch.int64)
    more = dict(lengths_out=ln, ring_state_out=st) if in_place else {}
    got = lib.attn_paged_plan(dev(asked), ln, tb, rg, st, P, n_slots, **more)
    for key, x in zip(("lengths", "state", "cu", "slots", "positions"), got):
        assert np.array_equal(x.cpu().numpy(), want[key]), key
    assert int(got[5]) == want["status"] == opaged.OK
    assert np.array_equal(tb.cpu().numpy(), want["table"])
    assert np.array_equal(rg.cpu().numpy(), want["ring"])


@pytest.mark.parametrize("B,longest", [(40, 100), (3000, 600)])
def test_plan_frees_held_pages_only(lib, B, longest):
    """entries that are not held in the rows of requests that end do not get
    into the ring"""
    P = 8
    asked, lengths, table, ring, state = plan_inputs(12, B, P, longest, 2)
    rng = np.random.default_rng(1)
    for b in np.flatnonzero(asked < 0)[::2]:
        for i in rng.integers(0, table.shape[1], 5):
            table[b, i] = rng.choice([-1, len(ring), 2 ** 31 - 1, -2 ** 31])
    n_slots = int(np.maximum(asked, 0).sum())
    want = opaged.plan(asked, lengths, table, ring, state, P, n_slots)
    tb, rg = dev(table), dev(ring)
    got = lib.attn_paged_plan(dev(asked), dev(lengths), tb, rg, dev(state, torch.int64), P, n_slots)
    for key, x in zip(("lengths", "state", "cu", "slots", "positions"), got):
        assert np.array_equal(x.cpu().numpy(), want[key]), key
    assert int(got[5]) == want["status"] == opaged.OK
    assert np.array_equal(tb.cpu().numpy(), want["table"])
    assert np.array_equal(rg.cpu().numpy(), want["ring"])
    assert want["state"][1] - state[1] < sum(opaged.n_pages_of(n, P)
                                             for n, a in zip(lengths, asked) if a < 0)


def test_plan_refuses_as_a_whole(lib):
    asked, lengths, table, ring, state = plan_inputs(3, 40, 8, 50, 20)
    n = int(np.maximum(asked, 0).sum())
    tb, rg = dev(table), dev(ring)
    got = lib.attn_paged_plan(dev(asked), dev(lengths), tb, rg, dev(state, torch.int64), 8, n - 1)
    assert int(got[5]) == lib.ERR_TOO_LARGE
    assert np.array_equal(got[0].cpu().numpy(), lengths) and (got[3] == -1).all()
    assert np.array_equal(got[1].cpu().numpy(), state) and (got[2] == 0).all()
    assert np.array_equal(tb.cpu().numpy(), table) and np.array_equal(rg.cpu().numpy(), ring)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,P,runs", [
    (1, 16, [(5, 30)]), (3, 8, [(0, 20), (64, 1), (47, 17), (200, 3)]),
    (8, 16, [(1000 * i + i, 1) for i in range(40)]), (2, 20, [(7, 900)])])
def test_append(lib, D, Hkv, P, runs):
    slots = [s + i for s, n in runs for i in range(n)] + [-1, 10 ** 14]
    n_pages = max(slots[:-2]) // P + 2
    n = len(slots)
    kn, vn = rows(1, n, 2 * Hkv + 1, D)[:, :Hkv], rows(2, n, Hkv, D)
    k, v = rows(3, n_pages, Hkv, P, D), rows(4, n_pages, Hkv, P, D)
    lo = rows(5, n_pages, Hkv, 1, D)
    bd = torch.cat([lo, lo + 1], 2)
    f32 = lambda t: t.float().numpy()  # noqa: E731
    wk, wv, wb = opaged.append(f32(kn), f32(vn), slots, f32(k), f32(v), f32(bd))
    big = rows(1, n, 2 * Hkv + 1, D).to(DEV)           # k_new: a part of wider rows
    sl = dev(slots, torch.int64)
    for bounds in (None, bd.to(DEV)):
        kd, vd = k.to(DEV), v.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
        lib.attn_cache_append(big[:, :Hkv], vn.to(DEV), kd, vd, sl, bounds)
        assert np.array_equal(f32(kd.cpu()), wk) and np.array_equal(f32(vd.cpu()), wv)
        if bounds is not None:
            assert np.array_equal(f32(bounds.cpu()), wb)


# ----------------------------------------------------------------- select

def select_inputs(seed, lengths, Hkv, G, Tq, D, P, spare=0):
    width = max(opaged.n_pages_of(n, P) for n in lengths) + spare
    n_pages = sum(opaged.n_pages_of(n, P) for n in lengths) + 2
    table = make_table(seed, lengths, P, width, n_pages)
    mid = rows(seed + 1, n_pages, Hkv, 1, D).float()
    wide = rows(seed + 2, n_pages, Hkv, 2, D).float().abs()
    bounds = torch.cat([mid - wide[:, :, :1], mid + wide[:, :, 1:]], 2).to(torch.bfloat16)
    return rows(seed + 3, len(lengths), Hkv * G, Tq, D), bounds, table


@pytest.mark.parametrize("lengths,Hkv,G,Tq,D,P,K,n_first,n_last", [
    ([4000, 3, 0, 777], 1, 1, 1, 64, 4, 37, 1, 1),
    ([9000], 2, 4, 1, 128, 8, 128, 0, 0),
    ([700, 6400], 3, 2, 4, 32, 16, 8, 2, 3),
    ([333], 1, 1, 2, 16, 3, 2, 1, 1),
    ([5000, 100], 1, 16, 1, 128, 16, 50, 1, 1),
    ([1200], 1, 1, 1, 16, 4, 290, 1, 1)])
def test_select(lib, lengths, Hkv, G, Tq, D, P, K, n_first, n_last):
    q, bounds, table = select_inputs(2, lengths, Hkv, G, Tq, D, P, spare=2)
    got = lib.attn_page_select(q.to(DEV), bounds.to(DEV), dev(table), dev(lengths), P, K,
                               n_first=n_first, n_last=n_last)
    want = opaged.select(as64(q), as64(bounds), table, lengths, P, K, n_first, n_last)
    assert np.array_equal(got.cpu().numpy(), want)


def test_select_ties_nan_and_pages_that_are_not_held(lib):
    L, P, K, D = 900, 4, 30, 64
    q, bounds, table = select_inputs(3, [L], 1, 2, 1, D, P)

    def check(q, bounds, table):
        got = lib.attn_page_select(q.to(DEV), bounds.to(DEV), dev(table), dev([L]), P, K)
        want = opaged.select(as64(q), as64(bounds), table, [L], P, K, 1, 1)
        assert np.array_equal(got.cpu().numpy(), want)
    check(q, bounds[:1].expand_as(bounds).contiguous(), table)
    check(torch.zeros_like(q), bounds, table)
    check(q, bounds * 1e-30, table)             # scores far apart from one
    check(q * 1e15, bounds * 1e15, table)
    # scores that differ in the last bits of a sum only
    near = bounds[:1].expand_as(bounds).clone()
    near[:, :, :, 0] *= 1000
    near[:, :, :, 1] = (torch.arange(len(near)) % 61)[:, None, None].to(torch.bfloat16) * 2e-3
    check(q, near, table)
    bounds[table[0, 11], 0, 1, 5] = float("nan")
    bounds[table[0, 13]] = float("-inf")
    bounds[table[0, 17], 0, 1] = float("inf")
    bounds[table[0, 17], 0, 0] = 0
    table[0, 4], table[0, 8] = -1, 10 ** 6
    check(q, bounds, table)
    table[0, 1:220] = -1
    check(q, bounds, table)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_select_nan_in_a_page_that_is_always_taken(lib, bad):
    """NaN or infinite bounds of the first page: the others are chosen by their
    exact sums all the same, here pairs whose terms of 2^20 cancel"""
    P, D, Hkv, L = 4, 64, 16, 1200
    q, bounds, table = select_inputs(5, [L], Hkv, 1, 1, D, P)
    q[:] = 1
    bounds[:] = bounds.clamp(-0.01, 0.01)
    bounds[:, :, 1] = 0
    bounds[table[0, 0]] = bad
    for page in range(8, 300, 8):
        x = rows(page, Hkv, 5).abs() / 16
        for h in range(Hkv):
            hi = bounds[table[0, page], h, 1]
            hi[0], hi[40] = 2.0 ** 20, -2.0 ** 20
            hi[[3, 5, 18, 21, 30]] = x[h]
    tb, ln = dev(table), dev([L])
    wide = torch.full((1, 20000), -1, dtype=torch.int32, device=DEV)   # two launches
    wide[:, :table.shape[1]] = tb
    for K in (2, 9):
        want = opaged.select(as64(q), as64(bounds), table, [L], P, K, 1, 0)
        for t in (tb, wide):
            got = lib.attn_page_select(q.to(DEV), bounds.to(DEV), t, ln, P, K, n_last=0)
            assert np.array_equal(got.cpu().numpy(), want)


def test_select_sure_pages_beside_ties(lib):
    """sure pages in several warps and ties at the border, many heads at once
    and again and again: the choice is the oracle's each time"""
    L, P, K, D, Hkv = 1200, 4, 150, 64, 32
    q, bounds, table = select_inputs(4, [L], Hkv, 1, 1, D, P)
    bounds[:] = bounds[:1]
    for h in range(Hkv):
        q[0, h, 0] = bounds[0, h, 1]
        for i in range(3 + h, 300, 37 + h):
            bounds[table[0, i], h] *= 2 + h % 7
    bounds[:, :, 0] = 0
    want = opaged.select(as64(q), as64(bounds), table, [L], P, K, 1, 1)
    qd, bd, tb, ln = q.to(DEV), bounds.to(DEV), dev(table), dev([L])
    got = [lib.attn_page_select(qd, bd, tb, ln, P, K) for _ in range(50)]
    wide = torch.full((1, 20000), -1, dtype=torch.int32, device=DEV)   # two launches
    wide[:, :table.shape[1]] = tb
    got += [lib.attn_page_select(qd, bd, wide, ln, P, K) for _ in range(50)]
    for x in got:
        assert np.array_equal(x.cpu().numpy(), want)


# ---------------------------------------------------------- run together

class Server:
    """A cache and the oracle's copy of it, driven step by step."""

    def __init__(self, lib, B, Hkv, G, D, P, n_pages, width, seed):
        self.lib, self.Hkv, self.G, self.D, self.P = lib, Hkv, G, D, P
        z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
        self.pool = torch.full((2, n_pages, P, Hkv, D), float("nan"), dtype=torch.bfloat16,
                               device=DEV).transpose(2, 3)
        self.bounds = torch.full((n_pages, Hkv, 2, D), float("nan"), dtype=torch.bfloat16,
                                 device=DEV)
        self.lengths, self.table = z(B), z(B, width) - 1
        self.ring = torch.arange(n_pages, dtype=torch.int32, device=DEV)
        self.state = torch.tensor([0, n_pages], device=DEV)
        self.asked = z(B)
        self.seen = [[] for _ in range(B)]     # the oracle's (k, v) of each request
        self.seed = seed

    def step(self, asked, Tq=1, K=0):
        lib, B = self.lib, len(asked)
        total = int(sum(max(n, 0) for n in asked))
        self.seed += 1
        kn, vn = rows(self.seed, total, self.Hkv, self.D), rows(-self.seed, total, self.Hkv, self.D)
        q = rows(self.seed + 10 ** 6, B, self.Hkv * self.G, Tq, self.D, std=1.5)
        at = 0
        for b, n in enumerate(asked):
            if n < 0:
                self.seen[b] = []
            self.seen[b] += [(kn[at + i], vn[at + i]) for i in range(max(n, 0))]
            at += max(n, 0)
        _, _, _, slots, positions, status = lib.attn_paged_plan(
            dev(asked), self.lengths, self.table, self.ring, self.state, self.P, total,
            lengths_out=self.lengths, ring_state_out=self.state)
        lib.attn_cache_append(kn.to(DEV), vn.to(DEV), self.pool[0], self.pool[1], slots, self.bounds)
        args = (q.to(DEV), self.pool[0], self.pool[1], self.table, self.lengths)
        pages = None
        if K:
            pages = lib.attn_page_select(q.to(DEV), self.bounds, self.table, self.lengths, self.P, K)
            o, lse = lib.attn_decode_sparse(*args, pages)
        else:
            o, lse = lib.attn_decode_paged(*args)
        torch.cuda.synchronize()
        assert int(status) == 0
        self.check(q, o, lse, pages)

    def check(self, q, o, lse, pages):
        lengths = [len(s) for s in self.seen]
        assert self.lengths.tolist() == lengths
        P, n = self.P, [opaged.n_pages_of(x, self.P) for x in lengths]
        k = torch.zeros(max(1, sum(n)), self.Hkv, P, self.D, dtype=torch.bfloat16)
        v = torch.zeros_like(k)
        table = np.full((len(n), max(n + [1])), -1, np.int32)
        at = 0
        for b, s in enumerate(self.seen):
            for p, (kr, vr) in enumerate(s):
                table[b, p // P] = at + p // P
                k[at + p // P, :, p % P], v[at + p // P, :, p % P] = kr, vr
            at += n[b]
        listed = None
        if pages is not None:
            bounds = torch.zeros(len(k), self.Hkv, 2, self.D, dtype=torch.bfloat16)
            for b, s in enumerate(self.seen):
                for i in range(n[b]):
                    keys = torch.stack([kr for kr, _ in s[i * P:(i + 1) * P]])
                    bounds[table[b, i], :, 0], bounds[table[b, i], :, 1] = keys.amin(0), keys.amax(0)
            listed = opaged.select(as64(q), as64(bounds), table, lengths, P, pages.shape[2], 1, 1)
            assert np.array_equal(pages.cpu().numpy(), listed)
        ref = opaged.decode(as64(q), as64(k), as64(v), table, lengths,
                            np.float32(self.D ** -0.5), listed)
        check_decode(as64(o.cpu()), as64(lse.cpu()), ref, max(lengths + [1]), self.D)


def test_a_server_run(lib):
    """requests come, grow and end; their pages are used again"""
    s = Server(lib, 4, 2, 2, 64, 8, 40, 30, seed=100)
    s.step([30, 0, 7, 0])
    for _ in range(10):
        s.step([1, 0, 1, 0])
    s.step([1, 90, -1, 3], K=5)
    for i in range(6):
        s.step([1, 1, 0, 1], K=5 if i % 2 else 0)
    s.step([-1, 2, 80, 1], Tq=2, K=6)
    s.step([60, -1, 1, 1])
    s.step([1, 100, 1, 1], K=4)
    free = int(s.state[1] - s.state[0])
    held = sum(opaged.n_pages_of(len(x), 8) for x in s.seen)
    assert free + held == 40


def test_packed_steps(lib):
    """requests that bring prompts, go on, idle and end in one step: the plan's
    packed rows, and the newest of each request for the attention"""
    B, Hkv, G, D, P, n_pages, width = 6, 2, 2, 64, 8, 60, 20
    s = Server(lib, B, Hkv, G, D, P, n_pages, width, seed=500)
    for i, asked in enumerate(([20, 0, 7, 1, 0, 33], [1, 12, 0, -1, 9, 1], [0, 1, 1, 5, -1, 1],
                               [-1, 1, 0, 1, 0, 2])):
        total = sum(max(n, 0) for n in asked)
        q_new = rows(600 + i, total, Hkv * G, D, std=1.5)
        kn, vn = rows(700 + i, total, Hkv, D), rows(800 + i, total, Hkv, D)
        at = 0
        for b, n in enumerate(asked):
            s.seen[b] = [] if n < 0 else s.seen[b] + [(kn[at + j], vn[at + j]) for j in range(n)]
            at += max(n, 0)
        _, _, cu_new, slots, _, status = lib.attn_paged_plan(
            dev(asked), s.lengths, s.table, s.ring, s.state, P, total, lengths_out=s.lengths,
            ring_state_out=s.state)
        lib.attn_cache_append(kn.to(DEV), vn.to(DEV), s.pool[0], s.pool[1], slots, s.bounds)
        newest = (cu_new[1:] - 1).clamp(min=0).long()
        q = q_new.to(DEV)[newest].unsqueeze(2)
        o, lse = lib.attn_decode_paged(q, s.pool[0], s.pool[1], s.table, s.lengths)
        torch.cuda.synchronize()
        assert int(status) == 0
        ends = np.cumsum([max(n, 0) for n in asked]) - 1
        for b, n in enumerate(asked):
            if n > 0:
                assert torch.equal(q[b, :, 0].cpu(), q_new[ends[b]])
        s.check(q.cpu(), o, lse, None)


def test_a_captured_step(lib):
    """plan, append, decode, selection and sparse decode in one CUDA graph,
    replayed while the requests grow, against the same calls made eagerly;
    two graphs share the workspaces"""
    B, Hkv, G, D, P, n_pages, width, K = 5, 2, 4, 128, 16, 200, 40, 4
    start = [100, 15, 16, 300, 0]

    def state(seed):
        st = dict(lengths=dev([0] * B), table=torch.full((B, width), -1, dtype=torch.int32,
                                                         device=DEV),
                  ring=torch.arange(n_pages, dtype=torch.int32, device=DEV),
                  state=torch.tensor([0, n_pages], device=DEV), asked=dev([1] * B),
                  pool=torch.zeros(2, n_pages, P, Hkv, D, dtype=torch.bfloat16,
                                   device=DEV).transpose(2, 3),
                  bounds=torch.zeros(n_pages, Hkv, 2, D, dtype=torch.bfloat16, device=DEV),
                  qkv=torch.zeros(B, Hkv * G + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV))
        got = lib.attn_paged_plan(dev(start), st["lengths"], st["table"], st["ring"], st["state"],
                                  P, sum(start), lengths_out=st["lengths"],
                                  ring_state_out=st["state"])
        x = rows(seed, sum(start), 2 * Hkv, D).to(DEV)
        lib.attn_cache_append(x[:, :Hkv], x[:, Hkv:], st["pool"][0], st["pool"][1], got[3],
                              st["bounds"])
        return st

    ws = torch.empty(max(lib.attn_decode_paged_workspace_bytes(B, Hkv * G, Hkv, 1, D),
                         lib.attn_page_select_workspace_bytes(B, Hkv, width)),
                     dtype=torch.uint8, device=DEV)

    def step(st):
        _, _, _, slots, _, _ = lib.attn_paged_plan(
            st["asked"], st["lengths"], st["table"], st["ring"], st["state"], P, B,
            lengths_out=st["lengths"], ring_state_out=st["state"])
        q = st["qkv"][:, :Hkv * G].unsqueeze(2)
        k, v = st["qkv"][:, Hkv * G:-Hkv], st["qkv"][:, -Hkv:]
        lib.attn_cache_append(k, v, st["pool"][0], st["pool"][1], slots, st["bounds"])
        args = (q, st["pool"][0], st["pool"][1], st["table"], st["lengths"])
        a = lib.attn_decode_paged(*args, workspace=ws)
        pages = lib.attn_page_select(q, st["bounds"], st["table"], st["lengths"], P, K,
                                     workspace=ws)
        return (*a, pages, *lib.attn_decode_sparse(*args, pages, workspace=ws))

    def feed(st, i):
        st["qkv"].copy_(rows(5000 + i, B, Hkv * G + 2 * Hkv, D).to(DEV))

    eager, graphs = state(1), [state(1), state(1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    captured = []
    for st in graphs:
        keep = {k: t.clone() for k, t in st.items()}
        with torch.cuda.stream(side):
            step(st)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = step(st)
        torch.cuda.synchronize()
        for k, t in keep.items():
            st[k].copy_(t)
        captured.append((g, out))
    for i in range(20):
        feed(eager, i)
        want = step(eager)
        for st, (g, out) in zip(graphs, captured):
            feed(st, i)
            g.replay()
        torch.cuda.synchronize()
        for _, out in captured:
            for x, y in zip(want, out):
                assert torch.equal(x, y), i
    assert eager["lengths"].tolist() == [n + 20 for n in start]


class LongWay:
    """TORCH_CALLS that recognises nothing."""

    def __getattr__(self, name):
        return lambda *args: -1


def test_both_ways_into_the_library(lib, monkeypatch):
    """the calls through TORCH_CALLS and the long way give the same bits"""
    lengths, Hkv, G, D, P, K = [300, 40, 77], 2, 3, 64, 16, 4
    q, k, v, kd, vd, table = setup(3, lengths, Hkv, G, 1, D, P)
    bounds = rows(8, k.shape[0], Hkv, 2, D).sort(2).values.to(DEV)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    x = rows(9, 4, 2 * Hkv, D).to(DEV)
    wide = torch.full((3, table.shape[1] + 3), -1, dtype=torch.int32, device=DEV)
    wide[:, 1:-2] = dev(table)

    def everything():
        kc, vc, bd = kd.clone(), vd.clone(), bounds.clone()
        tb = wide[:, 1:-2]
        o = torch.empty(3, 1, Hkv * G, D, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
        lse, pages = torch.empty(3, Hkv * G, 1, device=DEV), dev(np.zeros((3, Hkv, K)))
        out = [dev([0] * 3), dev([0, 0], torch.int64), dev([0] * 4), dev([0] * 5, torch.int64),
               dev([0] * 5), dev([7])]
        lib.attn_paged_plan(dev([1, 2, -1]), dev([30, 7, 40]), wide.clone()[:, 1:-2],
                            dev(range(9)), dev([0, 5], torch.int64), P, 5, *out)
        lib.attn_cache_append(x[:, :Hkv], x[:, Hkv:], kc, vc, dev([5, 6, 32, -1], torch.int64), bd)
        lib.attn_decode_paged(q.to(DEV), kc, vc, tb, dev(lengths), 0.2, o, lse, ws)
        got = [*out, kc, vc, bd, o.clone(), lse.clone()]
        lib.attn_page_select(q.to(DEV), bd, tb, dev(lengths), P, K, 1, 1, pages, ws)
        lib.attn_decode_sparse(q.to(DEV), kc, vc, tb, dev(lengths), pages, None, o, lse, ws)
        return got + [pages, o, lse]

    a = everything()
    monkeypatch.setattr(lib, "TORCH_CALLS", LongWay())
    for x1, x2 in zip(a, everything()):
        assert torch.equal(x1.nan_to_num(3.0), x2.nan_to_num(3.0))


def test_refusals_before_anything_runs(lib):
    """wrong types, shapes, devices and sizes, through both ways"""
    lengths = [30, 20]
    q, _, _, kd, vd, table = setup(3, lengths, 2, 2, 1, 64, 16)
    qd, tb, ln = q.to(DEV), dev(table), dev(lengths)
    o, lse = torch.full_like(qd, 5.0), torch.full((2, 4, 1), 5.0, device=DEV)
    ws = torch.empty(lib.attn_decode_paged_workspace_bytes(2, 4, 2, 1, 64), dtype=torch.uint8,
                     device=DEV)
    good = dict(q=qd, k_cache=kd, v_cache=vd, block_table=tb, lengths=ln, o=o, lse=lse,
                workspace=ws)
    for name, bad in [("q", qd.float()), ("q", qd.cpu()), ("q", qd[0]), ("k_cache", kd.float()),
                      ("v_cache", vd[:-1]), ("k_cache", kd[..., :32]), ("block_table", tb.long()),
                      ("block_table", tb[:1]), ("block_table", tb.t()), ("lengths", ln.long()),
                      ("lengths", ln[:1]), ("lengths", ln.cpu()), ("o", o.float()),
                      ("o", o[:, :2]), ("lse", lse[:1]), ("workspace", ws.cpu()),
                      ("workspace", ws[::2])]:
        with pytest.raises(ValueError):
            lib.attn_decode_paged(**{**good, name: bad})
    for name, bad in [("workspace", ws[:-1]), ("workspace", ws[8:]), ("scale", 0.0),
                      ("scale", float("nan"))]:
        with pytest.raises(lib.CattnError):
            lib.attn_decode_paged(**{**good, name: bad})
    with pytest.raises(lib.CattnError):      # nine new positions
        lib.attn_decode_paged(qd[:, :, :1].expand(2, 4, 9, 64).contiguous(), kd, vd, tb, ln)
    with pytest.raises(lib.CattnError):      # three heads on two
        lib.attn_decode_paged(qd[:, :3].contiguous(), kd, vd, tb, ln)
    with pytest.raises(lib.CattnError):      # rows of the table that overlap
        lib.attn_decode_paged(**{**good, "block_table": tb[:1].expand(2, tb.shape[1])})
    with pytest.raises(lib.CattnError):      # a cache whose rows overlap
        lib.attn_cache_append(qd[:1, :2, 0], qd[:1, :2, 0], kd.as_strided(kd.shape, (8, 8, 8, 1)),
                              vd, dev([0], torch.int64))
    torch.cuda.synchronize()
    assert (o == 5).all() and (lse == 5).all()


def test_on_another_stream(lib):
    """inputs written, the call made and its results read on a side stream
    that is not the current one"""
    lengths = [500, 40]
    q, k, v, kd, vd, table = setup(9, lengths, 2, 2, 1, 64, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = (torch.empty(2, 4, 1, *s, dtype=t, device=DEV)
              for s, t in (((64,), torch.bfloat16), ((), torch.float32)))
    ws = torch.empty(lib.attn_decode_paged_workspace_bytes(2, 4, 2, 1, 64), dtype=torch.uint8,
                     device=DEV)
    tb, ln, qd = dev(table), dev(lengths), torch.zeros_like(q, device=DEV)
    src = q.to(DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        qd.copy_(src)
    lib.attn_decode_paged(qd, kd, vd, tb, ln, o=o, lse=lse, workspace=ws, stream=side)
    side.synchronize()
    ref = opaged.decode(as64(q), as64(k), as64(v), table, lengths, np.float32(0.125))
    check_decode(as64(o.cpu()), as64(lse.cpu()), ref, 500, 64)


def test_on_another_stream_with_its_own_allocations(lib):
    """nothing given but the inputs, a side stream that runs late, and the
    current stream filling whatever it gets meanwhile"""
    lengths = [20000, 400]
    q, k, v, kd, vd, table = setup(9, lengths, 2, 2, 1, 64, 16)
    bounds = rows(8, k.shape[0], 2, 2, 64).sort(2).values.to(DEV)
    qd, tb, ln = q.to(DEV), dev(table), dev(lengths)
    want = lib.attn_decode_paged(qd, kd, vd, tb, ln)
    pages = lib.attn_page_select(qd, bounds, tb, ln, 16, 20)
    listed = lib.attn_decode_sparse(qd, kd, vd, tb, ln, pages)
    n = lib.attn_decode_paged_workspace_bytes(2, 4, 2, 1, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(4_000_000)
        got = [lib.attn_decode_paged(qd, kd, vd, tb, ln, stream=stream)]
        got.append((lib.attn_page_select(qd, bounds, tb, ln, 16, 20, stream=stream),))
        got.append(lib.attn_decode_sparse(qd, kd, vd, tb, ln, got[1][0], stream=stream))
        junk = [torch.full((size,), 0x7f, dtype=torch.uint8, device=DEV)
                for size in (n, n, 1 << 20, 2 * 4 * 64 * 2, 2 * 4 * 4, 2 * 2 * 20 * 4) * 3]
        side.synchronize()
        for x, y in zip((*want, pages, *listed), (t for g in got for t in g)):
            assert torch.equal(x, y)
        del junk
