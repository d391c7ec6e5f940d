"""The paged-cache kernels' own sources run on the CPU (tests/emu), built with
AddressSanitizer and UBSan over exactly sized buffers, against the fp64
oracle: any access outside a buffer fails the run.  Page numbers outside the
pool, lengths outside the table, slots outside the cache and the like are
tried here before any GPU sees them."""

from __future__ import annotations

import os
import shutil
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

import oracle.paged as opaged
from paged_util import as64, check_decode, make_table, poison_unread, rows

ROOT = Path(__file__).resolve().parents[1]
EMU = ROOT / "tests" / "emu"


@pytest.fixture(scope="module")
def emu(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("emu")
    exe = d / "paged_emu"
    cmd = [cxx, "-std=c++20", "-O1", "-g", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-pthread", "-I", str(EMU / "include"), "-I", str(EMU),
           "-I", str(ROOT / "causal_self_attention_flash_b200" / "csrc"),
           str(EMU / "paged_emu.cpp"), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        pytest.fail("emulator build failed:\n" + r.stderr[-3000:])

    def run(op, params, *arrays):
        with open(d / "in.bin", "wb") as f:
            for x in (np.array(params, dtype=np.int64), *arrays):
                x = np.ascontiguousarray(x)
                f.write(np.int64(x.nbytes).tobytes() + x.tobytes())
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0")
        r = subprocess.run([str(exe), op, str(d / "in.bin"), str(d / "out.bin")],
                           capture_output=True, text=True, timeout=900, env=env)
        assert r.returncode == 0, r.stderr[-3000:]
        return (d / "out.bin").read_bytes()
    return run


def bits(x):
    return x.contiguous().view(torch.int16).numpy()


def from_bits(b):
    return (np.frombuffer(b, np.uint16).astype(np.uint32) << 16).view(np.float32)


def take(raw, *parts):
    """Splits bytes into arrays of (dtype, count)."""
    at, out = 0, []
    for dtype, n in parts:
        size = np.dtype(dtype).itemsize * n
        out.append(np.frombuffer(raw[at:at + size], dtype))
        at += size
    assert at == len(raw)
    return out


def run_decode(emu, lengths, Hkv, G, Tq, D, P, grid, *, layout=1, spare=0, holes=(), pages=None,
               seed=0, poison=True):
    B, H = len(lengths), Hkv * G
    width = max(1, max(opaged.n_pages_of(n, P) for n in lengths) + spare)
    n_pages = max(1, sum(min(opaged.n_pages_of(n, P), width) for n in lengths) + 1)
    table = make_table(seed, lengths, P, width, n_pages)
    for (b, i), page in holes:
        table[b, i] = page
    k, v = (rows(seed + s, n_pages, Hkv, P, D) for s in (1, 2))
    if poison:
        poison_unread(k, v, table, lengths, P)
    q = rows(seed + 3, B, H, Tq, D, std=1.5)
    scale = D ** -0.5
    st = [x.transpose(1, 2) if layout else x for x in (k, v)]
    n_sel = 0 if pages is None else pages.shape[2]
    raw = emu("decode", [B, H, Hkv, Tq, D, n_pages, P, width, n_sel, grid, layout],
              bits(q), bits(st[0]), bits(st[1]), table, np.array(lengths, np.int32),
              np.zeros(0, np.int32) if pages is None else pages.astype(np.int32),
              np.array([scale], np.float32))
    n = B * H * Tq
    o = from_bits(raw[:2 * n * D]).astype(np.float64).reshape(B, H, Tq, D)
    lse = np.frombuffer(raw[2 * n * D:], np.float32).astype(np.float64).reshape(B, H, Tq)
    ref = opaged.decode(as64(q), as64(k), as64(v), table, lengths, np.float32(scale), pages)
    check_decode(o, lse, ref, max(1, max(lengths)), D)
    return o, lse


@pytest.mark.parametrize("lengths,Hkv,G,Tq,D,P,grid", [
    ([1], 1, 1, 1, 16, 16, 1),
    ([0, 5, -3, 1], 1, 1, 1, 64, 16, 2),       # empty requests between others
    ([-2 ** 31, 20, -2 ** 31], 1, 2, 8, 64, 16, 1),
    ([37], 1, 1, 1, 32, 16, 1),
    ([100, 3], 2, 4, 1, 64, 16, 1),            # several items per warp
    ([70], 1, 2, 1, 128, 16, 1),               # one item over several warps
    ([130, 64, 1], 1, 3, 1, 128, 20, 2),       # pages that end inside a chunk
    ([33, 90], 1, 1, 4, 64, 8, 1),             # several new positions
    ([2, 5, 40], 1, 2, 8, 32, 4, 1),           # fewer keys than new positions
    ([50, 18], 1, 5, 3, 64, 7, 1),             # 15 rows, odd pages
    ([40], 1, 8, 3, 16, 16, 1),                # 24 rows: two tiles
    ([45], 1, 9, 2, 128, 16, 1),               # 18 rows at D = 128
    ([200], 1, 1, 1, 64, 1, 1),                # pages of one position
    ([90, 30], 1, 1, 1, 64, 128, 1),           # pages beyond a chunk
])
def test_decode(emu, lengths, Hkv, G, Tq, D, P, grid):
    run_decode(emu, lengths, Hkv, G, Tq, D, P, grid, spare=2)
    if D <= 64:
        run_decode(emu, lengths, Hkv, G, Tq, D, P, -(1 + len(lengths) % 3), spare=2, seed=9)


@pytest.mark.parametrize("layout", [0, 1])
def test_decode_layouts(emu, layout):
    run_decode(emu, [61, 17], 2, 2, 1, 64, 16, 1, layout=layout)


def test_decode_many_requests(emu):
    """more requests than threads: several per thread of the scan"""
    lengths = [(i * 37) % 17 for i in range(150)]
    run_decode(emu, lengths, 1, 1, 1, 16, 8, 2)


@pytest.mark.parametrize("Tq", [1, 3])
def test_decode_pages_that_are_not_held(emu, Tq):
    """-1 and page numbers outside the pool: nothing is read there"""
    for grid in (2, -1, -2):
        run_decode(emu, [100, 40, 20], 1, 2, Tq, 64, 16, grid,
                   holes=[((0, 0), -1), ((0, 3), 10 ** 6), ((1, 2), -7), ((2, 0), 1 << 30),
                          ((2, 1), -1)])


def test_decode_longer_than_the_table(emu):
    """a length beyond width * P: the rows see what the table holds"""
    B, P, D, width = 1, 16, 64, 2
    table = np.array([[1, 0]], np.int32)
    k, v = rows(1, 2, 1, P, D), rows(2, 2, 1, P, D)
    q = rows(3, B, 1, 2, D)
    raw = emu("decode", [B, 1, 1, 2, D, 2, P, width, 0, 1, 0], bits(q), bits(k), bits(v), table,
              np.array([2 ** 31 - 1], np.int32), np.zeros(0, np.int32),
              np.array([0.125], np.float32))
    o = from_bits(raw[:2 * 2 * D]).astype(np.float64).reshape(1, 1, 2, D)
    ref, _, _, _ = opaged.decode(as64(q), as64(k), as64(v), table, [32 + 5], 0.125)
    assert np.abs(o - ref).max() < 0.02


def test_decode_unseen_keys_do_not_touch_a_row(emu):
    """NaN and infinities in keys and values that only later rows see: the
    earlier rows are those of clean inputs"""
    lengths, Tq, D, P = [40], 4, 64, 16
    table = np.array([[2, 0, 1]], np.int32)
    k, v = rows(1, 3, 1, P, D), rows(2, 3, 1, P, D)
    q = rows(3, 1, 2, Tq, D)

    def run():
        raw = emu("decode", [1, 2, 1, Tq, D, 3, P, 3, 0, 1, 0], bits(q), bits(k), bits(v), table,
                  np.array(lengths, np.int32), np.zeros(0, np.int32),
                  np.array([0.125], np.float32))
        return (from_bits(raw[:2 * 2 * Tq * D]).reshape(2, Tq, D),
                np.frombuffer(raw[2 * 2 * Tq * D:], np.float32).reshape(2, Tq))
    o, lse = run()
    for pos, bad_k, bad_v in ((37, 1.0, float("nan")), (38, float("nan"), float("inf"))):
        k[table[0, pos // P], 0, pos % P] *= bad_k
        v[table[0, pos // P], 0, pos % P, ::2] = bad_v
    o2, lse2 = run()
    assert np.array_equal(o[:, 0], o2[:, 0]) and np.array_equal(lse[:, 0], lse2[:, 0])
    assert np.isnan(o2[:, 1, ::2]).all() and np.array_equal(o[:, 1, 1::2], o2[:, 1, 1::2])
    assert np.isnan(o2[:, 2:]).all() and np.isnan(lse2[:, 2:]).all()


def decode_raw(emu, q, k, v, table, length, grid, scale):
    """one request, packed (n_pages, Hkv, P, D) pools"""
    (B, H, Tq, D), (n_pages, Hkv, P, _) = q.shape, k.shape
    raw = emu("decode", [B, H, Hkv, Tq, D, n_pages, P, table.shape[1], 0, grid, 0], bits(q),
              bits(k), bits(v), table, np.array([length], np.int32), np.zeros(0, np.int32),
              np.array([scale], np.float32))
    n = B * H * Tq
    o = from_bits(raw[:2 * n * D]).astype(np.float64).reshape(B, H, Tq, D)
    return o, np.frombuffer(raw[2 * n * D:], np.float32).astype(np.float64).reshape(B, H, Tq)


@pytest.mark.parametrize("D,G,Tq", [(64, 2, 1), (64, 3, 2), (128, 9, 1), (16, 5, 4)])
def test_decode_infinite_values(emu, D, G, Tq):
    """an infinite value that a row sees is its result (NaN where both signs
    meet), whatever the key's weight; other channels are as without it"""
    L, P = 75, 16
    table = np.arange(5, dtype=np.int32)[None, ::-1].copy()
    k, v, q = rows(1, 5, 1, P, D), rows(2, 5, 1, P, D), rows(3, 1, G, Tq, D, std=1.5)
    scale = np.float32(D ** -0.5)
    ref = opaged.decode(as64(q), as64(k), as64(v), table, [L], scale)

    def at(pos):
        return table[0, pos // P], 0, pos % P
    for pos, d in ((0, 0), (17, 1), (34, 2), (50, 3), (L - Tq, 4)):
        v[at(pos)][d] = float("inf")
        v[at(pos)][d + 5] = float("-inf")
    v[at(3)][11], v[at(40)][11] = float("inf"), float("-inf")
    for grid in (1, 2, -1, -2):
        o, lse = decode_raw(emu, q, k, v, table, L, grid, scale)
        assert (o[..., :5] == np.inf).all() and (o[..., 5:10] == -np.inf).all()
        assert np.isnan(o[..., 11]).all()
        o[..., [*range(10), 11]] = ref[0][..., [*range(10), 11]]
        check_decode(o, lse, ref, L, D)
    # one key: its weight is one
    v[at(0)][:] = float("inf")
    for grid in (1, -1):
        assert (decode_raw(emu, q, k, v, table, Tq, grid, scale)[0][:, :, -1] == np.inf).all()
        assert (decode_raw(emu, q[:, :, -1:], k, v, table, 1, grid, scale)[0] == np.inf).all()


@pytest.mark.parametrize("D,G,Tq", [(64, 1, 1), (128, 9, 1), (32, 3, 2)])
def test_decode_large_values(emu, D, G, Tq):
    """scores that rise by less than the running maximum follows, with values
    near the largest bf16: finite where the formula is"""
    L, P, n = 131 + Tq, 16, 9
    table = np.arange(n, dtype=np.int32)[None]
    k, v, q = rows(1, n, 1, P, D), rows(2, n, 1, P, D), rows(3, 1, G, Tq, D, std=1.5)
    q[..., 0], k[..., 0] = 1, 0
    q[..., 1:] = 0
    for pos, x in ((128, 5.25), (129, 5.5), (130, 5.375)):      # e^5.5 < 2^8
        k[table[0, pos // P], 0, pos % P, 0] = x
        v[table[0, pos // P], 0, pos % P, :] = 3e38 * (-1) ** pos
        v[table[0, pos // P], 0, pos % P, 1::2] = 1.5e38
    ref = opaged.decode(as64(q), as64(k), as64(v), table, [L], 1.0)
    for grid in (1, 2, -1, -2):
        o, lse = decode_raw(emu, q, k, v, table, L, grid, 1.0)
        check_decode(o, lse, ref, L, D)


@pytest.mark.parametrize("Tq,G", [(1, 1), (2, 3)])
def test_sparse(emu, Tq, G):
    pages = np.full((3, 2, 4), -1)
    pages[0, 0] = [0, 2, 5, 6]
    pages[0, 1] = [1, 1, 3, 6]          # a page listed twice counts twice
    pages[1, :, :2] = [0, 1]
    pages[2, 0] = [0, 99, -4, 2]        # entries that list nothing
    pages[2, 1] = [2, 1, 0, 7]          # any order; the fourth is behind the last page
    for grid in (2, -2):
        run_decode(emu, [100, 20, 45], 2, G, Tq, 64, 16, grid, spare=1, pages=pages,
                   holes=[((0, 5), -1)])


# ------------------------------------------------------------------- plan

def run_plan(emu, asked, lengths, table, ring, state, P, n_slots, ctas=1, in_place=False,
             threads=256, prompts=False):
    B, width = table.shape
    raw = emu("plan", [B, width, len(ring), P, n_slots, ctas, int(in_place), threads, int(prompts)],
              np.array(asked, np.int32), np.array(lengths, np.int32), table.astype(np.int32),
              np.array(ring, np.int32), np.array(state, np.int64))
    got = take(raw, (np.int32, B), (np.int64, 2), (np.int32, B + 1), (np.int64, n_slots),
               (np.int32, n_slots), (np.int32, 1), (np.int32, B * width), (np.int32, len(ring)))
    keys = ("lengths", "state", "cu", "slots", "positions", "status", "table", "ring")
    got = dict(zip(keys, got))
    got["table"] = got["table"].reshape(B, width)
    want = opaged.plan(np.array(asked), np.array(lengths), table, np.array(ring), state, P, n_slots)
    for key in keys:
        assert np.array_equal(got[key], np.ravel(want[key]) if key == "status" else want[key]), key
    return want


def plan_inputs(seed, B, P, longest, most, spare=4):
    rng = np.random.default_rng(seed)
    lengths = rng.integers(0, longest + 1, B)
    asked = rng.integers(-1, most + 1, B)
    width = opaged.n_pages_of(longest + most, P) + 1
    counts = [opaged.n_pages_of(n, P) for n in lengths]
    n_pages = sum(counts) + B * (most // P + 2) + spare
    table = make_table(seed, lengths, P, width, n_pages)
    free = sorted(set(range(n_pages)) - set(table[table >= 0].tolist()))
    head = int(rng.integers(0, 3 * n_pages))
    ring = np.full(n_pages, -5)
    for i, page in enumerate(free):
        ring[(head + i) % n_pages] = page
    return asked, lengths, table, ring, np.array([head, head + len(free)])


@pytest.mark.parametrize("B,P,longest,most,ctas,threads", [
    (1, 16, 40, 1, 1, 256), (5, 16, 100, 30, 1, 256), (40, 8, 60, 3, 2, 256),
    (9, 5, 33, 200, 2, 256), (300, 16, 64, 1, 2, 64), (7, 1, 9, 4, 1, 1024)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(emu, B, P, longest, most, ctas, threads, in_place):
    asked, lengths, table, ring, state = plan_inputs(B + P, B, P, longest, most)
    n_slots = int(np.maximum(asked, 0).sum()) + 3
    want = run_plan(emu, asked, lengths, table, ring, state, P, n_slots, ctas, in_place, threads)
    if in_place:
        run_plan(emu, asked, lengths, table, ring, state, P, n_slots, ctas, in_place, threads, True)
    assert want["status"] == opaged.OK


def test_plan_refusals_change_nothing(emu):
    asked, lengths, table, ring, state = plan_inputs(3, 6, 8, 50, 20)
    asked[2] = 17
    asked[3], lengths[3] = -1, 20
    n = int(np.maximum(asked, 0).sum())
    run = lambda **kw: run_plan(emu, **{**dict(  # noqa: E731
        asked=asked, lengths=lengths, table=table, ring=ring, state=state, P=8, n_slots=n), **kw})
    assert run()["status"] == opaged.OK
    assert run(n_slots=n - 1)["status"] == opaged.TOO_LARGE
    need = opaged.plan(asked, lengths, table, ring, state, 8, n)["state"][0] - state[0]
    assert run(state=np.array([state[0], state[0] + need - 1]))["status"] == opaged.TOO_LARGE
    big = asked.copy()
    big[1] = table.shape[1] * 8 + 1
    assert run(asked=big)["status"] == opaged.TOO_LARGE
    big[1] = 2 ** 31 - 1
    assert run(asked=big)["status"] == opaged.TOO_LARGE
    neg = lengths.copy()
    neg[4] = -1
    assert run(lengths=neg)["status"] == opaged.INVALID
    assert run(state=np.array([5, 4]))["status"] == opaged.INVALID
    assert run(state=np.array([-3, 4]))["status"] == opaged.INVALID
    assert run(state=np.array([0, len(ring) + 1]))["status"] == opaged.INVALID
    # more pages than the pool has would be free
    assert run(state=np.array([0, len(ring)]))["status"] == opaged.INVALID
    over = lengths.copy()
    over[3] = table.shape[1] * 8 + 1
    assert run(lengths=over)["status"] == opaged.INVALID


def test_plan_without_requests_and_with_foreign_pages(emu):
    run_plan(emu, [], [], np.zeros((0, 3), np.int32), [0, 1], np.array([0, 2]), 4, 2)
    # a page number outside the pool in the ring or in the table gives slot -1
    want = run_plan(emu, [3, 2], [2, 0], np.array([[77, -1], [-1, -1]]), [1, -9, 2],
                    np.array([1, 3]), 4, 5)
    assert (want["slots"] == -1).any() and (want["slots"] >= 0).any()


@pytest.mark.parametrize("ctas,threads,prompts", [(1, 256, False), (3, 64, False), (2, 128, True)])
def test_plan_frees_held_pages_only(emu, ctas, threads, prompts):
    """entries that are not held in the rows of requests that end: they are not
    put into the ring, and none is handed out afterwards"""
    B, P = 30, 4
    asked, lengths, table, ring, state = plan_inputs(11, B, P, 90, 3)
    asked = np.maximum(asked, 0)
    asked[::3], lengths[::3] = -1, np.maximum(lengths[::3], 5)
    for b in range(B):
        for i in range(opaged.n_pages_of(lengths[b], P), table.shape[1]):
            table[b, i] = -1
    for j, bad in enumerate((-1, len(ring), -2 ** 31, 2 ** 31 - 1, -1, -1)):
        table[6 * (j % 5), j % 2] = bad
    table[27, :2] = -1                              # a row without a held page in front
    n_slots = int(np.maximum(asked, 0).sum()) + 3
    want = run_plan(emu, asked, lengths, table, ring, state, P, n_slots, ctas, False, threads,
                    prompts)
    assert want["status"] == opaged.OK
    head, tail = want["state"]
    assert all(0 <= want["ring"][i % len(ring)] < len(ring) for i in range(head, tail))
    # more of them held than the ring has room for: refused, nothing changed
    many = table.copy()
    many[::3, :2] = 0
    want = run_plan(emu, asked, lengths, many, ring, np.array([0, len(ring)]), P, n_slots, ctas,
                    False, threads, prompts)
    assert want["status"] == opaged.INVALID
    # entries that are not held take no room
    none = table.copy()
    none[::3] = -1
    want = run_plan(emu, asked, lengths, none, ring, np.array([0, len(ring)]), P, n_slots, ctas,
                    False, threads, prompts)
    assert want["status"] == opaged.OK


# ----------------------------------------------------------------- append

def run_append(emu, slots, Hkv, D, n_pages, P, bounds=True, bad=None, seed=0, tile=1):
    n = len(slots)
    kn, vn = rows(seed + 1, n, Hkv, D), rows(seed + 2, n, Hkv, D)
    if bad is not None:
        kn[bad] = float("nan")
    k, v = rows(seed + 3, n_pages, Hkv, P, D), rows(seed + 4, n_pages, Hkv, P, D)
    lo = rows(seed + 5, n_pages, Hkv, 1, D)
    bd = torch.cat([lo, lo + 1], 2)
    raw = emu("append", [n, Hkv, D, n_pages, P, tile], bits(kn), bits(vn), np.array(slots, np.int64),
              bits(k.transpose(1, 2)), bits(v.transpose(1, 2)),
              bits(bd) if bounds else np.zeros(0, np.int16))
    size = k.numel()
    gk, gv = (from_bits(raw[2 * i * size:2 * (i + 1) * size]).reshape(n_pages, P, Hkv, D)
              .transpose(0, 2, 1, 3) for i in (0, 1))
    f32 = lambda t: t.float().numpy()  # noqa: E731
    wk, wv, wb = opaged.append(f32(kn), f32(vn), slots, f32(k), f32(v), f32(bd))
    assert np.array_equal(gk, wk, equal_nan=True) and np.array_equal(gv, wv)
    if bounds:
        gb = from_bits(raw[4 * size:]).reshape(n_pages, Hkv, 2, D)
        assert np.array_equal(gb, wb, equal_nan=True)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("bounds", [False, True])
def test_append(emu, D, bounds):
    # a run inside a page, a page boundary, skipped and foreign slots, lone rows
    slots = [21, 22, 23, 24, 25, 40, -1, 3, 10 ** 12, 8, 9, 50, 55, -2 ** 62]
    run_append(emu, slots, 3, D, 8, 8, bounds, tile=4 if D < 64 else 32)


def test_append_nan_keys_and_odd_pages(emu):
    run_append(emu, [3, 4, 5, 6, 7, 12], 1, 64, 4, 5, bad=2)
    run_append(emu, [0], 1, 16, 1, 1)
    for tile in (5, 32):
        run_append(emu, list(range(7, 60)), 2, 64, 3, 20, tile=tile)
    run_append(emu, list(range(3, 120)), 1, 16, 1, 130, tile=3)     # one run over many tiles
    run_append(emu, [5, 5 + 2 ** 40], 1, 16, 1, 16, tile=4)         # a run that breaks off
    # rows of a page in any order, with gaps, one of them twice, its first row late
    run_append(emu, [9, 12, 10, 10, 8, 15, 3, 1], 2, 32, 2, 8, tile=8)
    run_append(emu, [9, 12, 10, 10, 8, 15, 3, 1], 2, 32, 2, 8, tile=3)


# ----------------------------------------------------------------- select

def run_select(emu, lengths, Hkv, G, Tq, D, P, K, n_first=1, n_last=1, spare=0, holes=(),
               change=None, seed=0, groups=0):
    B, H = len(lengths), Hkv * G
    width = max(opaged.n_pages_of(n, P) for n in lengths) + spare
    n_pages = sum(opaged.n_pages_of(n, P) for n in lengths) + 2
    table = make_table(seed, lengths, P, width, n_pages)
    for (b, i), page in holes:
        table[b, i] = page
    mid = rows(seed + 1, n_pages, Hkv, 1, D).float()
    wide = rows(seed + 2, n_pages, Hkv, 2, D).float().abs()
    bounds = torch.cat([mid - wide[:, :, :1], mid + wide[:, :, 1:]], 2).to(torch.bfloat16)
    q = rows(seed + 3, B, H, Tq, D)
    if change:
        change(q, bounds, table)
    raw = emu("select", [B, H, Hkv, Tq, D, n_pages, P, width, K, n_first, n_last,
                         groups], bits(q),
              bits(bounds), table, np.array(lengths, np.int32))
    got = np.frombuffer(raw, np.int32).reshape(B, Hkv, K)
    want = opaged.select(as64(q), as64(bounds), table, lengths, P, K, n_first, n_last)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("lengths,Hkv,G,Tq,D,P,K,n_first,n_last", [
    ([400, 3, 0, 77], 1, 1, 1, 64, 4, 7, 1, 1),
    ([900], 2, 3, 1, 128, 8, 20, 0, 0),
    ([700, 640], 1, 2, 4, 32, 16, 8, 2, 3),
    ([333], 1, 1, 2, 16, 3, 2, 1, 1),          # nothing but the first and the last
    ([500], 1, 5, 4, 64, 8, 9, 1, 1),          # 20 rows: two tiles of 16
    ([1200], 1, 1, 1, 16, 4, 290, 1, 1),       # all but a few; more pages than threads
])
def test_select(emu, lengths, Hkv, G, Tq, D, P, K, n_first, n_last):
    # the fused kernel (2,048 host threads a cluster) for one, two kernels for all
    if len(lengths) == 2:
        run_select(emu, lengths, Hkv, G, Tq, D, P, K, n_first, n_last, spare=3)
    run_select(emu, lengths, Hkv, G, Tq, D, P, K, n_first, n_last, seed=20, groups=3)


def test_select_ties_nan_and_pages_that_are_not_held(emu):
    def same(q, bounds, table):
        bounds[:] = bounds[:1]                  # every page scores alike
    run_select(emu, [300], 1, 2, 1, 64, 4, 9, change=same, groups=1)

    def zero(q, bounds, table):
        q[:] = 0
        bounds[::2] *= -1                       # zeros of both signs
    run_select(emu, [300], 1, 1, 1, 64, 4, 9, change=zero, groups=2)

    def odd(q, bounds, table):
        bounds[table[0, 11], 0, 1, 5] = float("nan")
        bounds[table[0, 13]] = float("-inf")
        bounds[table[0, 17], 0, 1] = float("inf")
        bounds[table[0, 17], 0, 0] = 0
    run_select(emu, [300], 1, 1, 1, 64, 4, 9, change=odd,
               holes=[((0, 4), -1), ((0, 8), 10 ** 6)])
    # more pages that are not held than are left out
    run_select(emu, [40], 1, 1, 1, 16, 4, 8, holes=[((0, i), -1) for i in range(1, 7)])


@pytest.mark.parametrize("groups", [0, 1])
@pytest.mark.parametrize("gap", [2, 5, 100])
def test_select_with_a_late_warp(emu, monkeypatch, groups, gap):
    """sure pages and ties at the border, the ties that are just chosen in a
    warp that is late behind every barrier: what the others write then must not
    reach what it still reads.  The gap between the sure pages and the ties sets
    how many rounds the search for the border takes."""
    monkeypatch.setenv("LATE_WARP", "1")

    def change(q, bounds, table):
        bounds[:] = bounds[:1]
        q.copy_(bounds[0, 0, 1].expand_as(q))
        for i in (9, 20, 74):
            bounds[table[0, i]] *= gap
        bounds[:, :, 0] = 0
    run_select(emu, [320], 1, 1, 1, 16, 4, 45, change=change, groups=groups)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_select_nan_in_a_page_that_is_always_taken(emu, bad):
    """NaN or infinite bounds of the first page: the others are chosen by their
    exact sums all the same, here two whose terms of 2^20 cancel"""
    for seed in range(6):
        def change(q, bounds, table):
            q[:] = 1
            bounds[:] = bounds.clamp(-0.01, 0.01)
            bounds[:, :, 1] = 0
            bounds[table[0, 0]] = bad
            x = rows(seed + 50, 2, 5).abs()
            for i, page in ((0, 8), (1, 16)):
                hi = bounds[table[0, page], 0, 1]
                hi[0], hi[40] = 2.0 ** 20, -2.0 ** 20
                hi[[3, 5, 18, 21, 30]] = x[i] / 16
        run_select(emu, [120], 1, 1, 1, 64, 4, 2, n_last=0, change=change, seed=seed, groups=3)


# ------------------------- forms that the parameters above leave out

@pytest.mark.parametrize("lengths,Hkv,G,Tq,P,ctas", [
    ([70, 3], 1, 2, 1, 16, 1), ([45], 1, 9, 2, 16, 2), ([130], 2, 3, 2, 20, 2),
    ([0, 33], 1, 16, 1, 8, 1)])
def test_decode_an_item_per_cluster_d128(emu, lengths, Hkv, G, Tq, P, ctas):
    run_decode(emu, lengths, Hkv, G, Tq, 128, P, -ctas, spare=1, seed=3)


def test_decode_many_requests_of_some_chunks(emu):
    """several requests per thread of the scan, of one to three chunks each"""
    run_decode(emu, [(i * 37) % 90 for i in range(140)], 1, 1, 1, 16, 8, 2)


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_prompts(emu, in_place):
    asked, lengths, table, ring, state = plan_inputs(8, 9, 5, 33, 200)
    n_slots = int(np.maximum(asked, 0).sum()) + 3
    run_plan(emu, asked, lengths, table, ring, state, 5, n_slots, 2, in_place, 64, True)


@pytest.mark.parametrize("D,tile", [(16, 1), (64, 4), (128, 1), (128, 4), (32, 32)])
def test_append_tiles(emu, D, tile):
    slots = [21, 22, 23, 24, 25, 40, -1, 3, 10 ** 12, 8, 9, 50, 55, -2 ** 62]
    run_append(emu, slots, 3, D, 8, 8, True, tile=tile)
    if tile == 1:
        run_append(emu, list(range(7, 60)), 2, D, 3, 20, tile=1)


@pytest.mark.parametrize("ties", [False, True])
def test_select_in_one_launch(emu, ties):
    def same(q, bounds, table):
        bounds[:] = bounds[:1]
        bounds[::2, :, :, 3:5] *= -1            # zeros of both signs among them
        q[..., 3:5] = 0
    run_select(emu, [300, 21], 1, 2, 1, 128, 4, 9, change=same if ties else None, seed=6)
