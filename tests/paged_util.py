"""Inputs and error bounds shared by the tests of the paged cache."""

from __future__ import annotations

import numpy as np
import torch

import oracle.paged as opaged


def rows(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def as64(t):
    return t.to(torch.float64).numpy()


def make_table(seed, lengths, P, width, n_pages):
    """int32 (B, width): disjoint pages in random order, -1 behind a
    request's last."""
    order = np.random.default_rng(seed).permutation(n_pages)
    table = np.full((len(lengths), width), -1, dtype=np.int32)
    at = 0
    for b, length in enumerate(lengths):
        n = min(opaged.n_pages_of(length, P), width)
        table[b, :n] = order[at:at + n]
        at += n
    assert at <= n_pages
    return table


def poison_unread(k, v, table, lengths, P):
    """NaN in every cache row that holds no key of any request, infinities
    among them."""
    held = np.zeros((k.shape[0], P), dtype=bool)
    for b, length in enumerate(lengths):
        for p in range(min(int(length), table.shape[1] * P)):
            page = table[b, p // P]
            if 0 <= page < k.shape[0]:
                held[page, p % P] = True
    free = torch.from_numpy(~held)
    for t, x in ((k, float("nan")), (v, float("nan"))):
        t.transpose(1, 2)[free] = x
    if free.any():
        page, row = (int(i[0]) for i in torch.nonzero(free, as_tuple=True))
        k[page, :, row] = float("inf")
        v[page, :, row] = float("-inf")


def check_decode(o, lse, ref, n_keys, D):
    """Error bounds, from the formula's roundings.  With u = 2^-24 (fp32):
    a score is a sum of D products in fp32, off by at most (D + 2) 2u r where
    r bounds sum |q k| (twice u a step: the tensor cores may truncate), so a
    weight is off by twice that, plus 8u of its exponential and 2^-16 of its
    bf16 pair, and the sums over n keys and over the parts add (n + 64) 2u.
    All of it acts on a = sum w |v|; o is rounded once more, by 2^-8 |o|."""
    ro, rl, a, reach = ref
    u = 2.0 ** -24
    ds = (D + 2) * 2 * u * reach
    rel = 2 * ds + 8 * u + 2.0 ** -16 + 2 * (n_keys + 64) * 2 * u
    bound = 2.0 ** -8 * np.abs(ro) + rel[..., None] * a * (1 + 2.0 ** -8) + 1e-37
    bad = np.abs(o - ro) > bound
    assert np.isfinite(o).all() and not bad.any(), (
        np.abs(o - ro)[bad][:4], bound[bad][:4], np.argwhere(bad)[:4])
    empty = np.isinf(rl)
    assert np.array_equal(np.isneginf(lse), empty), "empty rows"
    tol = ds + 8 * u + (n_keys + 64) * 2 * u + 4 * u * np.abs(np.where(empty, 0, rl))
    d = np.abs(np.where(empty, 0, lse) - np.where(empty, 0, rl))
    assert (d <= tol).all(), (d.max(), tol[d > tol][:4])
