"""The gated feed-forward's work units (CPU): the kernels' own index code covers every tile and every k stage once.

A unit out of range would read or write out of range, a missing or doubled one would give a wrong gradient, so the
launches' units are enumerated here for random sizes, SM counts and the gradients asked for.
"""
import ctypes

import numpy as np
import pytest

from sparse_attention_long_moga_b200 import _lib
from sparse_attention_long_moga_b200.build import build


@pytest.fixture(scope="module")
def units():
    build()
    fn = _lib.load().moga_test_ffn_units
    fn.restype = ctypes.c_int64
    fn.argtypes = [ctypes.c_int32, ctypes.c_int64] + [ctypes.c_int32] * 6 + [ctypes.c_void_p, ctypes.c_int64]

    def call(*a):
        n = fn(*a, None, 0)
        out = np.zeros((n, 10), dtype=np.int32)
        assert fn(*a, out.ctypes.data_as(ctypes.c_void_p), n) == n
        return out
    return call


def ceil(a, b):
    return -(-a // b)


SIZES = [(1, 8, 8), (777, 264, 712), (32760, 1536, 4096), (8190, 5120, 13824), (65536, 64, 128), (300, 5120, 64),
         (64, 8, 100000), (5000, 128, 2048)]


def _sizes():
    rng = np.random.default_rng(0)
    for _ in range(60):
        yield tuple(int(np.exp(rng.uniform(np.log(a), np.log(b)))) * m for a, b, m in ((1, 70000, 1), (1, 640, 8),
                                                                                     (1, 1728, 8)))
    yield from SIZES


@pytest.mark.parametrize("sms", [148, 132, 7, 2])
def test_gradient_units(units, sms):
    for N, d, F in _sizes():
        for need_dx, need_dw in ((1, 1), (1, 0), (0, 1)):
            u = units(1, N, d, F, need_dx, need_dw, 256, sms)
            nt = ceil(d, 256)
            dx, dw = u[u[:, 1] == 1], u[u[:, 1] == 2]
            assert len(dx) + len(dw) == len(u) and u[:, 0].max() < max(1, sms // 2)
            # rows of a tile: 512, or 256 where there would be few tiles
            rows = 512 if 2 * nt * (ceil(N, 512) + 2 * ceil(F, 512)) >= 3 * max(1, sms // 2) else 256
            assert not dx[:, 2].any()
            halves = range(rows // 256)
            x_tiles = {(0, m, n, h) for m in range(ceil(N, rows)) for n in range(nt) for h in halves}
            tiles = {(up, m, n, h) for up in (0, 1) for m in range(ceil(F, rows)) for n in range(nt) for h in halves}
            x_tiles, tiles = x_tiles if need_dx else set(), tiles if need_dw else set()
            for part, want, stages in ((dx, x_tiles, 2 * ceil(F, 64)), (dw, tiles, ceil(N, 64))):
                seen = {}
                for _, _, up, m, n, split, k0, k1, h0, h1 in part.tolist():
                    assert 0 <= k0 < k1 <= stages and 0 <= h0 < h1 <= rows // 256
                    for h in range(h0, h1):
                        seen.setdefault((up, m, n, h), []).append((split, k0, k1))
                assert set(seen) == want
                for parts in seen.values():
                    parts.sort()
                    assert [p[0] for p in parts] == list(range(len(parts)))
                    assert parts[0][1] == 0 and parts[-1][2] == stages
                    assert all(a[2] == b[1] for a, b in zip(parts, parts[1:]))
            # no pair is given much more than its share: within two of the longest units of the mean
            if len(u):
                work = (u[:, 7] - u[:, 6]) * (u[:, 9] - u[:, 8])
                pairs = min(len(u), max(1, sms // 2))
                assert np.bincount(u[:, 0], weights=work).max() <= work.sum() / pairs + 2 * work.max()
                # a single half comes last, so that its pair's barriers stay in step
                single = np.flatnonzero(u[:, 9] - u[:, 8] < rows // 256)
                assert np.all((single == len(u) - 1) | (u[np.minimum(single + 1, len(u) - 1), 0] != u[single, 0]))


@pytest.mark.parametrize("bn", [128, 256])
def test_forward_tiles(units, bn):
    for N, d, F in _sizes():
        u = units(0, N, d, F, 0, 0, bn, 148)
        want = {(m, n) for m in range(ceil(N, 256)) for n in range(ceil(F, bn // 2))}
        got = [tuple(r) for r in u[:, 3:5].tolist()]
        assert len(got) == len(want) and set(got) == want
        assert np.all(u[:, 6] == 0) and np.all(u[:, 7] == ceil(d, 64)) and np.all(u[:, 1] == 0)
