"""Pins of the cache oracle (CPU only): worked examples, closed forms, a library's E4M3."""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co


def test_rope_hand_example_and_norm():
    # One position of a quarter turn: (a, b) -> (-b, a) for the pair with frequency pi / 2.
    f = np.zeros(32)
    f[0] = np.pi / 2
    x = np.arange(64.0).reshape(1, 1, 64) + 1
    y = co.rope(x, [[1]], f, [32], True)
    assert np.allclose(y[0, 0, :2], [-2, 1]) and np.allclose(y[0, 0, 2:], x[0, 0, 2:])
    z = co.rope(x, [[1]], f, [32], False)
    assert np.allclose(z[0, 0, [0, 32]], [-33, 1])
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64))
    for inter in (True, False):
        y = co.rope(x, rng.integers(0, 99, (3, 3)), rng.random(32), [8, 12, 12], inter)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))


def test_rope_relative_positions():
    rng = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(32) / 32)
    a, b = rng.standard_normal((2, 1, 1, 64))
    dots = [np.sum(co.rope(a, [[p]], f, [32], True) * co.rope(b, [[p + 7]], f, [32], True)) for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0])


def test_rope_axes_follow_their_sections():
    rng = np.random.default_rng(2)
    f = rng.random(32)
    x = rng.standard_normal((1, 1, 64))
    full = co.rope(x, [[3], [5], [7]], f, [8, 12, 12], True)
    for axis, (lo, hi) in zip((3, 5, 7), ((0, 16), (16, 40), (40, 64))):
        assert np.allclose(full[..., lo:hi], co.rope(x, [[axis]], f, [32], True)[..., lo:hi])


def test_quantise_against_the_library_conversion():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(40, 512, generator=g).to(torch.bfloat16).float()
    x[0] = 0
    codes, scales = co.quantise(x.numpy())
    assert (scales[0] == 1).all() and (codes[0] & 0x7F == 0).all()
    q = x.view(-1, 4, 128) / torch.from_numpy(scales)[..., None]
    lib = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 512)
    assert np.array_equal(codes, lib.numpy())


def test_quantise_non_finite_values():
    x = np.ones((1, 512), np.float32)
    x[0, 5], x[0, 130], x[0, 131] = np.inf, np.nan, 896.0
    codes, scales = co.quantise(x)
    assert codes[0, 5] == 0x7F and codes[0, 130] == 0x7F
    assert scales[0, 0] == np.float32(1) / np.float32(448) and scales[0, 1] == 2.0
    assert codes[0, 131] == 0x7E


def test_pool_hand_example():
    pool = co.Pool([[-1] * 4 for _ in range(4)], [0] * 4, [0] * 8, 4)
    assert pool.extend([0, 2], [6, 4], 12) == ([0, 6, 10], [0, 1, 2, 3, 4, 5, 8, 9, 10, 11, -1, -1], [0, 0])
    assert pool.table[0] == [0, 1, -1, -1] and pool.refs == [1, 1, 1, 0, 0, 0, 0, 0]
    # Row 1 shares page 0 and gets page 3 for the two tokens of page 1; row 3 shares page 2.
    assert pool.fork([0, 2], [1, 3]) == ([0, 0], [1, -1], [3, -1], [2, 0])
    assert pool.table[1] == [0, 3, -1, -1] and pool.refs == [2, 1, 2, 1, 0, 0, 0, 0]
    pool.free([0, 0, 9])
    assert pool.refs == [1, 0, 2, 1, 0, 0, 0, 0] and pool.lens == [0, 6, 4, 4]
    assert pool.compact() == (3, [3], [1])
    assert pool.table[1] == [0, 1, -1, -1] and pool.refs == [1, 1, 2, 0, 0, 0, 0, 0]


def test_pool_refusals():
    pool = co.Pool([[-1] * 2 for _ in range(3)], [0] * 3, [0] * 3, 4)
    # Two pages, then two more (one is left), then none needed, then a row twice and a bad row.
    ptr, slots, status = pool.extend([0, 1, 2, 0, 7], [8, 5, 0, 1, 1], 8)
    assert status == [0, co.NO_PAGES, 0, co.BAD_INDEX, co.BAD_INDEX] and ptr == [0, 8, 8, 8, 8, 8]
    assert pool.lens == [8, 0, 0]
    assert pool.extend([0], [1], 1)[2] == [co.BAD_INDEX]          # over the table's room
    assert pool.fork([0, 0], [0, 1])[0] == [co.BAD_INDEX, 0]      # its own parent
    assert pool.fork([0], [1])[0] == [co.BAD_INDEX]               # not empty
    pool.lens[0] = 6  # a row cut back into a page that row 1 holds too
    assert pool.extend([0], [1], 1)[2] == [co.BAD_INDEX]


@pytest.mark.parametrize("seed", range(5))
def test_pool_keeps_its_invariants(seed):
    """Every page's count is the number of rows that hold it, after any sequence of calls."""
    rng = np.random.default_rng(seed)
    pool = co.Pool([[-1] * 6 for _ in range(9)], [0] * 9, [0] * 30, 4)
    for _ in range(60):
        rows = rng.integers(-1, 10, 4).tolist()
        op = rng.integers(0, 4)
        if op == 0:
            pool.extend(rows, rng.integers(-1, 12, 4).tolist(), 20)
        elif op == 1:
            pool.fork(rows, rng.integers(0, 9, 4).tolist())
        elif op == 2:
            pool.free(rows[:2])
        else:
            live, src, dst = pool.compact()
            assert all(n > 0 for n in pool.refs[:live]) and not any(pool.refs[live:])
        held = [0] * 30
        for r, n in enumerate(pool.lens):
            for page in pool.table[r][:pool.blocks(n)]:
                held[page] += 1
        assert held == pool.refs
