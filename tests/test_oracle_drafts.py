"""Pins of the draft and branch oracle: closed forms, invariants and the
existing decode oracle on what both describe."""

import math

import numpy as np
import pytest

import oracle


def rng(seed):
    return np.random.default_rng(seed)


def table(n_pos, half):
    a = np.arange(n_pos)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.stack([np.cos(a), np.sin(a)], -1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 8])
def test_rotation_keeps_lengths_and_depends_on_relative_positions(interleaved, rot):
    g = rng(rot)
    q, k = g.normal(size=(1, 1, 1, 16)), g.normal(size=(1, 1, 1, 16))
    cs = table(64, rot // 2)
    at = lambda x, p: oracle.norm_rope(x, None, 0.0, cs, np.full((1, 1), p), interleaved=interleaved)
    assert np.allclose(at(q, 0), q)
    assert np.allclose(np.linalg.norm(at(q, 23)), np.linalg.norm(q))
    dots = [(at(q, 7 + s) * at(k, 2 + s)).sum() for s in (0, 11, 50)]
    assert np.allclose(dots, dots[0])
    assert np.array_equal(at(q, 9)[..., rot:], q[..., rot:])


def test_norm_has_unit_rms_and_ignores_scale():
    x = rng(1).normal(size=(1, 2, 3, 64))
    y = oracle.norm_rope(x, np.ones(64), 0.0, None, None)
    assert np.allclose((y * y).mean(-1), 1)
    assert np.allclose(y, oracle.norm_rope(37 * x, np.ones(64), 0.0, None, None))


def test_sections_take_each_axis_from_its_own_position():
    x = rng(2).normal(size=(1, 1, 1, 12))
    cs = table(32, 6)
    pos = np.array([3, 17, 30]).reshape(3, 1, 1)
    y = oracle.norm_rope(x, None, 0.0, cs, pos, sections=[1, 2, 3])
    for p, a in enumerate([0, 1, 1, 2, 2, 2]):
        one = oracle.norm_rope(x, None, 0.0, cs, pos[a])
        assert np.allclose(y[..., [p, p + 6]], one[..., [p, p + 6]])


def test_tree_of_one_token_is_decode_attention():
    g = rng(3)
    q, K, V = g.normal(size=(1, 4, 8)), g.normal(size=(2, 30, 8)), g.normal(size=(2, 30, 8))
    vis = np.array([[0, 4, 9], [1, 2, 19]])
    out, lse, _ = oracle.tree_attention(q, K, V, vis, 20, 9, [1], 0.3)
    ref, ref_lse = oracle.sparse_decode_attention(q, K[None], V[None], vis[None], 20, 10, scale=0.3)
    assert np.allclose(out, ref) and np.allclose(lse, ref_lse)


def test_tree_chain_mask_equals_no_mask_and_hidden_tokens_have_no_part():
    g = rng(4)
    T = 5
    q, K, V = g.normal(size=(T, 2, 8)), g.normal(size=(1, 12, 8)), g.normal(size=(1, 12, 8))
    chain = [(2 << t) - 1 for t in range(T)]
    a = oracle.tree_attention(q, K, V, None, 4, 3, chain, 0.2)
    b = oracle.tree_attention(q, K, V, None, 4, 3, None, 0.2)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
    K2, V2 = K.copy(), V.copy()
    K2[0, 11], V2[0, 11] = 1e9, -1e9                  # the last drafted token
    c = oracle.tree_attention(q, K2, V2, None, 4, 3, chain, 0.2)
    assert np.allclose(a[0][:4], c[0][:4])
    assert oracle.tree_sees([1 << 63], 0, 63) and not oracle.tree_sees([1 << 63], 0, 62)


def test_tree_row_that_sees_nothing_is_zero():
    q = rng(5).normal(size=(2, 1, 8))
    K = rng(6).normal(size=(1, 2, 8))
    out, lse, _ = oracle.tree_attention(q, K, K, None, 0, 0, [0, 2], 1.0)
    assert np.array_equal(out[0], np.zeros((1, 8))) and lse[0, 0] == -math.inf
    assert np.allclose(out[1, 0], K[0, 1])


def test_accept_moves_rows_down():
    X = np.arange(10.0).reshape(10, 1)
    assert np.array_equal(oracle.accept_path(X, 4, [0, 2, 5])[:, 0], [0, 1, 2, 3, 4, 6, 9, 7, 8, 9])


def test_page_book_conserves_references():
    """Forks, reservations and releases in any order: every held entry is one
    reference, no two writable entries share a page, and releasing everything
    frees everything."""
    g = rng(7)
    B, per, pages = 6, 8, 40
    book = oracle.PageBook(np.zeros(pages, int), np.full((B, per), -1), np.zeros(B, int))
    length = [0] * B
    book.reserve(length, [37, 0, 0, 0, 0, 0])
    length[0] = 37
    for _ in range(200):
        b, c = (int(x) for x in g.integers(0, B, 2))
        what = int(g.integers(0, 3))
        if what == 0 and b != c and book.n[c] == 0:
            book.fork([b], [c])
            length[c] = length[b]
        elif what == 1:
            new = [0] * B
            new[b] = int(g.integers(0, min(20, per * 16 - length[b]) + 1))
            book.reserve(length, new)
            if book.ok:
                for i in range(length[b] // 16, -(-(length[b] + new[b]) // 16) if new[b] else 0):
                    assert book.ref[book.table[b][i]] == 1
                length[b] += new[b]
        elif what == 2 and b:
            keep = [-1] * B
            keep[b] = int(g.integers(0, length[b] + 1))
            book.release(keep)
            length[b] = min(length[b], keep[b])
        held = [p for r, n in zip(book.table, book.n) for p in r[:n]]
        assert [held.count(p) for p in range(pages)] == book.ref
        assert all(-(-x // 16) <= n for x, n in zip(length, book.n))
    book.release([0] * B)
    assert book.ref == [0] * pages and book.n == [0] * B


def test_page_book_refuses_as_a_whole():
    book = oracle.PageBook([1, 0, 0], [[0, -1, -1], [-1, -1, -1]], [1, 0])
    book.reserve([16, 0], [1, 32])
    assert not book.ok and book.ref == [1, 0, 0] and book.n == [1, 0]
