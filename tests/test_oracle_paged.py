"""Pins of the paged-cache oracle: hand-worked tables and slots, brute force over every key of a
block, and agreement with plain softmax attention over the same tokens laid end to end."""
import numpy as np
import pytest

from oracle import attention as oattn
from oracle import paged


def test_extend_by_hand():
    """Blocks of 4 tokens, 2 heads.  Sequence 0 holds 3 tokens and takes 2 (one new block), 1 holds 4
    and takes none, 2 starts with 5 (two blocks), 3 wants more than its table holds, 4 finds the free
    list empty, 5 still has room in its block."""
    table = np.array([[7, -1], [3, -1], [-1, -1], [-1, -1], [-1, -1], [6, -1]])
    t, lens, granted, head, off, slots = paged.extend(table, [3, 4, 0, 0, 0, 1], [2, 0, 5, 9, 1, 2], [9, 8, 2, 5], 1, 21,
                                                      2, 4, 10)
    assert t.tolist() == [[7, 8], [3, -1], [2, 5], [-1, -1], [-1, -1], [6, -1]]
    assert lens.tolist() == [5, 4, 5, 0, 0, 3] and granted.tolist() == [2, 0, 5, 0, 0, 2]
    assert head == 4 and off.tolist() == [0, 2, 2, 7, 16, 17, 19]
    s = slots.reshape(21, 2)
    assert s[0].tolist() == [(7 * 2 + 0) * 4 + 3, (7 * 2 + 1) * 4 + 3] and s[1].tolist() == [64, 68]
    assert s[2:7, 0].tolist() == [16, 17, 18, 19, 40] and np.all(s[7:17] == -1)
    assert s[17].tolist() == [49, 53] and np.all(s[19:] == -1)


def test_extend_slots_are_the_attention_oracles():
    lens, new = [0, 17, 40], [33, 15, 1]
    table = np.full((3, 4), -1)
    table[1, :2], table[2, :3] = [11, 4], [0, 1, 2]
    free = [5, 6, 7, 8, 9]
    t, after, granted, _, off, slots = paged.extend(table, lens, new, free, 0, sum(new), 3, 16, 12)
    assert granted.tolist() == new
    for b in range(3):
        for h in range(3):
            want = oattn.token_slots(b, h, int(after[b]), 3, block_table=t)[lens[b]:]
            assert np.array_equal(slots.reshape(-1, 3)[off[b]:off[b + 1], h], want)


def test_refused_sequence_leaves_later_ones_without_blocks():
    """The free list serves sequences in order: after one that it cannot serve, a later one that
    needs a block is refused even where one block is left."""
    t, lens, granted, head, _, slots = paged.extend(np.full((3, 4), -1), [0, 0, 0], [4, 12, 4], [1, 2, 3], 0, 20, 1, 4, 4)
    assert granted.tolist() == [4, 0, 0] and head == 1 and np.all(slots[4:] == -1)


def test_bounds_and_scores_brute_force():
    rng = np.random.default_rng(0)
    n_kv, group, d, block = 2, 3, 8, 4
    k = rng.standard_normal((11, n_kv, d))
    caches = [np.zeros((5, n_kv, block, d)) for _ in range(2)]
    bounds = np.full((5, n_kv, 2, d), 99.0)
    table = np.array([[4, 1, 2]])
    for n, m in ((6, 6), (7, 1), (11, 4)):   # 6 tokens, then one, then four
        at = [0, m]
        *caches, bounds = paged.append(table, [n], [m], at, k[n - m:n], -k[n - m:n], *caches, bounds, block)
    for j, e in enumerate(table[0]):
        x = k[4 * j:4 * j + 4]
        assert np.array_equal(bounds[e, :, 0], x.min(0)) and np.array_equal(bounds[e, :, 1], x.max(0))
        assert np.array_equal(caches[0][e, :, :len(x)], x.transpose(1, 0, 2))
        assert np.array_equal(caches[1][e, :, :len(x)], -x.transpose(1, 0, 2))
    q = rng.standard_normal((1, n_kv * group, d))
    s = paged.block_scores(table, [11], q, bounds, block)
    for h in range(n_kv):
        for j in range(3):
            # the largest over every corner of the box, channel by channel, and above every key's product
            corners = [max(sum(max(x[c] * bounds[table[0, j], h, 0, c], x[c] * bounds[table[0, j], h, 1, c])
                               for c in range(d)) for x in q[0, h * group:(h + 1) * group])]
            assert s[h, j] == pytest.approx(corners[0])
            assert np.all(k[4 * j:4 * j + 4, h] @ q[0, h * group:(h + 1) * group].T <= s[h, j] + 1e-12)
    assert np.all(paged.block_scores(table, [4], q, bounds, block)[:, 1:] == -np.inf)


def test_select_by_hand():
    """Ten blocks, one of them forced in front, two behind; ties go to the lower index."""
    table = np.arange(10)[None] + 20
    scores = np.array([[0, 5, 1, 7, 5, 5, -3, np.nan, 100, 100.0]])
    t, n = paged.select(table, [10 * 8 - 3], scores, 1, 8, 40, 5, 1, 2)
    assert t.tolist() == [[20, 21, 23, 28, 29]] and n.tolist() == [4 * 8 + 5]
    t, n = paged.select(table, [10], scores, 1, 8, 21, 5, 1, 2)
    assert t.tolist() == [[20, -1, -1, -1, -1]] and n.tolist() == [10]
    t, n = paged.select(table, [0], scores, 1, 8, 40, 5, 1, 2)
    assert t.tolist() == [[-1] * 5] and n.tolist() == [0]


def test_attend_is_plain_softmax_attention():
    rng = np.random.default_rng(1)
    lens, n_kv, group, d, block = [9, 0, 1, 12], 2, 2, 8, 4
    table = rng.permutation(12).reshape(4, 3)
    kc, vc = rng.standard_normal((2, 12, n_kv, block, d))
    q = rng.standard_normal((4, n_kv * group, d))
    out = paged.attend(table, lens, q, kc, vc, block)
    for b, n in enumerate(lens):
        for hq in range(n_kv * group):
            h = hq // group
            k = np.concatenate([kc[e, h] for e in table[b]])[:n]
            v = np.concatenate([vc[e, h] for e in table[b]])[:n]
            if n == 0:
                assert np.all(out[b, hq] == 0)
                continue
            w = np.exp(k @ q[b, hq] / np.sqrt(d))
            np.testing.assert_allclose(out[b, hq], (w[:, None] * v).sum(0) / w.sum(), rtol=1e-12)
    # every block chosen: the selected table gives the same attention, one KV head at a time
    t, n = paged.select(table, lens, np.zeros((8, 3)), n_kv, block, 12, 3, 0, 1)
    flat = paged.attend(t, n, q.reshape(8, group, d), kc.reshape(24, 1, block, d), vc.reshape(24, 1, block, d), block)
    np.testing.assert_allclose(flat.reshape(out.shape), out, rtol=1e-12)


