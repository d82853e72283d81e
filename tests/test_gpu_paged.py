"""The paged-cache calls (tq_page_extend, tq_append_kv, tq_block_scores, tq_select_blocks,
tq_attend_paged) against the fp64 oracle, each alone and run together as a serving step.

Whole numbers and copies are equal.  Tolerances of the others count roundings of 32-bit arithmetic:
  products   bf16 x bf16 is exact in fp32.  An fp32 product made of TF32 parts: the query's or weight's parts are
             rounded to 11 bits each, which leaves 2^-22 of it; the cached value's head is cut to 11 bits, so its
             tail is below 2^-10 of it, and cutting that to 11 bits leaves 2^-20; the product of the two
             tails, below 2^-10 x 2^-11, is dropped.  Together (1 + 4 + 2) x 2^-22 of |x y|
  sums       n terms in any order: at most n roundings of 2^-23 (a tensor core's sum may truncate) of the
             sum of the absolute terms
  softmax    a logit that is off by e moves its weight by a factor e^(+-e); exp itself is within 2^-21; the
             weights, the value products and the sums then round like the above
  output     half a step of the output's type"""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import attention as oattn
from oracle import paged
from parity import Quantizer, assert_attention_close, oracle_heads

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def tq():
    from kv_cache_vector_06_b200 import tq as _tq
    return _tq


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def rows(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def tables(lens, width, block, seed, spare=3):
    """A block table with the blocks of `lens` in one random order (-1 behind them) and the number of blocks."""
    rng = np.random.default_rng(seed)
    held = [-(-n // block) for n in lens]
    n_blocks = sum(held) + spare
    perm = rng.permutation(n_blocks)
    t = np.full((len(lens), width), -1)
    at = 0
    for b, k in enumerate(held):
        t[b, :k] = perm[at:at + k]
        at += k
    return t, n_blocks


# ------------------------------------------------------------------------------------ page_extend
def check_extend(tq, table, lens, new, free, head, n_rows, n_kv, block, n_blocks, in_place):
    pages = tq.Pages(i32(table), n_kv, block, n_blocks)
    l, g, hd = i32(lens), i32(new), i32([head])
    outs = dict(seq_lens_out=l, granted=g, free_head_out=hd) if in_place else {}
    slots, after, granted, head2, off = tq.page_extend(pages, l, g, i32(free), hd, n_rows=n_rows, **outs)
    ref = paged.extend(table, lens, new, free, head, n_rows, n_kv, block, n_blocks)
    got = [x.cpu().numpy() for x in (pages.block_table, after, granted, head2, off, slots)]
    for name, x, y in zip(("table", "lens", "granted", "head", "offsets", "slots"), got, ref):
        assert np.array_equal(x.reshape(-1), np.asarray(y).reshape(-1)), name


@pytest.mark.parametrize("batch,n_kv,block,lo,hi,most", [(1, 1, 1, 0, 0, 1), (1, 8, 16, 40, 40, 1), (7, 3, 24, 0, 90, 50),
                                                        (64, 8, 16, 0, 300, 1), (33, 2, 128, 0, 700, 400),
                                                        (2500, 1, 16, 0, 60, 9), (3, 5, 7, 100, 3000, 20000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(tq, batch, n_kv, block, lo, hi, most, in_place):
    rng = np.random.default_rng(batch + block)
    lens, new = rng.integers(lo, hi + 1, batch), rng.integers(0, most + 1, batch)
    width = -(-(hi + most) // block)
    table, used = tables(lens, width, block, seed=1)
    need = int(sum(-(-(n + m) // block) - -(-n // block) for n, m in zip(lens, new)))
    free = rng.permutation(used + need + 4)
    for short, pad in ((0, 11), (max(1, need // 3), 0), (-2, -(int(new.sum()) // 2))):
        # enough blocks; too few of them; too few rows
        n_free = max(2, 2 + need - short)
        check_extend(tq, table, lens, new, free[:n_free], 2, int(new.sum()) + pad, n_kv, block, used + need + 4, in_place)


def test_extend_odd_values(tq):
    """Negative lengths, a length past the table, nothing to add, no rows at all, free entries and table
    entries that name no block, a head past the list, sums past 32 bits."""
    table = np.array([[0, 1, 2], [3, -1, 9], [4, 99, 5], [-7, -1, -1], [6, 7, 8]])
    for lens, new, free, head in (([-3, 5, 9, 2, 0], [4, 0, 2, 1, -5], [50, 11, 12], 0), ([12, 13, 2, 0, 1], [1, 1, 3, 12, 12], [10, -1, 11, 12, 13, 14], 1),
                                  ([1, 1, 1, 1, 1], [9, 9, 9, 9, 9], [10, 11], 7), ([1, 1, 1, 1, 1], [2**31 - 1] * 5, [10], 0)):
        for n_rows in (0, 1, 30):
            lens0 = [max(x, 0) for x in lens]
            if n_rows and head <= len(free):
                check_extend(tq, table, lens0, new, free, head, n_rows, 2, 4, 20, False)
            pages = tq.Pages(i32(table), 2, 4, 20)
            slots, after, granted, head2, off = tq.page_extend(pages, i32(lens), i32(new), i32(free), i32([head]), n_rows=n_rows)
            ref = paged.extend(table, lens, new, free, min(head, len(free)), n_rows, 2, 4, 20)
            assert np.array_equal(slots.cpu().numpy(), ref[5]) and np.array_equal(off.cpu().numpy(), ref[4])
            assert after.tolist() == ref[1].tolist() and granted.tolist() == ref[2].tolist() and head2.item() == ref[3]
    pages = tq.Pages(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 2, 4, 20)
    none = i32([])
    slots, _, _, head, off = tq.page_extend(pages, none, none, i32([1, 2]), i32([1]), n_rows=3)
    assert slots.tolist() == [-1] * 6 and head.item() == 1 and off.tolist() == [0]


def test_extend_many_heads(tq):
    """More heads than a block has threads, whole prompts and single tokens."""
    for n_kv in (1100, 514):
        table, used = tables([5, 0, 16], 9, 16, seed=1)
        check_extend(tq, table, [5, 0, 16], [100, 7, 1], np.arange(used, used + 12), 1, 120, n_kv, 16, used + 12, False)


def test_extend_is_stable_under_shifted_slots(tq):
    """new_slots at any 8-byte address (the wide stores want 16 or 32)."""
    for n_kv in (8, 2, 3):
        buf = torch.full((600 * n_kv + 8,), 77, dtype=torch.int64).cuda()
        for shift in (0, 1, 2, 4):
            table, used = tables([30, 0], 40, 16, seed=2)
            pages, free = tq.Pages(i32(table), n_kv, 16, used + 60), np.arange(used, used + 50)
            slots = buf[shift:shift + 600 * n_kv]
            tq.page_extend(pages, i32([30, 0]), i32([1, 555]), i32(free), i32([0]), new_slots=slots)
            ref = paged.extend(table, [30, 0], [1, 555], free, 0, 600, n_kv, 16, used + 60)
            assert np.array_equal(slots.cpu().numpy(), ref[5]) and buf[600 * n_kv + shift:].eq(77).all()
            buf.fill_(77)


# ------------------------------------------------------------------------------------ append_kv
def append_case(tq, lens, granted, n_kv, block, d, dtype, seed, gap=0, offsets=None, table=None, caches=True, with_bounds=True,
                n_rows=None):
    """lens: after the append."""
    width = max(1, max(-(-n // block) for n in lens) + 1)
    if table is None:
        table, n_blocks = tables(lens, width, block, seed)
    else:
        n_blocks = int(np.max(table)) + 1
    off = np.concatenate([[0], np.cumsum(granted)]) if offsets is None else np.asarray(offsets)
    n = int(off[-1]) if n_rows is None else n_rows
    kv = rows(n, 2, n_kv * d + gap, seed=seed, dtype=dtype).cuda()
    k, v = (kv[:, i, :n_kv * d].unflatten(1, (n_kv, d)) for i in (0, 1))
    kc, vc = (torch.full((n_blocks, n_kv, block, d), math.nan, dtype=dtype).cuda() for _ in (0, 1))
    bd = rows(n_blocks, n_kv, 2, d, seed=seed + 1, dtype=dtype).sort(2).values.cuda()
    pages = tq.Pages(i32(table), n_kv, block, n_blocks)
    before = [x.double().cpu().numpy() for x in (kc, vc, bd)]
    tq.append_kv(pages, i32(lens), i32(granted), torch.as_tensor(off).cuda(), k, v if caches else None,
                 kc if caches else None, vc if caches else None, bd if with_bounds else None)
    grown = [g if off[b] + g <= n else 0 for b, g in enumerate(granted)]
    ref = paged.append(table, lens, grown, off, k.double().cpu().numpy(), v.double().cpu().numpy(), *before, block)
    for name, x, y, z, on in zip(("k_cache", "v_cache", "bounds"), (kc, vc, bd), ref, before, (caches, caches, with_bounds)):
        np.testing.assert_array_equal(x.double().cpu().numpy(), y if on else z, err_msg=name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,n_kv,block", [(128, 8, 16), (64, 1, 16), (80, 3, 24), (256, 2, 128), (8, 5, 1), (192, 2, 7), (96, 16, 64)])
def test_append(tq, dtype, d, n_kv, block):
    append_case(tq, [1, 16, 17, 100, 33, 700, 5], [1, 16, 1, 99, 0, 650, 5], n_kv, block, d, dtype, seed=d + block, gap=24)


@pytest.mark.parametrize("granted", [[1], [0], [4]])
def test_append_one_sequence(tq, granted):
    append_case(tq, [37], granted, 2, 16, 128, BF16, seed=3, n_rows=4)


def test_append_one_row_beside_a_joint_projection(tq):
    """One row: keys from a projection's output, values by themselves, whose row strides differ and do not matter."""
    n_kv, d, block = 2, 64, 16
    joint = rows(1, 2, n_kv, d, seed=1, dtype=BF16).cuda()
    k, v = joint[:, 0], rows(1, n_kv, d, seed=2, dtype=BF16).cuda()
    assert k.stride(0) != v.stride(0)
    kc, vc = (torch.zeros(3, n_kv, block, d, dtype=BF16).cuda() for _ in (0, 1))
    tq.append_kv(tq.Pages(i32([[2]]), n_kv, block, 3), i32([5]), i32([1]), torch.tensor([0, 1]).cuda(), k, v, kc, vc)
    assert torch.equal(kc[2, :, 4], k[0]) and torch.equal(vc[2, :, 4], v[0]) and kc.count_nonzero() == k.count_nonzero()


def test_append_refused_rows_and_bounds_only(tq):
    """Refused sequences keep their rows unread (offsets count them); a sequence whose rows pass n_rows is
    not appended; caches and bounds each without the other; table entries that name no block."""
    lens, granted, off = [20, 7, 40, 9], [20, 0, 3, 9], [0, 20, 31, 34, 43]
    for kw in (dict(), dict(caches=False), dict(with_bounds=False), dict(n_rows=40)):
        append_case(tq, lens, granted, 2, 16, 64, BF16, seed=5, offsets=off, **kw)
    table = np.array([[3, -1, 4], [0, 0, 0], [1, 2, 70000], [-5, 6, 6]])
    table[2, 2] = -9
    append_case(tq, [40, 0, 48, 30], [33, 0, 48, 20], 2, 16, 64, F32, seed=6, table=table)


@pytest.mark.parametrize("first", [1, 16, 40, 333])
def test_append_rows_that_begin_later(tq, first):
    """The later sequences of a batch alone: their first row lies behind rows of k_new that nobody appends."""
    lens, granted = [100, 17, 64], [20, 1, 64]
    off = first + np.concatenate([[0], np.cumsum(granted)])
    for dtype, n_kv in ((BF16, 2), (F32, 9)):
        append_case(tq, lens, granted, n_kv, 16, 128, dtype, seed=first, offsets=off)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [8, 128, 256])
def test_append_bounds_pass_over_nan(tq, dtype, d):
    """A channel's bounds are those of its other values, and NaN where it has none."""
    k = rows(40, 2, d, seed=d, dtype=dtype).cuda()
    k[0, 0, 0] = k[39, 0, 1] = math.nan
    k[5, 1] = math.nan
    k[16:32, 0, 3] = math.nan
    pages = tq.Pages(i32([[0, 1, 2]]), 2, 16, 3)
    bd = torch.zeros(3, 2, 2, d, dtype=dtype).cuda()
    tq.append_kv(pages, i32([40]), i32([40]), torch.tensor([0, 40]).cuda(), k, bounds=bd)
    for j in range(3):
        x = k[16 * j:16 * j + 16].double().cpu().numpy()
        ref = np.stack([np.fmin.reduce(x, axis=0), np.fmax.reduce(x, axis=0)], axis=1)
        np.testing.assert_array_equal(bd[j].double().cpu().numpy(), ref)


# ------------------------------------------------------------------------------------ block_scores
def check_scores(tq, lens, n_kv, group, block, d, dtype, seed, width=None, table=None):
    if table is None:
        table, n_blocks = tables([max(n, 0) for n in lens], width or max(1, max(-(-n // block) for n in lens)), block, seed)
    else:
        n_blocks = 7
    bd = (rows(n_blocks, n_kv, 2, d, seed=seed, dtype=dtype) * torch.exp(rows(n_kv, 1, d, seed=seed + 1, dtype=dtype))).sort(2).values.cuda()
    q = rows(len(lens), n_kv * group, d, seed=seed + 2, dtype=dtype).cuda()
    pages = tq.Pages(i32(table), n_kv, block, n_blocks)
    got = tq.block_scores(pages, i32(lens), q, bd).double().cpu().numpy()
    b64, q64 = bd.double().cpu().numpy(), q.double().cpu().numpy()
    ref = paged.block_scores(table, lens, q64, b64, block)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)) and np.all(got[~np.isfinite(ref)] == -np.inf)
    # sum of the absolute terms of the largest query head bounds every head's rounding
    big = paged.block_scores(table, lens, np.abs(q64), np.repeat(np.abs(b64).max(2, keepdims=True), 2, axis=2), block)
    fin = np.isfinite(ref)
    tol = (2 * d * 2.0 ** -23 + 3 * 2.0 ** -22) * big[fin]
    assert np.all(np.abs(got[fin] - ref[fin]) <= tol), np.max(np.abs(got[fin] - ref[fin]) / tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,n_kv,group,block", [(128, 8, 4, 16), (64, 1, 1, 16), (80, 3, 5, 24), (256, 2, 8, 128), (8, 2, 16, 1),
                                                (192, 2, 7, 32), (96, 4, 2, 64), (128, 1, 16, 8), (256, 1, 9, 16), (128, 2, 8, 16)])
def test_scores(tq, dtype, d, n_kv, group, block):
    check_scores(tq, [1, 0, 16, 17, 1000, 333, 2049, 5], n_kv, group, block, d, dtype, seed=d + group)


def test_scores_odd_tables(tq):
    """Entries that name no block, a table wider than the sequences, a length past the table, a negative one."""
    t = np.array([[0, -1, 5, 3, 7], [6, 100, -4, 2, 1], [1, 2, 3, 4, 5], [5, 5, 5, 5, 5]])
    check_scores(tq, [80, 65, -4, 200], 2, 4, 16, 128, BF16, seed=9, table=t)
    check_scores(tq, [80, 65, -4, 200], 2, 4, 16, 64, F32, seed=9, table=t)
    check_scores(tq, [3, 30], 2, 4, 16, 128, BF16, seed=10, width=70)


def test_scores_bound_the_keys(tq):
    """Scores from appended bounds are not below any key's product (the sums' rounding apart)."""
    n, n_kv, group, d, block = 1000, 2, 4, 128, 16
    table, n_blocks = tables([n], 63, block, 4)
    pages = tq.Pages(i32(table), n_kv, block, n_blocks)
    k = rows(n, n_kv, d, seed=1, dtype=BF16).cuda()
    bd = torch.empty(n_blocks, n_kv, 2, d, dtype=BF16).cuda()
    tq.append_kv(pages, i32([n]), i32([n]), torch.tensor([0, n]).cuda(), k, bounds=bd)
    q = rows(1, n_kv * group, d, seed=2, dtype=BF16).cuda()
    s = tq.block_scores(pages, i32([n]), q, bd).double().cpu()
    prod = torch.einsum("hgd,nhd->hgn", q.double().cpu().view(n_kv, group, d), k.double().cpu()).amax(1)
    best = torch.nn.functional.pad(prod, (0, 63 * 16 - n), value=-math.inf).view(n_kv, 63, 16).amax(2)
    assert torch.all(best <= s + 1e-3) and torch.all(s < best + 200)


# ------------------------------------------------------------------------------------ select_blocks
def check_select(tq, lens, scores, n_kv, block, keep, first, last, seed=0, table=None):
    width = scores.shape[1]
    if table is None:
        table, n_blocks = tables([min(max(n, 0), width * block) for n in lens], width, block, seed)
    else:
        n_blocks = 9
    pages = tq.Pages(i32(table), n_kv, block, n_blocks)
    t, n = tq.select_blocks(pages, i32(lens), torch.as_tensor(scores, dtype=F32).cuda(), keep, n_first=first, n_last=last)
    rt, rn = paged.select(table, lens, scores.astype(np.float32).astype(np.float64), n_kv, block, n_blocks, keep, first, last)
    assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(n.cpu().numpy(), rn)


@pytest.mark.parametrize("n_kv,block,width,keep,first,last", [(1, 16, 1, 1, 0, 1), (2, 16, 40, 8, 1, 2), (3, 24, 600, 64, 4, 8),
                                                             (2, 1, 5000, 1000, 0, 1), (1, 64, 33, 33, 1, 1), (1, 16, 100, 300, 2, 3),
                                                             (2, 16, 9000, 3, 1, 2), (1, 8, 70000, 257, 1, 4), (1, 8, 513, 512, 0, 512)])
def test_select(tq, n_kv, block, width, keep, first, last):
    rng = np.random.default_rng(width + keep)
    lens = [width * block, 0, 1, width * block - 1, (width * block + 1) // 2, min(width, keep) * block, min(width, keep + 1) * block]
    for kind in range(3):
        s = rng.standard_normal((len(lens) * n_kv, width))
        if kind == 1:
            s = np.round(s * 2)  # many ties, -0 and +0 among them
        if kind == 2:
            s = s * 1e-30 * (rng.random(s.shape) < 0.5) - (rng.random(s.shape) < 0.3) * 1e30
        check_select(tq, lens, s, n_kv, block, keep, first, last)


def test_select_odd_scores(tq):
    """All equal; infinities and NaN; scores behind the last block are not read as candidates; lengths past
    the table; entries that name no block."""
    inf, nan = math.inf, math.nan
    lens = [160, 1000, -2, 75]
    s = np.zeros((4, 10))
    check_select(tq, lens, s, 1, 16, 4, 1, 1)
    s[0] = [inf, nan, -inf, inf, 0.0, -0.0, nan, 3, -inf, 1]
    s[1] = nan
    s[3] = [1, 2, 3, 4, 5, inf, nan, inf, nan, inf]
    for keep in (2, 3, 4, 5, 9):
        check_select(tq, lens, s, 1, 16, keep, 1, 1)
    t = np.array([[0, 1, -1, 3, 50, 5, 6, 7, 8, 2]] * 4)
    check_select(tq, lens, s, 1, 16, 6, 0, 1, table=t)


# ------------------------------------------------------------------------------------ attend_paged
def attend_tolerance(table, lens, q, kc, vc, block, scale, dtype, out_dtype):
    """Bound on |out - reference| [batch, n_q, d] by the counts of this file's docstring."""
    n_kv, d = kc.shape[1], q.shape[2]
    group = q.shape[1] // n_kv
    tol = np.zeros(q.shape)
    for b in range(len(lens)):
        t = np.arange(max(int(lens[b]), 0))
        e = np.asarray(table[b], dtype=np.int64)[t // block]
        ok = (e >= 0) & (e < kc.shape[0])
        t, e = t[ok] % block, e[ok]
        for hq in range(q.shape[1]) if len(t) else ():
            k, v = kc[e, hq // group, t], vc[e, hq // group, t]
            s = scale * (k @ q[b, hq])
            mag = abs(scale) * (np.abs(k) @ np.abs(q[b, hq]))  # the absolute terms, whatever the sign of scale
            off = np.max(mag) * (d * 2.0 ** -23 + 7 * 2.0 ** -22) + 2 * np.max(np.abs(s)) * 2.0 ** -23 + 2.0 ** -20
            w = np.exp(s - s.max())
            w /= w.sum()
            av = w @ np.abs(v)
            o = np.abs(w @ v)
            tol[b, hq] = (2 * off + (2 * len(t) + 8) * 2.0 ** -23 + 7 * 2.0 ** -22) * av
            tol[b, hq] += torch.finfo(out_dtype).eps / 2 * (o + tol[b, hq])
    return tol


def check_attend(tq, lens, n_kv, group, block, d, dtype, out_dtype=F32, seed=0, scale=0.0, table=None, max_len=None, poison=True,
                 key_scale=1.0, ws=None):
    width = max(1, max(-(-max(n, 0) // block) for n in lens))
    if table is None:
        table, n_blocks = tables([max(n, 0) for n in lens], width, block, seed)
    else:
        n_blocks = 9
        width = np.shape(table)[1]
    kc, vc = (rows(n_blocks, n_kv, block, d, seed=seed + i, dtype=dtype) for i in (1, 2))
    kc = (kc * key_scale).to(dtype)
    ref_k, ref_v = kc.double().numpy(), vc.double().numpy()
    if poison:
        # whatever lies outside the sequences must not be looked at
        held = torch.zeros(n_blocks, block, dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in range(min(max(n, 0), width * block if max_len is None else max_len)):
                if 0 <= table[b][t // block] < n_blocks:
                    held[table[b][t // block], t % block] = True
        bad = (~held)[:, None, :, None].expand_as(kc)
        kc, vc = kc.masked_fill(bad, math.nan), vc.masked_fill(bad, math.inf)
    q = rows(len(lens), n_kv * group, d, seed=seed + 3, dtype=dtype)
    pages = tq.Pages(i32(table), n_kv, block, n_blocks)
    max_len = width * block if max_len is None else max_len
    out = torch.full(q.shape, math.nan, dtype=out_dtype).cuda()
    got = tq.attend_paged(pages, i32(lens), max_len, q.cuda(), kc.cuda(), vc.cuda(), scale=scale, out=out, ws=ws)
    got = got.double().cpu().numpy()
    n = [min(max(x, 0), max_len) for x in lens]
    q64 = q.double().numpy()
    ref = paged.attend(table, n, q64, ref_k, ref_v, block, scale)
    tol = attend_tolerance(table, n, q64, ref_k, ref_v, block, scale or d ** -0.5, dtype, out_dtype)
    err = np.abs(got - ref)
    assert np.all(err <= tol), f"{np.max(err[tol > 0] / tol[tol > 0])} of the tolerance, zeros {np.max(err[tol == 0], initial=0)}"
    assert np.all(got[[x == 0 for x in n]] == 0)
    # the same rows under a bound on their lengths so large that they are dealt out in pieces
    wide = np.concatenate([table, np.full((len(lens), -(-200000 // block)), -1)], axis=1)
    cut = [min(x, max_len) for x in lens]
    out = torch.full(q.shape, math.nan, dtype=out_dtype).cuda()
    got2 = tq.attend_paged(tq.Pages(i32(wide), n_kv, block, n_blocks), i32(cut), wide.shape[1] * block, q.cuda(), kc.cuda(), vc.cuda(),
                           scale=scale, out=out)
    assert np.all(np.abs(got2.double().cpu().numpy() - ref) <= tol)
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,n_kv,group,block", [(128, 8, 4, 16), (64, 1, 1, 16), (80, 3, 5, 24), (256, 2, 8, 128), (8, 2, 16, 1),
                                                (192, 2, 7, 32), (96, 4, 2, 64), (128, 1, 16, 8), (256, 1, 9, 16), (128, 2, 8, 16),
                                                (64, 2, 12, 5), (16, 1, 3, 16), (120, 2, 6, 16)])
def test_attend(tq, dtype, d, n_kv, group, block):
    check_attend(tq, [1, 0, 16, 17, 1000, 333, 2049, 5], n_kv, group, block, d, dtype, seed=d + group)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[1], [0], [15], [16], [9001], [40000], [0, 0, 0], [4096] * 3, [20000, 1, 1, 1, 1, 1, 1, 1]])
def test_attend_lengths(tq, dtype, lens):
    check_attend(tq, lens, 2, 4, 16, 128, dtype, seed=len(lens) + lens[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_long_sums_do_not_shrink(tq, dtype):
    """Equal weights over values of one sign, some 120 steps per warp: sums rounded to nearest stay within a few
    roundings (2^-24 x sqrt(120) x 4, and 8 cuts of 2^-23 inside a step: 3.6e-6 at the very most, 1e-6 as it comes);
    a sum cut at each step loses half of 2^-23 every time, 7e-6."""
    batch, n_kv, d, block, n = 16, 8, 64, 16, 20000
    table = torch.randperm(batch * n // block, generator=torch.Generator().manual_seed(1)).view(batch, -1).to(torch.int32)
    v = (torch.rand(batch * n // block, n_kv, block, d, generator=torch.Generator("cuda").manual_seed(2), device="cuda") + 1).to(dtype)
    pages = tq.Pages(table.cuda(), n_kv, block, batch * n // block)
    q = torch.zeros(batch, 2 * n_kv, d, dtype=dtype).cuda()
    got = tq.attend_paged(pages, i32([n] * batch), n, q, torch.zeros_like(v), v).double()
    ref = v[table.long().cuda()].double().mean((1, 3)).repeat_interleave(2, dim=1)
    err = (got - ref) / ref
    assert err.abs().max() <= 3.6e-6 and err.mean().abs() <= 1.5e-6, (err.abs().max(), err.mean())


@pytest.mark.parametrize("dtype,d,group", [(BF16, 128, 4), (F32, 64, 4), (F32, 128, 16), (BF16, 64, 16)])
@pytest.mark.parametrize("lens", [[9999, 12000, 16], [300, 500, 16]])
def test_attend_passes_nan_on(tq, dtype, d, group, lens):
    """NaN in one head's query, in one token's key of one KV head and in one value: exactly the outputs that
    read them are NaN, for rows that several blocks share and for whole ones, and the others are as without."""
    n_kv, block = 2, 16
    table, n_blocks = tables(lens, -(-max(lens) // block), block, seed=4)
    q, k, v = (rows(*s, seed=i, dtype=dtype).cuda() for i, s in
               enumerate([(3, n_kv * group, d), (n_blocks, n_kv, block, d), (n_blocks, n_kv, block, d)]))
    pages = tq.Pages(i32(table), n_kv, block, n_blocks)
    clean = tq.attend_paged(pages, i32(lens), max(lens), q, k, v)
    assert clean.isfinite().all()
    bad = torch.zeros_like(clean, dtype=torch.bool)
    q[0, 1, 3] = math.nan
    bad[0, 1] = True
    k[int(table[1][200 // block]), 1, 200 % block, 5] = math.nan
    bad[1, group:] = True
    v[int(table[2][0]), 0, 7, d - 1] = math.nan
    bad[2, :group, d - 1] = True
    got = tq.attend_paged(pages, i32(lens), max(lens), q, k, v)
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], clean[~bad])


def test_attend_many_sequences(tq):
    """More rows than the GPU has room for at once, ragged."""
    rng = np.random.default_rng(0)
    check_attend(tq, rng.integers(0, 200, 301).tolist(), 3, 2, 16, 64, BF16, seed=8)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_bf16_output(tq, d):
    check_attend(tq, [700, 0, 31, 3000], 2, 4, 16, d, BF16, out_dtype=BF16, seed=11)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_scales_and_sharp_softmax(tq, dtype):
    """A given scale, a negative one, and logits so far apart that one token holds the weight."""
    for scale, key_scale in ((1.0, 1.0), (-0.25, 1.0), (0.0, 16.0)):
        check_attend(tq, [500, 3, 1500], 2, 4, 16, 128, dtype, seed=12, scale=scale, key_scale=key_scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_odd_tables(tq, dtype):
    """Entries that name no block leave their tokens out (a row of nothing else gives zeros), blocks shared by
    two sequences, lengths past max_seq_len and negative ones."""
    t = np.array([[0, -1, 5, 3], [100, -4, 9, 1 << 30], [5, 2, 3, 4], [1, 2, -1, -1]])
    check_attend(tq, [64, 64, 50, 40], 2, 4, 16, 128, dtype, seed=13, table=t)
    check_attend(tq, [1000, -5, 33, 30], 2, 4, 16, 64, dtype, seed=14, table=t, max_len=33)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_no_tokens_at_all(tq, dtype):
    check_attend(tq, [5, 0, 9], 2, 4, 16, 64, dtype, seed=15, max_len=0)


def test_attend_workspace_reused(tq):
    """One workspace, filled with NaN, for calls of different shapes in a row."""
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8).cuda()
    for seed, lens in enumerate(([3000, 20, 700], [40], [9000], [1, 0, 2], [3000, 20, 700])):
        check_attend(tq, lens, 2, 4, 16, 128, BF16, seed=20 + seed, ws=ws)


def test_attend_workspace_reused_by_shared_rows(tq):
    """One workspace, filled with NaN, for calls whose rows are all cut into pieces that lie in it: other shapes, head
    counts and types in a row."""
    ws = torch.full((1 << 25,), 255, dtype=torch.uint8).cuda()
    for seed, (lens, group, d, dtype) in enumerate((([9001, 20, 700], 4, 128, BF16), ([12000], 8, 64, F32), ([9500] * 5, 1, 128, F32),
                                                    ([10000, 0, 1], 16, 64, BF16), ([9001, 20, 700], 4, 128, BF16))):
        check_attend(tq, lens, 2, group, 16, d, dtype, seed=30 + seed, ws=ws)


@pytest.mark.parametrize("dtype,out_dtype,d,group", [
    (BF16, F32, 64, 1), (BF16, BF16, 64, 16), (BF16, F32, 80, 4), (BF16, BF16, 128, 4), (BF16, F32, 128, 9), (BF16, F32, 192, 5),
    (BF16, BF16, 256, 8), (BF16, F32, 256, 16), (F32, F32, 64, 4), (F32, F32, 64, 16), (F32, F32, 80, 1), (F32, F32, 128, 4),
    (F32, F32, 128, 16), (F32, F32, 192, 9), (F32, F32, 256, 4), (F32, F32, 256, 16)])
def test_attend_many_short_rows(tq, dtype, out_dtype, d, group):
    """More rows than the GPU has room for, of few steps each, which single warps take; rows of a long one among them
    are shared by many warps."""
    rng = np.random.default_rng(d + group)
    lens = rng.integers(0, 60, 301)
    lens[rng.integers(0, 301)] = 3001
    check_attend(tq, lens.tolist(), 3, group, 16, d, dtype, out_dtype=out_dtype, seed=d + group)


def test_attend_captured_calls_share_a_workspace(tq):
    """Two captured calls of different shapes and an eager one on one workspace, replayed in turn: the same bits
    every time, whatever the call before left there."""
    d, block, group = 128, 16, 4
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8).cuda()
    calls = []
    for lens, n_kv in (([30000, 20, 700], 2), ([19000], 1), ([5, 4000, 0, 33] * 40, 4)):
        table, n_blocks = tables(lens, max(-(-n // block) for n in lens), block, seed=n_kv)
        kc, vc = (rows(n_blocks, n_kv, block, d, seed=s, dtype=BF16).cuda() for s in (1, 2))
        q, out = rows(len(lens), n_kv * group, d, seed=3, dtype=BF16).cuda(), torch.empty(len(lens), n_kv * group, d).cuda()
        pages, n = tq.Pages(i32(table), n_kv, block, n_blocks), i32(lens)
        calls.append((lambda p=pages, n=n, m=table.shape[1] * block, q=q, k=kc, v=vc, o=out:
                      tq.attend_paged(p, n, m, q, k, v, out=o, ws=ws), out))
    want = []
    for call, out in calls:
        ws.random_(256)
        want.append(call().clone())
    graphs = []
    for call, out in calls[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g.replay)
    for i in (0, 1, 1, 0, 2, 0, 0, 2, 1, 2, 0):
        calls[i][1].fill_(math.nan)
        (graphs + [calls[2][0]])[i]()
        assert torch.equal(calls[i][1], want[i]), i


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_offsets(tq, dtype):
    """A cache whose element offsets pass 2^32: append to its last blocks, then score and attend there."""
    d, n_kv, block = 128, 4, 16
    n_blocks = (1 << 32) // (d * n_kv * block) + 500
    kc, vc = (torch.empty(n_blocks, n_kv, block, d, dtype=dtype, device="cuda") for _ in (0, 1))
    bd = torch.empty(n_blocks, n_kv, 2, d, dtype=dtype, device="cuda")
    n, group = 900, 2
    rng = np.random.default_rng(1)
    held = -(-n // block)
    table = np.stack([n_blocks - 1 - rng.permutation(400)[:held], rng.permutation(400)[:held]])
    k, v = (rows(2 * n, n_kv, d, seed=s, dtype=dtype) for s in (1, 2))
    pages = tq.Pages(i32(table), n_kv, block, n_blocks)
    lens = i32([n, n])
    tq.append_kv(pages, lens, lens, torch.tensor([0, n, 2 * n]).cuda(), k.cuda(), v.cuda(), kc, vc, bd)
    q = rows(2, n_kv * group, d, seed=3, dtype=dtype)
    got = tq.attend_paged(pages, lens, n, q.cuda(), kc, vc).double().cpu().numpy()
    small = np.stack([np.arange(held), np.arange(held) + held])  # the same tokens in a small cache
    kc2, vc2 = (np.pad(x.double().numpy().reshape(2, n, n_kv, d), ((0, 0), (0, held * block - n), (0, 0), (0, 0)))
                .reshape(2 * held, block, n_kv, d).transpose(0, 2, 1, 3) for x in (k, v))
    q64 = q.double().numpy()
    ref = paged.attend(small, [n, n], q64, kc2, vc2, block)
    assert np.all(np.abs(got - ref) <= attend_tolerance(small, [n, n], q64, kc2, vc2, block, d ** -0.5, dtype, F32))
    s = tq.block_scores(pages, lens, q.cuda(), bd).cpu().double().numpy()
    pad = np.concatenate([k.double().numpy().reshape(2, n, n_kv, d), np.repeat(k.double().numpy().reshape(2, n, n_kv, d)[:, -1:], held * block - n, axis=1)], 1)
    x = pad.reshape(2 * held, block, n_kv, d)
    bounds = np.stack([x.min(1), x.max(1)], axis=2)
    np.testing.assert_allclose(s, paged.block_scores(small, [n, n], q64, bounds, block), rtol=1e-4)


# ------------------------------------------------------------------------------------ together
def serve(tq, steps, graph, stream=None, seed=0):
    """Admit four sequences, then `steps` decode steps: grow, append, score, choose, attend, all on the GPU.  Returns
    what every step attended and the state."""
    n_kv, group, d, block, width, keep = 2, 4, 128, 16, 24, 9
    dev = torch.device("cuda")
    pages = tq.Pages(torch.full((4, width), -1, dtype=torch.int32, device=dev), n_kv, block, 64)
    free = torch.randperm(64, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    head, lens = torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
    kc, vc = (torch.zeros(64, n_kv, block, d, dtype=BF16, device=dev) for _ in (0, 1))
    bd = torch.zeros(64, n_kv, 2, d, dtype=BF16, device=dev)
    new = i32([301, 0, 16, 100])
    k, v = (rows(417, n_kv, d, seed=seed + i, dtype=BF16).cuda() for i in (1, 2))
    _, _, granted, _, off = tq.page_extend(pages, lens, new, free, head, n_rows=417, seq_lens_out=lens, free_head_out=head)
    tq.append_kv(pages, lens, granted, off, k, v, kc, vc, bd)
    ks, vs = (rows(steps, 4, n_kv, d, seed=seed + i, dtype=BF16).cuda() for i in (3, 4))
    qs = rows(steps, 4, n_kv * group, d, seed=seed + 5, dtype=BF16).cuda()
    one, knew, vnew, q = i32([1, 1, 1, 1]), ks[0].clone(), vs[0].clone(), qs[0].clone()
    keep_all = {}

    def step():
        slots, _, granted, _, off = tq.page_extend(pages, lens, one, free, head, n_rows=4, seq_lens_out=lens, free_head_out=head)
        tq.append_kv(pages, lens, granted, off, knew, vnew, kc, vc, bd)
        s = tq.block_scores(pages, lens, q, bd)
        table, held = tq.select_blocks(pages, lens, s, keep, n_first=1, n_last=2)
        sub = pages.selected(table)
        full = tq.attend_paged(pages, lens, width * block, q, kc, vc)
        part = tq.attend_paged(sub, held, keep * block, q.view(4 * n_kv, group, d), kc, vc)
        keep_all["out"] = (slots, s, table, held, full, part)

    if graph:
        g = torch.cuda.CUDAGraph()
        saved = [x.clone() for x in (pages.block_table, lens, head, kc, vc, bd)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(g):
            step()
        for x, y in zip((pages.block_table, lens, head, kc, vc, bd), saved):
            x.copy_(y)
    outs = []
    for i in range(steps):
        knew.copy_(ks[i]), vnew.copy_(vs[i]), q.copy_(qs[i])
        g.replay() if graph else step()
        outs.append([x.clone() for x in keep_all["out"]])
    torch.cuda.synchronize()
    return outs, dict(pages=pages, lens=lens, kc=kc, vc=vc, bd=bd, qs=qs, free=free, group=group, keep=keep, block=block)


def test_serving_steps(tq):
    """Prompts, then 20 decode steps (sequences cross block borders, one starts empty): every step's choice and
    both attentions follow the oracle on the cache as it is; the eager and the captured run give the same bits."""
    outs, s = serve(tq, 20, graph=False)
    assert s["lens"].tolist() == [321, 20, 36, 120]
    kc, vc = s["kc"].double().cpu().numpy(), s["vc"].double().cpu().numpy()
    bd, table = s["bd"].double().cpu().numpy(), s["pages"].block_table.cpu().numpy()
    lens, q64 = s["lens"].cpu().numpy(), s["qs"][-1].double().cpu().numpy()
    _, sc, sel, held, full, part = (x.cpu().numpy() for x in outs[-1])
    ref_bd = np.zeros_like(bd)
    for b, n in enumerate(lens):
        for j in range(-(-n // 16)):
            x = kc[table[b, j], :, :min(16, n - 16 * j)]
            ref_bd[table[b, j], :, 0], ref_bd[table[b, j], :, 1] = x.min(1), x.max(1)
    used = np.unique(table[table >= 0])
    assert np.array_equal(bd[used], ref_bd[used])
    ref_sel, ref_held = paged.select(table, lens, sc.astype(np.float64), 2, 16, 64, s["keep"], 1, 2)
    assert np.array_equal(sel, ref_sel) and np.array_equal(held, ref_held)
    assert np.all(np.abs(full - paged.attend(table, lens, q64, kc, vc, 16)) <=
                  attend_tolerance(table, lens, q64, kc, vc, 16, 128 ** -0.5, BF16, F32))
    k1, v1, q1 = kc.reshape(128, 1, 16, 128), vc.reshape(128, 1, 16, 128), q64.reshape(8, 4, 128)
    assert np.all(np.abs(part - paged.attend(sel, held, q1, k1, v1, 16)) <=
                  attend_tolerance(sel, held, q1, k1, v1, 16, 128 ** -0.5, BF16, F32))
    again, _ = serve(tq, 20, graph=True)
    for x, y in zip(outs, again):
        for u, w in zip(x, y):
            assert torch.equal(u, w)


def test_serving_steps_on_two_streams(tq):
    """Two independent runs queued on two streams at once give what each gives alone."""
    alone = [serve(tq, 6, graph=False, seed=s)[0] for s in (0, 50)]
    streams = [torch.cuda.Stream() for _ in (0, 1)]
    torch.cuda.synchronize()
    both = []
    for s, st in zip((0, 50), streams):
        with torch.cuda.stream(st):
            both.append(serve(tq, 6, graph=False, seed=s)[0])
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        for u, w in zip(x, y):
            assert all(torch.equal(a, b) for a, b in zip(u, w))


class Serving:
    """Three sequences over a cache of their own: grow, append, score, choose, attend (rows cut into pieces, and the
    chosen blocks), every step's results kept."""

    def __init__(self, tq, seed):
        self.tq, self.n_kv, self.group, self.d, self.block, self.steps = tq, 2, 4, 128, 16, 12
        held = [20000 + seed, 700, 3000]
        width = 1300
        table, used = tables(held, width, self.block, seed)
        n_blocks = used + 40
        self.pages = tq.Pages(i32(table), self.n_kv, self.block, n_blocks)
        self.free, self.head, self.lens = i32(np.arange(used, n_blocks)), i32([0]), i32(held)
        self.k, self.v = (rows(n_blocks, self.n_kv, self.block, self.d, seed=seed + i, dtype=BF16).cuda() for i in (1, 2))
        self.bounds = self.k.aminmax(dim=2)
        self.bounds = torch.stack([self.bounds.min, self.bounds.max], dim=2)
        self.new = rows(self.steps, 2, 3, self.n_kv, self.d, seed=seed + 3, dtype=BF16).cuda()
        self.q = rows(self.steps, 3, self.n_kv * self.group, self.d, seed=seed + 4, dtype=BF16).cuda()
        self.one, self.max_len, self.kept = i32([1, 1, 1]), width * self.block, []

    def step(self, i):
        tq, keep = self.tq, 40
        slots, _, granted, _, off = tq.page_extend(self.pages, self.lens, self.one, self.free, self.head, n_rows=3,
                                                   seq_lens_out=self.lens, free_head_out=self.head)
        tq.append_kv(self.pages, self.lens, granted, off, self.new[i, 0], self.new[i, 1], self.k, self.v, self.bounds)
        s = tq.block_scores(self.pages, self.lens, self.q[i], self.bounds)
        table, held = tq.select_blocks(self.pages, self.lens, s, keep)
        full = tq.attend_paged(self.pages, self.lens, self.max_len, self.q[i], self.k, self.v)
        part = tq.attend_paged(self.pages.selected(table), held, keep * self.block, self.q[i].view(3 * self.n_kv, self.group, self.d),
                               self.k, self.v)
        self.kept += [slots, s, table, held, full, part]

    def state(self):
        return self.kept + [self.pages.block_table, self.lens, self.head, self.k, self.v, self.bounds]


@pytest.mark.parametrize("threads", [False, True])
def test_serving_at_once_on_two_streams(tq, threads):
    """Two caches served at once, every step of both queued before either begins, by one thread in turn or by a thread
    each: what each gives alone."""
    import threading
    seeds, alone = (100, 200), []
    for s in seeds:
        alone.append(Serving(tq, s))
        for i in range(alone[-1].steps):
            alone[-1].step(i)
    both, streams = [Serving(tq, s) for s in seeds], [torch.cuda.Stream() for _ in seeds]
    torch.cuda.synchronize()

    def queue(x, st, some):
        with torch.cuda.stream(st):
            for i in some:
                x.step(i)

    for st in streams:
        with torch.cuda.stream(st):
            torch.cuda._sleep(100_000_000)  # some 50 ms: the steps are queued meanwhile
    if threads:
        runs = [threading.Thread(target=queue, args=(x, st, range(x.steps))) for x, st in zip(both, streams)]
        for t in runs:
            t.start()
        for t in runs:
            t.join()
    else:
        for i in range(both[0].steps):
            for x, st in zip(both, streams):
                queue(x, st, [i])
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        assert len(y.kept) == 6 * x.steps
        for k, (u, w) in enumerate(zip(x.state(), y.state())):
            assert torch.equal(u, w), k


def test_calls_on_a_given_stream(tq):
    """stream=: the work runs there, not on the current stream, and what the calls allocate stays theirs."""
    n_kv, group, d, block = 2, 4, 128, 16
    table, n_blocks = tables([700], 44, block, 3)
    pages, lens = tq.Pages(i32(table), n_kv, block, n_blocks), i32([700])
    k, v = (rows(700, n_kv, d, seed=s, dtype=BF16).cuda() for s in (1, 2))
    q = rows(1, n_kv * group, d, seed=3, dtype=BF16).cuda()
    kc, vc = (torch.zeros(n_blocks, n_kv, block, d, dtype=BF16).cuda() for _ in (0, 1))
    bd, off = torch.zeros(n_blocks, n_kv, 2, d, dtype=BF16).cuda(), torch.tensor([0, 700]).cuda()

    def run(stream):
        for x in (kc, vc, bd):
            x.zero_()
        torch.cuda.synchronize()
        tq.append_kv(pages, lens, lens, off, k, v, kc, vc, bd, stream=stream)
        t, n = tq.select_blocks(pages, lens, tq.block_scores(pages, lens, q, bd, stream=stream), 7, stream=stream)
        o = tq.attend_paged(pages.selected(t), n, 7 * block, q.view(n_kv, group, d), kc, vc, stream=stream)
        torch.empty(1 << 22, device="cuda").fill_(math.nan)  # takes what the current stream may reuse
        torch.cuda.synchronize()
        return t, n, o

    for x, y in zip(run(None), run(torch.cuda.Stream())):
        assert torch.equal(x, y)


def test_calls_on_a_given_stream_leave_queued_work_alone(tq):
    """stream= while the current stream still holds queued reads and writes of memory that it has freed: what the calls
    make for themselves is none of it.  Sizes are those of their outputs and workspace."""
    n_kv, group, d, block, batch, keep = 2, 4, 128, 16, 3, 7
    n = [20000, 700, 3000]
    table, n_blocks = tables(n, 1250, block, 3)
    pages, lens, side = tq.Pages(i32(table), n_kv, block, n_blocks), i32(n), torch.cuda.Stream()
    q = rows(batch, n_kv * group, d, seed=3, dtype=BF16).cuda()
    kc, vc = (rows(n_blocks, n_kv, block, d, seed=s, dtype=BF16).cuda() for s in (1, 2))
    bd = rows(n_blocks, n_kv, 2, d, seed=4, dtype=BF16).sort(2).values.cuda()
    scores = tq.block_scores(pages, lens, q, bd)
    free, one, head = i32(range(n_blocks, n_blocks + 9)), i32([1] * batch), i32([0])
    ws = tq.attend_paged_workspace_size(pages, max(n), n_kv * group, d)
    calls = [(lambda st: [tq.block_scores(pages, lens, q, bd, stream=st)], [scores.nbytes]),
             (lambda st: list(tq.select_blocks(pages, lens, scores, keep, stream=st)), [4 * batch * n_kv * keep, 4 * batch * n_kv]),
             (lambda st: [tq.attend_paged(pages, lens, max(n), q, kc, vc, stream=st)], [4 * q.numel(), ws]),
             (lambda st: list(tq.page_extend(pages, lens, one, free, head, n_rows=batch, stream=st)),
              [8 * batch * n_kv, 4 * batch, 4 * batch, 4, 8 * (batch + 1)])]
    for call, sizes in calls:
        want = [x.clone() for x in call(None)]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        copies = [torch.empty(size, dtype=torch.uint8, device="cuda") for size in sizes]
        freed = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for size in sizes]
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)  # some 0.1 s
        for c, f in zip(copies, freed):
            c.copy_(f)
            f.fill_(255)
        del freed, f
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(c.eq(7).all() for c in copies)


def test_calls_on_a_forked_stream_of_a_capture(tq):
    """stream= names a stream that joined a capture, not the capturing one: what the calls make for themselves stays
    the graph's, whatever is allocated between replays."""
    n_kv, group, d, block = 2, 4, 128, 16
    n = [20000, 700]
    table, n_blocks = tables(n, 1250, block, 3)
    pages, lens, side = tq.Pages(i32(table), n_kv, block, n_blocks), i32(n), torch.cuda.Stream()
    q = rows(2, n_kv * group, d, seed=3, dtype=BF16).cuda()
    kc, vc = (rows(n_blocks, n_kv, block, d, seed=s, dtype=BF16).cuda() for s in (1, 2))
    bd = rows(n_blocks, n_kv, 2, d, seed=4, dtype=BF16).sort(2).values.cuda()

    def run(st):
        s = tq.block_scores(pages, lens, q, bd, stream=st)
        t, held = tq.select_blocks(pages, lens, s, 30, stream=st)
        part = tq.attend_paged(pages.selected(t), held, 30 * block, q.view(2 * n_kv, group, d), kc, vc, stream=st)
        return [s, t, held, part, tq.attend_paged(pages, lens, max(n), q, kc, vc, stream=st)]

    want = [x.clone() for x in run(None)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = run(side)
        torch.cuda.current_stream().wait_stream(side)
    for i in range(3):
        other = [torch.full((1 << (8 + k),), 255, dtype=torch.uint8, device="cuda") for k in range(18)]
        for x in got:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and all(x.eq(255).all() for x in other)


def test_profiled_calls(tq):
    """Per-kernel timing counts the paged-cache kernels under their names, and the results stay the same."""
    plain = serve(tq, 2, graph=False)[0]
    tq.profile_reset()
    tq.profile_enable(True)
    try:
        timed = serve(tq, 2, graph=False)[0]
    finally:
        tq.profile_enable(False)
    n = {k: v[0] for k, v in tq.profile_read().items()}
    tq.profile_reset()
    assert (n["page_extend"], n["append_kv"], n["block_scores"], n["select_blocks"], n["attend_paged"]) == (3, 3, 2, 2, 4)
    for x, y in zip(plain, timed):
        assert all(torch.equal(a, b) for a, b in zip(x, y))


@pytest.mark.parametrize("vlayout", [0, 1])
def test_compressed_cache_through_pages(tq, vlayout):
    """page_extend's slots encode the compressed cache, its new_slots serve tq_decode_step, and the chosen blocks
    are attended with tq_attend_decode as one-head sequences (general and tensor-core attention)."""
    n_kv, group, d, block, width, keep = 2, 4, 128, 16, 40, 6
    new = [301, 16, 600, 33]
    kq, vq = Quantizer(d, 2, d, seed=60), Quantizer(d, 3, 0, seed=61, layout=vlayout)
    cap = 90
    kp, vp = tq.Packed.allocate(kq.ctx, cap * n_kv * block), tq.Packed.allocate(vq.ctx, cap * n_kv * block)
    pages = tq.Pages(torch.full((4, width), -1, dtype=torch.int32, device="cuda"), n_kv, block, cap)
    free = torch.randperm(cap, generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    head, lens = i32([0]), i32([0, 0, 0, 0])
    n = sum(new) + 7  # a padded batch: the rows behind the last sequence are not stored
    k, v = (rows(n, n_kv, d, seed=s, dtype=BF16).cuda() for s in (62, 63))
    slots, lens, granted, head, off = tq.page_extend(pages, lens, i32(new), free, head, n_rows=n)
    tq.encode_kv(kq.ctx, k.view(-1, d), kp, slots=slots)
    tq.encode_kv(vq.ctx, v.view(-1, d), vp, slots=slots)
    bd = torch.empty(cap, n_kv, 2, d, dtype=BF16, device="cuda")
    tq.append_kv(pages, lens, granted, off, k, bounds=bd)
    # one decode step of the compressed path with the slots of the grown sequences
    k1, v1 = (rows(4, n_kv, d, seed=s, dtype=BF16).cuda() for s in (64, 65))
    q = rows(4, n_kv * group, d, seed=66, dtype=BF16).cuda()
    slots, lens, granted, head, off = tq.page_extend(pages, lens, i32([1] * 4), free, head, n_rows=4)
    desc = tq.make_attn_desc(kq.ctx, vq.ctx, q.shape, kp, vp, lens, width * block, block_table=pages.block_table,
                             block_size=block, n_kv_heads=n_kv)
    out = tq.decode_step(kq.ctx, vq.ctx, q, k1.view(-1, d), v1.view(-1, d), slots, desc)
    tq.append_kv(pages, lens, granted, off, k1, bounds=bd)
    s = tq.block_scores(pages, lens, q, bd)
    table, held = tq.select_blocks(pages, lens, s, keep, n_first=1, n_last=2)
    part = tq.attend_decode(kq.ctx, vq.ctx, q.view(4 * n_kv, group, d), kp, vp, held, keep * block, n_kv_heads=1,
                            block_table=table, block_size=block)
    torch.cuda.synchronize()
    assert lens.tolist() == [x + 1 for x in new] and tq.device_status() == 0
    tab, sel = pages.block_table.cpu().numpy(), table.cpu().numpy()
    got, gotp = out.cpu().numpy(), part.cpu().numpy()
    slots_of = lambda b, h, m: oattn.token_slots(b, h, m, n_kv, block_table=tab)
    pairs = [(b, h) for b in range(4) for h in (0, 5)]
    ref = oracle_heads(kq, vq, kp, vp, q.cpu(), pairs, lens.tolist(), slots_of, group)
    for pr in pairs:
        assert_attention_close(got[pr][None], ref[pr][None])
    pairs = [(r, g) for r in range(4 * n_kv) for g in (0, 3)]
    slots_of = lambda b, h, m: oattn.token_slots(b, h, m, 1, block_table=sel)
    ref = oracle_heads(kq, vq, kp, vp, q.cpu().view(4 * n_kv, group, d), pairs, held.tolist(), slots_of, group)
    for pr in pairs:
        assert_attention_close(gotp[pr][None], ref[pr][None])
