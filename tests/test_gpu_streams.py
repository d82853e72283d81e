"""Calls on a given stream while the current one still holds queued work on memory that it has freed: the outputs
and workspaces that a call makes for itself are none of that memory."""
import pytest
import torch

import synth
from parity import Quantizer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    from kv_cache_vector_06_b200 import tq as _tq
    return _tq


def while_work_is_queued(call, sizes):
    """What call() returns on a side stream, with a copy out of and a write to freed memory of `sizes` bytes each
    queued on the current one; fails where the copies are not what was there."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    copies = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    freed = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # some 0.1 s
    for c, f in zip(copies, freed):
        c.copy_(f)
        f.fill_(255)
    del freed, f
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(c.eq(7).all() for c in copies)
    return got


def cache(tq, d, n, layout):
    kq, vq = Quantizer(d, 2, d, seed=5), Quantizer(d, 3, 0, seed=6, layout=layout)
    x = synth.channel_scaled(1, 1, n, d, seed=7)[0, 0].cuda()
    kp, vp = tq.Packed.allocate(kq.ctx, n), tq.Packed.allocate(vq.ctx, n)
    tq.encode_kv(kq.ctx, x, kp)
    tq.encode_kv(vq.ctx, x, vp)
    return kq, vq, kp, vp, x


def test_encode_on_a_given_stream(tq):
    kq, _, kp, _, x = cache(tq, 128, 40000, 0)
    again = tq.Packed.allocate(kq.ctx, 40000)
    while_work_is_queued(lambda st: tq.encode_kv(kq.ctx, x, again, stream=st), [max(1, tq.encode_workspace_size(kq.ctx, 40000))])
    for name in ("codes", "signs", "norm", "rnorm"):
        assert torch.equal(getattr(again, name), getattr(kp, name)), name


def test_scores_and_search_on_a_given_stream(tq):
    n, nq, k = 40000, 24, 10
    kq, _, kp, _, _ = cache(tq, 128, n, 0)
    q = synth.unit_rows(nq, 128, seed=8).cuda()
    want = tq.scores(kq.ctx, q, kp)
    got = while_work_is_queued(lambda st: tq.scores(kq.ctx, q, kp, stream=st),
                               [want.nbytes, max(1, tq.scores_workspace_size(kq.ctx, nq))])
    assert torch.equal(got, want)
    want = tq.search_topk(kq.ctx, q, kp, k)
    got = while_work_is_queued(lambda st: tq.search_topk(kq.ctx, q, kp, k, stream=st),
                               [4 * nq * k, 8 * nq * k, max(1, tq.search_workspace_size(kq.ctx, nq, n, k))])
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("layout", [0, 1])
def test_decode_on_a_given_stream(tq, layout):
    """General and tensor-core attention, and the fused step (whose appended rows are the same both times)."""
    n, group, d = 30000, 4, 128
    kq, vq, kp, vp, x = cache(tq, d, n, layout)
    q = synth.decode_queries(1, group, d, seed=9).cuda()
    desc = tq.make_attn_desc(kq.ctx, vq.ctx, q.shape, kp, vp, torch.tensor([n], dtype=torch.int32).cuda(), n, n_kv_heads=1)
    out = 4 * q.numel()
    want = tq.attend_decode(kq.ctx, vq.ctx, q, kp, vp, None, n, 1, desc=desc)
    got = while_work_is_queued(lambda st: tq.attend_decode(kq.ctx, vq.ctx, q, kp, vp, None, n, 1, desc=desc, stream=st),
                               [out, max(1, tq.attend_workspace_size(kq.ctx, vq.ctx, desc))])
    assert torch.equal(got, want)
    slot, row = torch.tensor([n - 1]).cuda(), x[5:6].contiguous()
    want = tq.decode_step(kq.ctx, vq.ctx, q, row, row, slot, desc)
    got = while_work_is_queued(lambda st: tq.decode_step(kq.ctx, vq.ctx, q, row, row, slot, desc, stream=st),
                               [out, max(1, tq.decode_step_workspace_size(kq.ctx, vq.ctx, desc, 1))])
    assert torch.equal(got, want)
