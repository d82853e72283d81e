"""Argument checks of the paged-cache calls that need no GPU: every refusal comes from the host, before
any CUDA call, with a message.  Pointers are host addresses that nothing reads."""
import ctypes

import pytest

EINVAL, EUNSUPPORTED, OK = 1, 2, 0
P = 1 << 20  # an aligned address; refused calls never use it


@pytest.fixture(scope="module")
def lib():
    from kv_cache_vector_06_b200.build import build
    build()
    from kv_cache_vector_06_b200 import tq
    return tq


def pages(lib, **over):
    f = dict(device=0, batch=3, n_kv_heads=2, block_size=16, max_blocks=8, n_blocks=100, block_table=P) | over
    return ctypes.byref(lib.PagesC(*[f[n] for n, _ in lib.PagesC._fields_]))


def extend(lib, pg, **over):
    a = dict(seq_lens=P, new_lens=2 * P, free=3 * P, n_free=10, head=P, lens_out=4 * P, granted=5 * P, head_out=P, offsets=P,
             slots=P, n_slots=6) | over
    return lib.LIB.tq_page_extend(pg, *a.values(), None)


def append(lib, pg, **over):
    a = dict(seq_lens=P, granted=P, offsets=P, k=P, v=P, dtype=1, d=64, n_rows=3, ld=128, kc=P, vc=P, bounds=P) | over
    return lib.LIB.tq_append_kv(pg, *a.values(), None)


def scores(lib, pg, **over):
    a = dict(seq_lens=P, q=P, dtype=1, hq=8, d=64, bounds=P, out=P) | over
    return lib.LIB.tq_block_scores(pg, *a.values(), None)


def select(lib, pg, **over):
    a = dict(seq_lens=P, scores=P, keep=4, first=1, last=2, table=P, lens=P) | over
    return lib.LIB.tq_select_blocks(pg, *a.values(), None)


def attend(lib, pg, **over):
    a = dict(seq_lens=P, max_len=100, q=P, k=P, v=P, dtype=1, hq=8, d=64, scale=0.0, out=P, out_dtype=0, ws=P,
             ws_bytes=1 << 40) | over
    return lib.LIB.tq_attend_paged(pg, *a.values(), None)


CALLS = [extend, append, scores, select, attend]


@pytest.mark.parametrize("call", CALLS)
def test_pages_are_checked(lib, call):
    assert call(lib, None) == EINVAL and b"pages is NULL" in lib.LIB.tq_last_error()
    for bad in (dict(batch=-1), dict(n_kv_heads=0), dict(block_size=0), dict(max_blocks=0), dict(n_blocks=-1),
                dict(block_table=None), dict(block_table=P + 2)):
        assert call(lib, pages(lib, **bad)) == EINVAL, bad
        assert b"pages" in lib.LIB.tq_last_error()
    for big in (dict(batch=1 << 30, n_kv_heads=2), dict(n_blocks=1 << 30), dict(n_kv_heads=65536, n_blocks=10), dict(max_blocks=1 << 20, block_size=1 << 11)):
        assert call(lib, pages(lib, **big)) == EUNSUPPORTED, big


def test_empty_batch_is_no_work(lib):
    empty = pages(lib, batch=0, block_table=None)
    for call in (append, scores, select, attend):
        assert call(lib, empty) == OK


@pytest.mark.parametrize("over", [dict(seq_lens=None), dict(new_lens=None), dict(free=None), dict(head=None),
                                  dict(lens_out=None), dict(granted=None), dict(head_out=None), dict(offsets=None),
                                  dict(slots=None), dict(n_free=-1), dict(n_slots=-2), dict(n_slots=5), dict(seq_lens=P + 1),
                                  dict(offsets=P + 4), dict(slots=P + 4), dict(head=P + 2),
                                  dict(lens_out=2 * P), dict(granted=P), dict(granted=4 * P), dict(lens_out=3 * P),
                                  dict(granted=3 * P)])
def test_extend_refusals(lib, over):
    assert extend(lib, pages(lib), **over) == EINVAL and lib.LIB.tq_last_error()


@pytest.mark.parametrize("over,st", [(dict(seq_lens=None), EINVAL), (dict(granted=None), EINVAL), (dict(offsets=None), EINVAL),
                                     (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(kc=None), EINVAL),
                                     (dict(vc=None), EINVAL), (dict(kc=None, vc=None, bounds=None), EINVAL),
                                     (dict(dtype=7), EINVAL), (dict(d=60), EUNSUPPORTED), (dict(d=0), EUNSUPPORTED),
                                     (dict(d=264), EUNSUPPORTED), (dict(ld=127), EINVAL), (dict(ld=132), EINVAL),
                                     (dict(n_rows=-1), EINVAL), (dict(k=P + 8), EINVAL), (dict(bounds=P + 8), EINVAL),
                                     (dict(kc=P + 8), EINVAL)])
def test_append_refusals(lib, over, st):
    assert append(lib, pages(lib), **over) == st and lib.LIB.tq_last_error()


@pytest.mark.parametrize("over,st", [(dict(seq_lens=None), EINVAL), (dict(q=None), EINVAL), (dict(bounds=None), EINVAL),
                                     (dict(out=None), EINVAL), (dict(dtype=2), EINVAL), (dict(hq=7), EINVAL),
                                     (dict(hq=0), EINVAL), (dict(hq=34), EUNSUPPORTED), (dict(d=12), EUNSUPPORTED),
                                     (dict(q=P + 4), EINVAL), (dict(out=P + 4), EINVAL), (dict(bounds=P + 2), EINVAL)])
def test_score_refusals(lib, over, st):
    assert scores(lib, pages(lib), **over) == st and lib.LIB.tq_last_error()


@pytest.mark.parametrize("over,st", [(dict(seq_lens=None), EINVAL), (dict(scores=None), EINVAL), (dict(table=None), EINVAL),
                                     (dict(lens=None), EINVAL), (dict(keep=0), EINVAL), (dict(first=-1), EINVAL),
                                     (dict(last=0), EINVAL), (dict(first=3), EINVAL),
                                     (dict(first=(1 << 31) - 1, last=(1 << 31) - 1), EINVAL),
                                     (dict(keep=1 << 28), EUNSUPPORTED), (dict(scores=P + 4), EINVAL), (dict(lens=P + 2), EINVAL)])
def test_select_refusals(lib, over, st):
    assert select(lib, pages(lib), **over) == st and lib.LIB.tq_last_error()


@pytest.mark.parametrize("over,st", [(dict(seq_lens=None), EINVAL), (dict(q=None), EINVAL), (dict(k=None), EINVAL),
                                     (dict(v=None), EINVAL), (dict(out=None), EINVAL), (dict(max_len=-1), EINVAL),
                                     (dict(max_len=129), EINVAL), (dict(dtype=3), EINVAL), (dict(dtype=0, out_dtype=1), EINVAL),
                                     (dict(out_dtype=9), EINVAL), (dict(hq=9), EINVAL), (dict(hq=64), EUNSUPPORTED),
                                     (dict(d=4), EUNSUPPORTED), (dict(d=512), EUNSUPPORTED), (dict(q=P + 8), EINVAL),
                                     (dict(out=P + 8), EINVAL), (dict(k=P + 2), EINVAL)])
def test_attend_refusals(lib, over, st):
    assert attend(lib, pages(lib), **over) == st and lib.LIB.tq_last_error()


def test_attend_workspace(lib):
    n = ctypes.c_size_t()
    pg = pages(lib)
    assert lib.LIB.tq_attend_paged_workspace_size(pg, 100, 8, 64, ctypes.byref(n)) == OK
    assert lib.LIB.tq_attend_paged_workspace_size(pg, 100, 8, 64, None) == EINVAL
    assert lib.LIB.tq_attend_paged_workspace_size(pg, 129, 8, 64, ctypes.byref(n)) == EINVAL


def test_binding_refuses_host_tensors(lib):
    import torch
    with pytest.raises(ValueError):
        lib.Pages(torch.zeros(2, 3, dtype=torch.int32), 1, 16, 4)
    with pytest.raises(ValueError):
        lib.Pages(torch.zeros(3, dtype=torch.int32), 1, 16, 4)


def test_own_tensors_come_from_the_given_stream(lib, monkeypatch):
    """A tensor that a call makes for itself belongs to the stream that it works on, and the caller's stream keeps it
    from reuse.  Streams and tensors are stand-ins: what matters is which stream is current at the allocation."""
    import contextlib
    now, made = ["caller"], []

    class Made:
        def __init__(self):
            self.of, self.kept_by = now[0], []
            made.append(self)

        def record_stream(self, s):
            self.kept_by.append(s)

    @contextlib.contextmanager
    def switch(s):
        before, now[0] = now[0], s
        yield
        now[0] = before

    monkeypatch.setattr(lib.torch, "empty", lambda *a, **k: Made())
    monkeypatch.setattr(lib.torch.cuda, "current_stream", lambda device=None: now[0])
    monkeypatch.setattr(lib.torch.cuda, "stream", switch)
    for given in (None, "caller", "other"):
        lib._new((2, 3), lib.torch.int32, "cuda:0", given)
    assert [(t.of, t.kept_by) for t in made] == [("caller", []), ("caller", []), ("other", ["caller"])] and now == ["caller"]


def test_no_call_allocates_for_itself_but_on_its_stream(lib):
    """Every call that makes outputs or workspaces makes them where its stream is heeded."""
    import ast
    import inspect
    for f in ast.walk(ast.parse(inspect.getsource(lib))):
        if isinstance(f, ast.FunctionDef) and f.name != "_new" and "stream" in [a.arg for a in f.args.args]:
            made = [n.func.attr for n in ast.walk(f) if isinstance(n, ast.Call) and isinstance(n.func, ast.Attribute)
                    and isinstance(n.func.value, ast.Name) and n.func.value.id == "torch"]
            assert not {"empty", "zeros", "full", "empty_like"} & set(made), f.name
    for name in ("encode_kv", "scores", "attend_decode", "decode_step", "search_topk"):
        assert "_workspace(" in inspect.getsource(getattr(lib, name)) and ", ws, stream)" in inspect.getsource(getattr(lib, name)), name


def test_workspace_lives_until_the_launches_are_queued(lib, monkeypatch):
    """The address that a call passes on holds the tensor behind it: the library works without the interpreter's
    lock, and a thread that allocates meanwhile must not be given the same memory."""
    import gc
    import weakref
    import torch
    seen = []

    def made(*a):
        t = torch.empty(64, dtype=torch.uint8)
        seen.append(weakref.ref(t))
        return t

    monkeypatch.setattr(lib, "_new", made)
    monkeypatch.setattr(lib, "_dev", lambda t, *a, **k: lib.c_void_p(t.data_ptr()))
    w, n = lib._workspace(64, 0, None, None)
    gc.collect()
    assert n == 64 and seen[0]() is not None and w.value == seen[0]().data_ptr()
    del w
    gc.collect()
    assert seen[0]() is None


def host_pages(lib, n_kv, block, n_blocks, batch=2, width=4):
    """Pages of a table in host memory: what the binding checks before it calls the library."""
    import torch
    p = object.__new__(lib.Pages)
    p.device, p.batch, p.max_blocks, p.n_kv_heads, p.block_size, p.n_blocks = -1, batch, width, n_kv, block, n_blocks
    p._dims = (n_blocks, n_kv)
    p.rows, p.block_table = batch * n_kv, torch.zeros(batch, width, dtype=torch.int32)
    p._c = lib.PagesC(-1, batch, n_kv, block, width, n_blocks, p.block_table.data_ptr())
    p.ref = ctypes.byref(p._c)
    return p


@pytest.mark.parametrize("n_kv,block,shape,fits", [
    (2, 16, (5, 2, 16, 8), True),
    (2, 16, (10, 16, 8), True), (2, 16, (5, 32, 8), True), (2, 16, (160, 8), True),  # neighbours joined
    (1, 16, (5, 2, 16, 8), True),    # ten blocks of one head: the heads counted among the blocks
    (2, 16, (1, 160, 8), True), (1, 16, (5, 1, 2, 16, 8), True), (1, 16, (10, 16, 1, 8), True), (2, 1, (5, 1, 2, 8), True),
    (2, 16, (5, 16, 2, 8), False),   # token before head
    (1, 16, (5, 16, 2, 8), False),
    (2, 16, (2, 5, 16, 8), False),   # head before block
    (2, 16, (5, 2, 8, 16), False), (2, 16, (5, 2, 16, 4), False), (2, 16, (6, 2, 16, 8), False),
    (2, 16, (80, 2, 8), False), (2, 16, (1280,), False), (2, 16, (), False)])
def test_caches_of_another_order_are_refused(lib, n_kv, block, shape, fits):
    """An array of as many entries in another order of blocks, heads and tokens is not read as this one."""
    import torch
    p = host_pages(lib, n_kv, block, 10 // n_kv)
    t = torch.zeros(shape)
    if fits:
        assert p._cache(t, "k_cache", block, 8, torch.float32) == t.data_ptr()
    else:
        with pytest.raises(ValueError, match="k_cache must"):
            p._cache(t, "k_cache", block, 8, torch.float32)


def test_caches_of_selected_pages(lib, monkeypatch):
    """Pages over chosen blocks take the caches of the pages that they were made from."""
    import torch
    monkeypatch.setattr(lib.Pages, "__init__", lambda self, table, h, bs, n: self.__dict__.update(
        host_pages(lib, h, bs, n, *table.shape).__dict__))
    p = host_pages(lib, 2, 16, 5).selected(torch.zeros(4, 3, dtype=torch.int32))
    assert (p.n_kv_heads, p.n_blocks, p.rows) == (1, 10, 4)
    for shape in ((5, 2, 16, 8), (5, 32, 8), (10, 16, 8), (160, 8)):
        p._cache(torch.zeros(shape), "k_cache", 16, 8, torch.float32)
    with pytest.raises(ValueError):
        p._cache(torch.zeros(5, 16, 2, 8), "k_cache", 16, 8, torch.float32)


def test_empty_caches_pass(lib):
    import torch
    host_pages(lib, 2, 16, 0)._cache(torch.zeros(0, 2, 16, 8), "k_cache", 16, 8, torch.float32)


class FakeLibrary:
    """Takes the arguments of tq_append_kv and does nothing."""

    def tq_append_kv(self, *a):
        self.args = a
        return OK


class FakeStream:
    cuda_stream = 0


@pytest.mark.parametrize("n,n_kv,split,ok", [(1, 2, "k", True), (1, 2, "v", True), (1, 1, "k", True), (0, 2, "k", True),
                                             (3, 1, "both", True), (3, 2, "both", True), (3, 2, "k", False), (3, 2, "v", False),
                                             (1, 2, "heads", False), (3, 2, "heads", False), (3, 1, "heads", True)])
def test_append_rows_of_any_stride_that_matters(lib, monkeypatch, n, n_kv, split, ok):
    """k_new, v_new or both halves of one projection's rows: with one row (or head) their strides along it may
    differ; with more, they must agree, and heads must lie side by side."""
    import torch
    monkeypatch.setattr(lib, "LIB", FakeLibrary())
    p, d = host_pages(lib, n_kv, 16, 5), 8
    joint = torch.zeros(n, 2, n_kv, d)
    k, v = joint[:, 0], joint[:, 1]
    if split == "heads":  # heads lie apart
        k = v = torch.zeros(n_kv, n, d).transpose(0, 1) if n > 1 else torch.zeros(n, n_kv, 2, d)[:, :, 0]
    k, v = k if split != "v" else torch.zeros(k.shape), v if split != "k" else torch.zeros(v.shape)
    ints = [torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)]
    kc = torch.zeros(5, n_kv, 16, d)
    if not ok:
        with pytest.raises(ValueError):
            lib.append_kv(p, *ints, k, v, kc, kc.clone(), stream=FakeStream)
        return
    lib.append_kv(p, *ints, k, v, kc, kc.clone(), stream=FakeStream)
    a = lib.LIB.args
    assert a[4] == k.data_ptr() and a[5] == v.data_ptr() and a[7] == d and a[8] == n
    assert a[9] == (k.stride(0) if n > 1 else n_kv * d) and a[9] >= n_kv * d


def test_append_refuses_other_heads_and_types(lib, monkeypatch):
    import torch
    monkeypatch.setattr(lib, "LIB", FakeLibrary())
    p = host_pages(lib, 2, 16, 5)
    ints = [torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)]
    k, kc = torch.zeros(3, 2, 8), torch.zeros(5, 2, 16, 8)
    for kn, vn in ((k, k.bfloat16()), (k, k[:2]), (torch.zeros(3, 4, 8), torch.zeros(3, 4, 8)), (k[0], k[0])):
        with pytest.raises(ValueError):
            lib.append_kv(p, *ints, kn, vn, kc, kc.clone(), stream=FakeStream)
