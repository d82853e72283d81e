"""Python binding of libtq (ctypes): argument marshalling only.

Every step of the path runs in the CUDA library; this module only turns torch tensors into
device pointers, checks that they live on the right device with the right dtype and layout,
allocates workspaces with torch when the caller gives none, and raises on a non-zero status.
There is no CPU fallback: if libtq.so is missing or cannot be loaded, importing this module
raises.

`stream` names the stream that a call's work is queued on (default: the current one).  Ordering the arguments'
other uses with it is the caller's; outputs and workspaces that a call makes for itself belong to that stream.
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import POINTER, c_char_p, c_double, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtq.so")

TQ_F32, TQ_BF16 = 0, 1
STATUS = {0: "TQ_OK", 1: "TQ_EINVAL", 2: "TQ_EUNSUPPORTED", 3: "TQ_ENOMEM", 4: "TQ_ECUDA", 5: "TQ_ETIMEOUT"}


class TqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class Spec(ctypes.Structure):
    _fields_ = [("d", c_int32), ("mse_bits", c_int32), ("qjl_m", c_int32), ("layout", c_int32),
                ("norm_bits", c_int32)]


LAYOUT_ROWS, LAYOUT_BLOCK16 = 0, 1


class PackedC(ctypes.Structure):
    _fields_ = [("codes", c_void_p), ("signs", c_void_p), ("norm", c_void_p), ("rnorm", c_void_p),
                ("capacity", c_int64)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32), ("scale", c_float),
                ("seq_lens", c_void_p), ("block_table", c_void_p), ("max_blocks", c_int32),
                ("block_size", c_int32), ("ctx_stride", c_int64), ("max_seq_len", c_int32),
                ("k", PackedC), ("v", PackedC), ("sparse_v", c_float)]


class PagesC(ctypes.Structure):
    _fields_ = [("device", c_int32), ("batch", c_int32), ("n_kv_heads", c_int32), ("block_size", c_int32),
                ("max_blocks", c_int32), ("n_blocks", c_int64), ("block_table", c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m kv_cache_vector_06_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    st = c_int
    sig = {
        "tq_make_codebook": (st, [c_int32, c_int32, POINTER(c_double), POINTER(c_double), POINTER(c_double)]),
        "tq_ctx_create": (st, [POINTER(Spec), c_void_p, c_void_p, c_int32, POINTER(c_void_p)]),
        "tq_ctx_create_srht": (st, [POINTER(Spec), c_void_p, c_void_p, c_int32, POINTER(c_void_p)]),
        "tq_ctx_create_polar": (st, [POINTER(Spec), c_void_p, c_void_p, c_int32, POINTER(c_void_p)]),
        "tq_polar_codebook": (st, [c_int32, c_int32, POINTER(c_double), POINTER(c_double)]),
        "tq_ctx_destroy": (st, [c_void_p]),
        "tq_ctx_layout": (st, [c_void_p, POINTER(c_int64), POINTER(c_int64)]),
        "tq_encode_workspace_size": (st, [c_void_p, c_int64, POINTER(c_size_t)]),
        "tq_encode_kv": (st, [c_void_p, c_void_p, c_int, c_int64, c_int64, c_void_p, PackedC, c_void_p,
                              c_size_t, c_void_p]),
        "tq_scores_workspace_size": (st, [c_void_p, c_int32, POINTER(c_size_t)]),
        "tq_scores": (st, [c_void_p, c_void_p, c_int, c_int32, PackedC, c_int64, c_void_p, c_void_p,
                           c_size_t, c_void_p]),
        "tq_attend_workspace_size": (st, [c_void_p, c_void_p, POINTER(AttnDesc), POINTER(c_size_t)]),
        "tq_attend_decode": (st, [c_void_p, c_void_p, POINTER(AttnDesc), c_void_p, c_int, c_void_p,
                                  c_void_p, c_size_t, c_void_p]),
        "tq_attend_decode_noalloc": (st, [c_void_p, c_void_p, POINTER(AttnDesc), c_void_p, c_int, c_void_p,
                                          c_void_p]),
        "tq_decode_step_workspace_size": (st, [c_void_p, c_void_p, POINTER(AttnDesc), c_int64, POINTER(c_size_t)]),
        "tq_decode_step": (st, [c_void_p, c_void_p, POINTER(AttnDesc), c_void_p, c_void_p, c_int, c_int64, c_void_p,
                                c_void_p, c_int, c_void_p, c_void_p, c_size_t, c_void_p]),
        "tq_device_status": (st, [c_int32, POINTER(c_int32), c_int32]),
        "tq_debug_wait_probe": (st, [c_int32, c_int32]),
        "tq_search_workspace_size": (st, [c_void_p, c_int32, c_int64, c_int32, POINTER(c_size_t)]),
        "tq_search_topk": (st, [c_void_p, c_void_p, c_int, c_int32, PackedC, c_int64, c_int32, c_void_p,
                                c_void_p, c_void_p, c_size_t, c_void_p]),
        "tq_page_extend": (st, [POINTER(PagesC), c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p, c_int64, c_void_p]),
        "tq_append_kv": (st, [POINTER(PagesC), c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int32, c_int64,
                              c_int64, c_void_p, c_void_p, c_void_p, c_void_p]),
        "tq_block_scores": (st, [POINTER(PagesC), c_void_p, c_void_p, c_int, c_int32, c_int32, c_void_p, c_void_p,
                                 c_void_p]),
        "tq_select_blocks": (st, [POINTER(PagesC), c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p,
                                  c_void_p]),
        "tq_attend_paged_workspace_size": (st, [POINTER(PagesC), c_int32, c_int32, c_int32, POINTER(c_size_t)]),
        "tq_attend_paged": (st, [POINTER(PagesC), c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_int, c_int32, c_int32,
                                 c_float, c_void_p, c_int, c_void_p, c_size_t, c_void_p]),
        "tq_profile_enable": (st, [c_int32]),
        "tq_profile_reset": (st, []),
        "tq_profile_read": (st, [c_int32, ctypes.c_char_p, c_int32, POINTER(c_int64), POINTER(c_double)]),
        "tq_last_error": (c_char_p, []),
        "tq_version": (c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def _check(status: int):
    if status != 0:
        raise TqError(status, LIB.tq_last_error().decode())


def version() -> str:
    return LIB.tq_version().decode()


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TQ_F32
    if t.dtype == torch.bfloat16:
        return TQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _dev(t: torch.Tensor, device: int, name: str, dtype=None, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.device.index != device:
        raise ValueError(f"{name} must be a CUDA tensor on device {device} (got {t.device})")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return c_void_p(t.data_ptr())


def make_polar_codebook(level: int, bits: int):
    """PolarQuant angle codebook of one level, computed by the library on the host (fp64)."""
    L = 1 << bits
    c = (c_double * L)()
    t = (c_double * max(L - 1, 1))()
    _check(LIB.tq_polar_codebook(level, bits, c, t))
    return [c[i] for i in range(L)], [t[i] for i in range(L - 1)]


def make_codebook(d: int, bits: int):
    """Lloyd-Max codebook computed by the library on the host (fp64)."""
    L = 1 << bits
    c = (c_double * L)()
    t = (c_double * max(L - 1, 1))()
    mse = c_double()
    _check(LIB.tq_make_codebook(d, bits, c, t, ctypes.byref(mse)))
    return [c[i] for i in range(L)], [t[i] for i in range(L - 1)], mse.value


class Context:
    """Quantizer constants for one tensor role, resident on one device."""

    def __init__(self, d: int, mse_bits: int, qjl_m: int, rot_signs, qjl_matrix=None, device: int = 0,
                 layout: int = LAYOUT_ROWS, qjl_signs=None, polar: bool = False, norm_bits: int = 32):
        """qjl_matrix: the dense JL matrix [qjl_m, d] (tq_ctx_create); or qjl_signs: the sign
        vector D2 [d] of the structured matrix S = P H D2 (tq_ctx_create_srht).  polar: the
        PolarQuant first stage (tq_ctx_create_polar).  norm_bits: 32 or 16, the storage of the
        norms (tq_spec.norm_bits)."""
        rs = torch.as_tensor(rot_signs).to(torch.int8).contiguous().cpu()
        if rs.numel() != d:
            raise ValueError("rot_signs must have d entries")
        self.d, self.mse_bits, self.qjl_m, self.device, self.layout = d, mse_bits, qjl_m, device, layout
        self.srht = qjl_signs is not None
        self.norm_bits = norm_bits
        self.norm_dtype = torch.float16 if norm_bits == 16 else torch.float32
        spec = Spec(d, mse_bits, qjl_m, layout, norm_bits)
        h = c_void_p()
        if self.srht:
            d2 = torch.as_tensor(qjl_signs).to(torch.int8).contiguous().cpu()
            if d2.numel() != d:
                raise ValueError("qjl_signs must have d entries")
            _check(LIB.tq_ctx_create_srht(ctypes.byref(spec), c_void_p(rs.data_ptr()), c_void_p(d2.data_ptr()),
                                          device, ctypes.byref(h)))
        else:
            if qjl_m > 0:
                S = torch.as_tensor(qjl_matrix).to(torch.float32).contiguous().cpu()
                if tuple(S.shape) != (qjl_m, d):
                    raise ValueError(f"qjl_matrix must be [{qjl_m}, {d}]")
                sptr = c_void_p(S.data_ptr())
            else:
                sptr = c_void_p(None)
            create = LIB.tq_ctx_create_polar if polar else LIB.tq_ctx_create
            _check(create(ctypes.byref(spec), c_void_p(rs.data_ptr()), sptr, device, ctypes.byref(h)))
        self.polar = polar
        self._h = h
        cb, sb = c_int64(), c_int64()
        _check(LIB.tq_ctx_layout(h, ctypes.byref(cb), ctypes.byref(sb)))
        self.code_bytes, self.sign_bytes = cb.value, sb.value

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("context is closed")
        return self._h

    def close(self):
        if getattr(self, "_h", None) is not None:
            LIB.tq_ctx_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Packed:
    """Caller-owned packed arrays (torch tensors on the context's device), indexed by slot."""

    def __init__(self, codes, norm, signs=None, rnorm=None):
        self.codes, self.norm, self.signs, self.rnorm = codes, norm, signs, rnorm

    @staticmethod
    def allocate(ctx: Context, capacity: int) -> "Packed":
        dev = torch.device("cuda", ctx.device)
        codes = torch.zeros(capacity, ctx.code_bytes, dtype=torch.uint8, device=dev)
        norm = torch.zeros(capacity, dtype=ctx.norm_dtype, device=dev)
        signs = rnorm = None
        if ctx.qjl_m > 0:
            signs = torch.zeros(capacity, ctx.sign_bytes, dtype=torch.uint8, device=dev)
            rnorm = torch.zeros(capacity, dtype=ctx.norm_dtype, device=dev)
        return Packed(codes, norm, signs, rnorm)

    @property
    def capacity(self) -> int:
        return self.codes.shape[0]

    def c(self, ctx: Context) -> PackedC:
        if self.codes.dim() != 2 or self.codes.shape[1] != ctx.code_bytes or self.codes.dtype != torch.uint8:
            raise ValueError(f"codes must be uint8 [capacity, {ctx.code_bytes}]")
        p = PackedC(_dev(self.codes, ctx.device, "codes", torch.uint8),
                    c_void_p(None), _dev(self.norm, ctx.device, "norm", ctx.norm_dtype),
                    c_void_p(None), self.codes.shape[0])
        if self.norm.numel() < self.capacity:
            raise ValueError("norm is shorter than codes")
        if ctx.qjl_m > 0 and self.signs is not None:
            if self.signs.shape != (self.capacity, ctx.sign_bytes) or self.signs.dtype != torch.uint8:
                raise ValueError(f"signs must be uint8 [capacity, {ctx.sign_bytes}]")
            if self.rnorm is None or self.rnorm.numel() < self.capacity:
                raise ValueError("rnorm must have capacity entries")
            p.signs = _dev(self.signs, ctx.device, "signs", torch.uint8)
            p.rnorm = _dev(self.rnorm, ctx.device, "rnorm", ctx.norm_dtype)
        return p


def _new(shape, dtype, device, stream):
    """A tensor that a call makes for itself.  On a given stream it comes from that stream's own memory: a block of
    the current stream's may still be in use by what is queued there, which the given stream does not wait for.  The
    current stream, where the caller goes on, keeps it from reuse too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    if stream == here:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _workspace(nbytes: int, device: int, ws, stream):
    if nbytes == 0:
        return c_void_p(None), 0
    if ws is None:
        ws = _new(nbytes, torch.uint8, torch.device("cuda", device), stream)
    p = _dev(ws, device, "ws")
    p.keep = ws  # until the caller's launches are queued: another thread must not be given its memory in between
    return p, ws.numel() * ws.element_size()


def encode_workspace_size(ctx: Context, n: int) -> int:
    b = c_size_t()
    _check(LIB.tq_encode_workspace_size(ctx.handle, n, ctypes.byref(b)))
    return b.value


def encode_kv(ctx: Context, x: torch.Tensor, out: Packed, slots: torch.Tensor = None, ws=None, stream=None):
    """Encode the rows of x ([n, d] or [n, ld] with a row stride) into `out` at `slots`."""
    if x.dim() != 2 or x.shape[1] < ctx.d or x.stride(1) != 1:
        raise ValueError("x must be [n, >=d] with unit column stride")
    n, ld = x.shape[0], x.stride(0)
    xp = _dev(x, ctx.device, "x", contiguous=False)
    sp = c_void_p(None)
    if slots is not None:
        sp = _dev(slots, ctx.device, "slots", torch.int64)
        if slots.numel() != n:
            raise ValueError("slots must have n entries")
    w, wb = _workspace(encode_workspace_size(ctx, n), ctx.device, ws, stream)
    _check(LIB.tq_encode_kv(ctx.handle, xp, _dtype_code(x), n, ld, sp, out.c(ctx), w, wb, _stream_ptr(stream)))
    return out


def scores_workspace_size(ctx: Context, nq: int) -> int:
    b = c_size_t()
    _check(LIB.tq_scores_workspace_size(ctx.handle, nq, ctypes.byref(b)))
    return b.value


def scores(ctx: Context, q: torch.Tensor, keys: Packed, n: int = None, out=None, ws=None, stream=None):
    """Estimated inner products [nq, n] of queries q [nq, d] with slots 0..n-1 of `keys`."""
    if q.dim() != 2 or q.shape[1] != ctx.d:
        raise ValueError(f"q must be [nq, {ctx.d}]")
    n = keys.capacity if n is None else n
    nq = q.shape[0]
    if out is None:
        out = _new((nq, n), torch.float32, q.device, stream)
    if tuple(out.shape) != (nq, n):
        raise ValueError("out must be [nq, n]")
    w, wb = _workspace(scores_workspace_size(ctx, nq), ctx.device, ws, stream)
    _check(LIB.tq_scores(ctx.handle, _dev(q, ctx.device, "q"), _dtype_code(q), nq, keys.c(ctx), n,
                         _dev(out, ctx.device, "out", torch.float32), w, wb, _stream_ptr(stream)))
    return out


def make_attn_desc(kctx: Context, vctx: Context, q_shape, kcache: Packed, vcache: Packed, seq_lens,
                   max_seq_len: int, ctx_stride: int = None, block_table=None, block_size: int = 16,
                   scale: float = 0.0, n_kv_heads: int = None, sparse_v: float = 0.0) -> AttnDesc:
    batch, hq, _ = q_shape
    if n_kv_heads is None:
        raise ValueError("n_kv_heads is required")
    desc = AttnDesc()
    desc.batch, desc.n_q_heads, desc.n_kv_heads, desc.scale = batch, hq, n_kv_heads, scale
    desc.seq_lens = _dev(seq_lens, kctx.device, "seq_lens", torch.int32)
    if seq_lens.numel() != batch:
        raise ValueError("seq_lens must have batch entries")
    if block_table is not None:
        if block_table.dim() != 2 or block_table.shape[0] != batch:
            raise ValueError("block_table must be [batch, max_blocks]")
        desc.block_table = _dev(block_table, kctx.device, "block_table", torch.int32)
        desc.max_blocks = block_table.shape[1]
        desc.block_size = block_size
        desc.ctx_stride = 0
    else:
        desc.block_table = c_void_p(None)
        desc.max_blocks = 0
        desc.block_size = block_size
        desc.ctx_stride = max_seq_len if ctx_stride is None else ctx_stride
    desc.max_seq_len = max_seq_len
    desc.k = kcache.c(kctx)
    desc.v = vcache.c(vctx)
    desc.sparse_v = sparse_v
    # the descriptor holds raw device pointers: it keeps the tensors they point into alive
    desc._keep = (seq_lens, block_table, kcache, vcache)
    return desc


def attend_workspace_size(kctx: Context, vctx: Context, desc: AttnDesc) -> int:
    b = c_size_t()
    _check(LIB.tq_attend_workspace_size(kctx.handle, vctx.handle, ctypes.byref(desc), ctypes.byref(b)))
    return b.value


def attend_decode(kctx: Context, vctx: Context, q: torch.Tensor, kcache: Packed, vcache: Packed, seq_lens,
                  max_seq_len: int, n_kv_heads: int, ctx_stride: int = None, block_table=None,
                  block_size: int = 16, scale: float = 0.0, out=None, ws=None, stream=None, desc=None):
    """One decode step: q [batch, n_q_heads, d] -> out fp32 [batch, n_q_heads, d]."""
    if q.dim() != 3 or q.shape[2] != kctx.d:
        raise ValueError(f"q must be [batch, heads, {kctx.d}]")
    if desc is None:
        desc = make_attn_desc(kctx, vctx, tuple(q.shape), kcache, vcache, seq_lens, max_seq_len, ctx_stride,
                              block_table, block_size, scale, n_kv_heads)
    if out is None:
        out = _new(q.shape, torch.float32, q.device, stream)
    w, wb = _workspace(attend_workspace_size(kctx, vctx, desc), kctx.device, ws, stream)
    _check(LIB.tq_attend_decode(kctx.handle, vctx.handle, ctypes.byref(desc), _dev(q, kctx.device, "q"),
                                _dtype_code(q), _dev(out, kctx.device, "out", torch.float32), w, wb,
                                _stream_ptr(stream)))
    return out


def decode_step_workspace_size(kctx: Context, vctx: Context, desc: AttnDesc, n_new: int) -> int:
    b = c_size_t()
    _check(LIB.tq_decode_step_workspace_size(kctx.handle, vctx.handle, ctypes.byref(desc), n_new, ctypes.byref(b)))
    return b.value


def decode_step(kctx: Context, vctx: Context, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                new_slots: torch.Tensor, desc: AttnDesc, out=None, ws=None, stream=None):
    """tq_decode_step: append k_new / v_new ([n_new, d]) at new_slots, then attend with q
    ([batch, n_q_heads, d]); desc from make_attn_desc with seq_lens already counting the new tokens."""
    if k_new.shape != v_new.shape or k_new.dim() != 2 or k_new.shape[1] != kctx.d or k_new.dtype != v_new.dtype:
        raise ValueError(f"k_new and v_new must both be [n_new, {kctx.d}] with one dtype")
    n_new = k_new.shape[0]
    if new_slots.numel() != n_new:
        raise ValueError("new_slots must have n_new entries")
    if out is None:
        out = _new(q.shape, torch.float32, q.device, stream)
    w, wb = _workspace(decode_step_workspace_size(kctx, vctx, desc, n_new), kctx.device, ws, stream)
    _check(LIB.tq_decode_step(kctx.handle, vctx.handle, ctypes.byref(desc), _dev(k_new, kctx.device, "k_new"),
                              _dev(v_new, kctx.device, "v_new"), _dtype_code(k_new), n_new,
                              _dev(new_slots, kctx.device, "new_slots", torch.int64), _dev(q, kctx.device, "q"),
                              _dtype_code(q), _dev(out, kctx.device, "out", torch.float32), w, wb, _stream_ptr(stream)))
    return out


DEVFLAG_STAGING_TIMEOUT = 1


TQ_ETIMEOUT = 5


def device_status(device: int = 0, clear: bool = False) -> int:
    """TQ_DEVFLAG_* bits raised by the library's kernels on `device` (synchronizes it).  The C call
    returns TQ_ETIMEOUT when a kernel gave up a bounded wait; the flags say so here, and
    check_device() raises for it."""
    f = c_int32()
    st = LIB.tq_device_status(device, ctypes.byref(f), 1 if clear else 0)
    if st not in (0, TQ_ETIMEOUT):
        _check(st)
    return f.value


def check_device(device: int = 0, clear: bool = False):
    """Raise TqError(TQ_ETIMEOUT) if a kernel on `device` gave up waiting since the last clear."""
    f = c_int32()
    _check(LIB.tq_device_status(device, ctypes.byref(f), 1 if clear else 0))


def debug_wait_probe(device: int, polls: int):
    """Test hook: make one bounded wait of every tensor-core attention CTA run out after `polls`
    polls (0 switches it off); see tq_debug_wait_probe."""
    _check(LIB.tq_debug_wait_probe(device, polls))


NOALLOC_SCRATCH_BYTES = 8 << 20


def attend_decode_noalloc(kctx: Context, vctx: Context, q: torch.Tensor, out: torch.Tensor, desc: AttnDesc,
                          stream=None):
    """tq_attend_decode_noalloc: decode attention whose scratch is the library's fixed 8 MiB
    device array, for callers that cannot allocate device memory.  `out` must be preallocated
    (fp32 [batch, n_q_heads, d]); `desc` comes from make_attn_desc.  Calls that overlap on the GPU
    share that array and race; order them on one stream."""
    if q.dim() != 3 or q.shape[2] != kctx.d:
        raise ValueError(f"q must be [batch, heads, {kctx.d}]")
    _check(LIB.tq_attend_decode_noalloc(kctx.handle, vctx.handle, ctypes.byref(desc), _dev(q, kctx.device, "q"),
                                        _dtype_code(q), _dev(out, kctx.device, "out", torch.float32),
                                        _stream_ptr(stream)))
    return out


def search_workspace_size(ctx: Context, nq: int, n: int, k: int) -> int:
    b = c_size_t()
    _check(LIB.tq_search_workspace_size(ctx.handle, nq, n, k, ctypes.byref(b)))
    return b.value


def search_topk(ctx: Context, q: torch.Tensor, db: Packed, k: int, n: int = None, out_scores=None,
                out_idx=None, ws=None, stream=None):
    """Top-k (scores fp32 [nq, k], indices int64 [nq, k]) of queries q [nq, d] over slots 0..n-1."""
    if q.dim() != 2 or q.shape[1] != ctx.d:
        raise ValueError(f"q must be [nq, {ctx.d}]")
    n = db.capacity if n is None else n
    nq = q.shape[0]
    if out_scores is None:
        out_scores = _new((nq, k), torch.float32, q.device, stream)
    if out_idx is None:
        out_idx = _new((nq, k), torch.int64, q.device, stream)
    w, wb = _workspace(search_workspace_size(ctx, nq, n, k), ctx.device, ws, stream)
    _check(LIB.tq_search_topk(ctx.handle, _dev(q, ctx.device, "q"), _dtype_code(q), nq, db.c(ctx), n, k,
                              _dev(out_scores, ctx.device, "out_scores", torch.float32),
                              _dev(out_idx, ctx.device, "out_idx", torch.int64), w, wb, _stream_ptr(stream)))
    return out_scores, out_idx


# the current stream's handle without a Stream object around it (a microsecond per call), where torch has it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _raw_stream(device: int, stream) -> int:
    return _current_stream(device) if stream is None else stream.cuda_stream


@functools.lru_cache(maxsize=256)
def _same_order(shape, whole) -> bool:
    """Whether a contiguous array of `shape` holds what one of shape `whole` = (n_blocks, n_kv_heads, rows, d) does, in
    its order: neighbouring dimensions may be joined, and the blocks split into several dimensions (heads counted
    among the blocks).  An array with the same number of entries in another order is not."""
    blocks, allowed, at = whole[0], set(), 1
    for n in whole:
        at *= n
        allowed.add(at)
    ends, end = set(), 1
    for n in shape:
        end *= n
        ends.add(end)
    if not shape or shape[-1] != whole[3] or end != at:
        return False
    return at == 0 or all(e == 1 or e in allowed or (e < blocks and blocks in ends) for e in ends)


class Pages:
    """Paged-cache addressing (tq_pages): the block table [batch, max_blocks] and the cache's shape.
    Holds the table's tensor; the calls below run on its device."""

    def __init__(self, block_table: torch.Tensor, n_kv_heads: int, block_size: int, n_blocks: int):
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
            raise ValueError("block_table must be a tensor [batch, max_blocks]")
        self.device = block_table.device.index
        self.batch, self.max_blocks = block_table.shape
        self.block_table = block_table
        self.n_kv_heads, self.block_size, self.n_blocks = n_kv_heads, block_size, n_blocks
        self.rows = self.batch * n_kv_heads
        self._dims = (n_blocks, n_kv_heads)  # of the caches, whatever heads the sequences have
        self._c = PagesC(self.device if block_table.is_cuda else -1, self.batch, n_kv_heads, block_size, self.max_blocks,
                         n_blocks, _dev(block_table, self.device, "block_table", torch.int32))
        self.ref = ctypes.byref(self._c)

    def selected(self, sel_table: torch.Tensor) -> "Pages":
        """The same cache as batch * n_kv_heads sequences of one KV head each, over the blocks that
        select_blocks chose."""
        p = Pages(sel_table, 1, self.block_size, self.n_blocks * self.n_kv_heads)
        p._dims = self._dims
        return p

    def _arg(self, t: torch.Tensor, name: str, dtype, shape) -> int:
        """Address of a contiguous tensor of this device with the given type and shape (an int: its number
        of entries)."""
        if (not isinstance(t, torch.Tensor) or t.get_device() != self.device or t.dtype is not dtype or not t.is_contiguous()
                or (t.numel() if type(shape) is int else t.shape) != shape):
            _dev(t, self.device, name, dtype)
            raise ValueError(f"{name} must have shape {shape} (got {tuple(t.shape)})")
        return t.data_ptr()

    def _cache(self, t: torch.Tensor, name: str, per_block: int, d: int, dtype) -> int:
        """Address of an array of `per_block` rows of d per (block, KV head)."""
        whole = (*self._dims, per_block, d)
        if (isinstance(t, torch.Tensor) and t.get_device() == self.device and t.dtype is dtype and t.is_contiguous()
                and (t.shape == whole or _same_order(t.shape, whole))):
            return t.data_ptr()
        _dev(t, self.device, name, dtype)
        raise ValueError(f"{name} must be {list(whole)} (got {list(t.shape)})")


def page_extend(pages: Pages, seq_lens, new_lens, free_blocks, free_head, n_rows: int = None, new_slots=None,
                seq_lens_out=None, granted=None, free_head_out=None, row_offsets=None, stream=None):
    """tq_page_extend: take blocks from free_blocks[free_head:] for new_lens more tokens per sequence,
    write them into pages.block_table, and return (new_slots int64 [n_rows * n_kv_heads], seq_lens_out,
    granted, free_head_out, row_offsets int64 [batch + 1]).  Outputs may be given; new_slots (or n_rows)
    bounds the rows of one call."""
    i32, i64, n = torch.int32, torch.int64, pages.batch
    if new_slots is None:
        if n_rows is None:
            raise ValueError("n_rows or new_slots is required")
        new_slots = _new(n_rows * pages.n_kv_heads, i64, free_head.device, stream)
    if seq_lens_out is None:
        seq_lens_out = _new(n, i32, free_head.device, stream)
    if granted is None:
        granted = _new(n, i32, free_head.device, stream)
    if free_head_out is None:
        free_head_out = _new(1, i32, free_head.device, stream)
    if row_offsets is None:
        row_offsets = _new(n + 1, i64, free_head.device, stream)
    n_free, n_slots, arg = free_blocks.numel(), new_slots.numel(), pages._arg
    _check(LIB.tq_page_extend(
        pages.ref, arg(seq_lens, "seq_lens", i32, n), arg(new_lens, "new_lens", i32, n),
        arg(free_blocks, "free_blocks", i32, n_free), n_free, arg(free_head, "free_head", i32, 1),
        arg(seq_lens_out, "seq_lens_out", i32, n), arg(granted, "granted", i32, n),
        arg(free_head_out, "free_head_out", i32, 1), arg(row_offsets, "row_offsets", i64, n + 1),
        arg(new_slots, "new_slots", i64, n_slots), n_slots, _raw_stream(pages.device, stream)))
    return new_slots, seq_lens_out, granted, free_head_out, row_offsets


def append_kv(pages: Pages, seq_lens, granted, row_offsets, k_new, v_new=None, k_cache=None, v_cache=None, bounds=None,
              stream=None):
    """tq_append_kv: write rows k_new, v_new ([n_rows, n_kv_heads, d], any row stride) into k_cache, v_cache
    ([n_blocks, n_kv_heads, block_size, d]) and keep bounds ([n_blocks, n_kv_heads, 2, d]); lengths, granted
    and row_offsets as page_extend returns them.  Without caches (None) only the bounds are kept."""
    n, h, d = k_new.shape if k_new.dim() == 3 else (0, -1, 0)
    strides, dt, dev, b = k_new.stride(), k_new.dtype, pages.device, pages.batch
    if h != pages.n_kv_heads or (v_new is not None and (v_new.shape != k_new.shape or v_new.dtype is not dt)):
        raise ValueError(f"k_new and v_new must both be [n_rows, {pages.n_kv_heads}, d] with one dtype")
    # the stride of a dimension with one entry says nothing
    v_strides = strides if v_new is None else v_new.stride()
    if (d > 1 and (strides[2] != 1 or v_strides[2] != 1)) or (h > 1 and (strides[1] != d or v_strides[1] != d)):
        raise ValueError("the heads of a row must lie side by side")
    if n > 1 and v_strides[0] != strides[0]:
        raise ValueError("k_new and v_new must have one row stride")
    if k_new.get_device() != dev or (v_new is not None and v_new.get_device() != dev):
        raise ValueError(f"k_new and v_new must be CUDA tensors on device {dev}")
    arg, cache, i32 = pages._arg, pages._cache, torch.int32
    _check(LIB.tq_append_kv(
        pages.ref, arg(seq_lens, "seq_lens", i32, b), arg(granted, "granted", i32, b),
        arg(row_offsets, "row_offsets", torch.int64, b + 1), k_new.data_ptr(), None if v_new is None else v_new.data_ptr(),
        _dtype_code(k_new), d, n, strides[0] if n > 1 else h * d,
        None if k_cache is None else cache(k_cache, "k_cache", pages.block_size, d, dt),
        None if v_cache is None else cache(v_cache, "v_cache", pages.block_size, d, dt),
        None if bounds is None else cache(bounds, "bounds", 2, d, dt), _raw_stream(dev, stream)))


def _queries(pages: Pages, q: torch.Tensor):
    """(address, query heads, d) of q [batch, n_q_heads, d]."""
    shape = q.shape
    if len(shape) != 3 or shape[0] != pages.batch:
        raise ValueError(f"q must be [{pages.batch}, n_q_heads, d]")
    return pages._arg(q, "q", q.dtype, shape), shape[1], shape[2]


def block_scores(pages: Pages, seq_lens, q, bounds, out=None, stream=None):
    """tq_block_scores: upper bounds fp32 [batch * n_kv_heads, max_blocks] of the products of q
    ([batch, n_q_heads, d]) with the keys of every block, from the bounds that append_kv keeps."""
    qp, hq, d = _queries(pages, q)
    if out is None:
        out = _new((pages.rows, pages.max_blocks), torch.float32, q.device, stream)
    _check(LIB.tq_block_scores(
        pages.ref, pages._arg(seq_lens, "seq_lens", torch.int32, pages.batch), qp, _dtype_code(q), hq, d,
        pages._cache(bounds, "bounds", 2, d, q.dtype),
        pages._arg(out, "out", torch.float32, (pages.rows, pages.max_blocks)), _raw_stream(pages.device, stream)))
    return out


def select_blocks(pages: Pages, seq_lens, scores, n_keep: int, n_first: int = 1, n_last: int = 1, table=None, lens=None,
                  stream=None):
    """tq_select_blocks: the first n_first, the last n_last and the best-scored other blocks of every
    (sequence, KV head), n_keep in all, as a block table [batch * n_kv_heads, n_keep] and the tokens in it.
    pages.selected(table) reads the same cache through it; for make_attn_desc it is the block_table of
    batch * n_kv_heads sequences with n_kv_heads = 1."""
    if table is None:
        table = _new((pages.rows, max(n_keep, 0)), torch.int32, scores.device, stream)
    if lens is None:
        lens = _new(pages.rows, torch.int32, scores.device, stream)
    arg, i32 = pages._arg, torch.int32
    _check(LIB.tq_select_blocks(
        pages.ref, arg(seq_lens, "seq_lens", i32, pages.batch),
        arg(scores, "scores", torch.float32, (pages.rows, pages.max_blocks)), n_keep, n_first, n_last,
        arg(table, "table", i32, (pages.rows, max(n_keep, 0))), arg(lens, "lens", i32, pages.rows),
        _raw_stream(pages.device, stream)))
    return table, lens


def attend_paged_workspace_size(pages: Pages, max_seq_len: int, n_q_heads: int, d: int) -> int:
    b = c_size_t()
    _check(LIB.tq_attend_paged_workspace_size(pages.ref, max_seq_len, n_q_heads, d, ctypes.byref(b)))
    return b.value


def attend_paged(pages: Pages, seq_lens, max_seq_len: int, q, k_cache, v_cache, scale: float = 0.0, out=None, ws=None,
                 stream=None):
    """tq_attend_paged: attention of one new token per sequence, q [batch, n_q_heads, d], over the
    uncompressed caches [n_blocks, n_kv_heads, block_size, d] of q's dtype.  out: fp32 (the default) or
    q's dtype."""
    qp, hq, d = _queries(pages, q)
    dev, dt = pages.device, q.dtype
    if out is None:
        out = _new(q.shape, torch.float32, q.device, stream)
    if ws is None:
        ws = _new(attend_paged_workspace_size(pages, max_seq_len, hq, d), torch.uint8, q.device, stream)
    elif ws.get_device() != dev or not ws.is_contiguous():
        _dev(ws, dev, "ws")
    _check(LIB.tq_attend_paged(
        pages.ref, pages._arg(seq_lens, "seq_lens", torch.int32, pages.batch), max_seq_len, qp,
        pages._cache(k_cache, "k_cache", pages.block_size, d, dt), pages._cache(v_cache, "v_cache", pages.block_size, d, dt),
        _dtype_code(q), hq, d, scale, pages._arg(out, "out", out.dtype, q.shape), _dtype_code(out),
        ws.data_ptr(), ws.numel() * ws.element_size(), _raw_stream(dev, stream)))
    return out


def profile_enable(on: bool = True):
    _check(LIB.tq_profile_enable(1 if on else 0))


def profile_reset():
    _check(LIB.tq_profile_reset())


def profile_read() -> dict:
    """{kernel name: (launches, total device ms)} since the last reset."""
    out = {}
    i = 0
    buf = ctypes.create_string_buffer(64)
    while True:
        n, ms = c_int64(), c_double()
        if LIB.tq_profile_read(i, buf, 64, ctypes.byref(n), ctypes.byref(ms)) != 0:
            break
        out[buf.value.decode()] = (n.value, ms.value)
        i += 1
    return out
