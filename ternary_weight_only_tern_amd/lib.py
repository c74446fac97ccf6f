"""ctypes binding of libtern (include/tern.h), with the same names.

Argument marshalling only: torch supplies device memory and streams, every
step of packing and of the products runs in the HIP kernels behind the C ABI.
There is no CPU fallback: importing this module on a machine without the
built library raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_double, c_float, c_int32, c_int64, c_size_t, c_uint32, c_void_p

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtern.so")

TERN_OK = 0
TERN_E_INVAL = -1
TERN_E_ALIGN = -2
TERN_E_UNSUPPORTED = -3
TERN_E_CORRUPT = -4
TERN_E_WORKSPACE = -5
TERN_E_HIP = -6

TERN_FMT_2BIT = 0
TERN_FMT_B3 = 1
TERN_OFF_NONE = 0
TERN_OFF_ROW = 1
TERN_OFF_GROUP = 2
TERN_F16 = 0
TERN_F32 = 1
TERN_SCORE_SOFTMAX = 0
TERN_SCORE_SIGMOID = 1
(TERN_ROPE_PLAIN, TERN_ROPE_LINEAR, TERN_ROPE_BASE, TERN_ROPE_RAMP, TERN_ROPE_WAVES) = range(5)
TERN_KV_PAGE = 64
TERN_KV_SCALE_BITS = 36

(TERN_BUF_PLANE0, TERN_BUF_SCALE0, TERN_BUF_OFFSET, TERN_BUF_MASK, TERN_BUF_ROWPTR,
 TERN_BUF_BLOCKS1, TERN_BUF_BLOCKS2, TERN_BUF_RSCALE1, TERN_BUF_RSCALE2, TERN_NBUF) = range(10)

SYMBOLS = ["tern_row_stride", "tern_check", "tern_packed_sizes", "tern_workspace_bytes",
           "tern_pack", "tern_unpack", "tern_gemv", "tern_gemm", "tern_batch_workspace_bytes",
           "tern_gemv_batched", "tern_plan_create", "tern_plan_run", "tern_plan_run_events", "tern_plan_launches", "tern_plan_destroy", "tern_b3_min_stages", "tern_gemv_noalloc",
           "tern_rotated_workspace_bytes", "tern_plan_create_rotated",
           "tern_bits", "tern_quantize", "tern_rotate", "tern_rotate_batched", "tern_q4_check", "tern_q4_pack", "tern_q4_unpack", "tern_q4_workspace_bytes", "tern_q4_gemm",
           "tern_route", "tern_q4_experts_workspace_bytes", "tern_q4_experts", "tern_q4_tile_rows", "tern_q4_experts_tile_rows",
           "tern_rope_frequencies", "tern_rope", "tern_kv_check", "tern_kv_write", "tern_kv_read",
           "tern_kv_attention_workspace_bytes", "tern_kv_attention", "tern_kv_attention_parts", "tern_kv_tile_rows",
           "tern_read_probe", "tern_status_str", "tern_last_error"]


class tern_matrix(ctypes.Structure):
    _fields_ = [("n", c_int32), ("k", c_int32), ("group", c_int32), ("planes", c_int32),
                ("format", c_int32), ("offset_mode", c_int32),
                ("plane0", c_void_p), ("scale0", c_void_p),
                ("mask", c_void_p * 2), ("rowptr", c_void_p * 2), ("blocks", c_void_p * 2),
                ("rscale", c_void_p * 2), ("offset", c_void_p), ("nnz", c_uint32 * 2)]


class tern_q4(ctypes.Structure):
    _fields_ = [("n", c_int32), ("k", c_int32), ("group", c_int32), ("count", c_int32),
                ("codes", c_void_p), ("scale", c_void_p), ("zero", c_void_p)]


class tern_router(ctypes.Structure):
    _fields_ = [("experts", c_int32), ("topk", c_int32), ("score", c_int32), ("groups", c_int32),
                ("group_best", c_int32), ("keep_groups", c_int32), ("renorm", c_int32), ("scale", c_float),
                ("bias", c_void_p)]


class tern_rotary(ctypes.Structure):
    _fields_ = [("rot", c_int32), ("interleaved", c_int32), ("freq", c_void_p), ("amp", c_float), ("eps", c_float),
                ("norm", c_void_p)]


class tern_kv(ctypes.Structure):
    _fields_ = [("heads", c_int32), ("dim", c_int32), ("pages", c_int32), ("k", c_void_p), ("v", c_void_p),
                ("k_scale", c_void_p), ("v_scale", c_void_p)]


class tern_kv_batch(ctypes.Structure):
    _fields_ = [("count", c_int32), ("rows", c_int32), ("max_rows", c_int32), ("max_len", c_int32),
                ("max_pages", c_int32), ("start", c_void_p), ("len", c_void_p), ("pages", c_void_p)]


class TernError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_str(status)}: {message}")
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load libtern.so (built in-tree by ternary_weight_only_tern_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m ternary_weight_only_tern_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = POINTER(tern_matrix)
    sig = {
        "tern_row_stride": (c_size_t, [c_int32, c_int32, c_int32]),
        "tern_check": (c_int32, [P]),
        "tern_packed_sizes": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, POINTER(c_uint32), c_int32, POINTER(c_size_t)]),
        "tern_workspace_bytes": (c_size_t, [P, c_int32]),
        "tern_pack": (c_int32, [c_void_p, c_void_p, P, c_void_p, c_size_t, c_void_p]),
        "tern_unpack": (c_int32, [P, c_void_p, c_void_p, c_size_t, c_void_p]),
        "tern_gemv": (c_int32, [P, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]),
        "tern_gemm": (c_int32, [P, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]),
        "tern_batch_workspace_bytes": (c_size_t, [P, c_int32, c_int32]),
        "tern_gemv_batched": (c_int32, [P, POINTER(c_void_p), POINTER(c_void_p), c_int32, c_int32, c_int32, c_void_p, c_size_t, c_void_p]),
        "tern_plan_create": (c_int32, [P, POINTER(c_void_p), POINTER(c_void_p), c_int32, c_int32, c_int32, c_void_p, c_size_t, POINTER(c_void_p)]),
        "tern_plan_run": (c_int32, [c_void_p, c_void_p]),
        "tern_plan_run_events": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p]),
        "tern_plan_launches": (c_int32, [c_void_p]),
        "tern_b3_min_stages": (ctypes.c_int64, [ctypes.c_int64]),
        "tern_rotated_workspace_bytes": (c_size_t, [c_void_p, c_int32, c_int32]),
        "tern_plan_create_rotated": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_int32,
                                              c_int32, c_void_p, c_size_t, c_void_p]),
        "tern_gemv_noalloc": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p]),
        "tern_plan_destroy": (None, [c_void_p]),
        "tern_bits": (c_int32, [P, POINTER(c_double), POINTER(c_double), POINTER(c_double)]),
        "tern_quantize": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                                    c_void_p, c_void_p]),
        "tern_rotate": (c_int32, [c_void_p, c_int32, c_void_p, c_int32, c_int32, c_void_p, c_void_p]),
        "tern_rotate_batched": (c_int32, [c_int32, POINTER(c_void_p), c_int32, POINTER(c_void_p), POINTER(c_int32),
                                          c_int32, POINTER(c_void_p), c_void_p]),
        "tern_q4_check": (c_int32, [c_void_p]),
        "tern_q4_pack": (c_int32, [c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
        "tern_q4_unpack": (c_int32, [c_void_p, c_void_p, c_void_p]),
        "tern_q4_workspace_bytes": (c_size_t, [c_void_p, c_int32]),
        "tern_q4_gemm": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]),
        "tern_route": (c_int32, [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p]),
        "tern_q4_experts_workspace_bytes": (c_size_t, [c_void_p, c_void_p, c_int32, c_int32]),
        "tern_q4_experts": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_void_p,
                                      c_int32, c_void_p, c_size_t, c_void_p]),
        "tern_q4_tile_rows": (c_int32, [c_void_p, c_int32]),
        "tern_q4_experts_tile_rows": (c_int32, [c_void_p, c_void_p, c_int32, c_int32]),
        "tern_rope_frequencies": (c_int32, [c_int32, c_double, c_int32, c_double, c_double, c_double, c_int32,
                                            POINTER(c_double), POINTER(c_float)]),
        "tern_rope": (c_int32, [c_void_p, c_int64, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int64,
                                c_void_p]),
        "tern_kv_check": (c_int32, [c_void_p]),
        "tern_kv_write": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p,
                                    c_int64, c_int32, c_void_p, c_void_p, c_void_p]),
        "tern_kv_read": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_void_p]),
        "tern_kv_attention_workspace_bytes": (c_size_t, [c_void_p, c_void_p, c_int32]),
        "tern_kv_attention": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int32, c_float, c_int32, c_int32,
                                        c_void_p, c_void_p, c_size_t, c_void_p]),
        "tern_kv_attention_parts": (c_int32, [c_void_p, c_void_p, c_int32, c_int32]),
        "tern_kv_tile_rows": (c_int32, [c_int32]),
        "tern_read_probe": (c_int32, [c_void_p, c_size_t, c_void_p, c_void_p]),
        "tern_status_str": (ctypes.c_char_p, [c_int32]),
        "tern_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load().tern_status_str(status).decode()


def last_error() -> str:
    return load().tern_last_error().decode()


def check(status: int) -> None:
    if status != TERN_OK:
        raise TernError(status, last_error())


# ---------------------------------------------------------------- thin wrappers
def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def tern_row_stride(k: int, group: int, fmt: int) -> int:
    return load().tern_row_stride(k, group, fmt)


def tern_packed_sizes(n, k, group, fmt, planes, nnz, offset_mode) -> list:
    out = (c_size_t * TERN_NBUF)()
    nz = (c_uint32 * 2)(*(list(nnz) + [0, 0])[:2])
    check(load().tern_packed_sizes(n, k, group, fmt, planes, nz, offset_mode, out))
    return list(out)


class PackedMatrix:
    """Device buffers of one packed matrix (torch tensors) and its descriptor."""

    def __init__(self, n, k, group, planes, fmt, offset_mode, nnz, device="cuda"):
        import torch
        self.n, self.k, self.group, self.planes, self.fmt = n, k, group, planes, fmt
        self.offset_mode = offset_mode
        self.nnz = [int(v) for v in (list(nnz) + [0, 0])[:2]]
        sz = tern_packed_sizes(n, k, group, fmt, planes, self.nnz, offset_mode)
        u8 = dict(dtype=torch.uint8, device=device)
        ng = k // group if group else 0
        self.plane0 = torch.zeros(max(sz[TERN_BUF_PLANE0], 1), **u8)
        self.scale0 = torch.zeros((n, ng), dtype=torch.float16, device=device)
        self.mask, self.rowptr, self.blocks, self.rscale = [], [], [], []
        for p in range(planes - 1):
            self.mask.append(torch.zeros((n, (ng + 31) // 32), dtype=torch.int32, device=device))
            self.rowptr.append(torch.zeros(n + 1, dtype=torch.int32, device=device))
            self.blocks.append(torch.zeros(max(sz[TERN_BUF_BLOCKS1 + p], 1), **u8))
            self.rscale.append(torch.zeros(max(self.nnz[p], 1), dtype=torch.float16, device=device))
        shape = (n,) if offset_mode == TERN_OFF_ROW else (n, ng)
        self.offset = (torch.zeros(shape, dtype=torch.float16, device=device)
                       if offset_mode != TERN_OFF_NONE else None)

    def desc(self) -> tern_matrix:
        d = tern_matrix()
        d.n, d.k, d.group, d.planes = self.n, self.k, self.group, self.planes
        d.format, d.offset_mode = self.fmt, self.offset_mode
        d.plane0, d.scale0 = _ptr(self.plane0), _ptr(self.scale0)
        for p in range(self.planes - 1):
            d.mask[p] = _ptr(self.mask[p])
            d.rowptr[p] = _ptr(self.rowptr[p])
            d.blocks[p] = _ptr(self.blocks[p])
            d.rscale[p] = _ptr(self.rscale[p])
            d.nnz[p] = self.nnz[p]
        d.offset = _ptr(self.offset)
        return d

    def nbytes(self) -> int:
        """Bytes of the representation a product reads (every buffer)."""
        sz = tern_packed_sizes(self.n, self.k, self.group, self.fmt, self.planes, self.nnz,
                               self.offset_mode)
        extra = max(self.planes - 2, 0) * (sz[TERN_BUF_MASK] + sz[TERN_BUF_ROWPTR])
        return sum(sz) + extra


def _zeroed(nbytes: int, device, stream):
    """A zero-filled workspace for a call on `stream`.  The fill is queued on
    torch's current stream.  When the call goes to a stream of the caller's,
    which may be another one, that stream waits for the fill, and the
    allocator is told that the stream uses the buffer, so that it does not
    hand the memory out again (and fill it on torch's stream) before the
    call has finished there."""
    import torch
    ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
    if stream is not None:
        ext = torch.cuda.ExternalStream(stream, device=ws.device)
        ext.wait_stream(torch.cuda.current_stream(ws.device))
        ws.record_stream(ext)
    return ws


def _workspace(desc: tern_matrix, m: int, device="cuda", stream=None):
    return _zeroed(load().tern_workspace_bytes(ctypes.byref(desc), m), device, stream)


def tern_pack(pm: PackedMatrix, trits, scales, mask_bits, offset=None, stream=None, ws=None):
    """Fill pm from device trits [P][N][K] int8, scales [P][N][K/G] fp16 and
    mask_bits [P-1][N][W] int32 (copied into pm.mask); plane-0 scales and the
    offset are copied into pm as given."""
    pm.scale0.copy_(scales[0])
    for p in range(pm.planes - 1):
        pm.mask[p].copy_(mask_bits[p])
    if pm.offset is not None:
        pm.offset.copy_(offset)
    d = pm.desc()
    ws = ws if ws is not None else _workspace(d, 1, pm.plane0.device, stream)
    rs = scales[1:].contiguous() if pm.planes > 1 else None
    check(load().tern_pack(_ptr(trits), _ptr(rs), ctypes.byref(d), _ptr(ws), ws.numel(), _stream(stream)))
    return pm


def tern_unpack(pm: PackedMatrix, out=None, stream=None, ws=None):
    import torch
    d = pm.desc()
    if out is None:
        out = torch.empty((pm.planes, pm.n, pm.k), dtype=torch.int8, device=pm.plane0.device)
    ws = ws if ws is not None else _workspace(d, 1, pm.plane0.device, stream)
    check(load().tern_unpack(ctypes.byref(d), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def _product(fn, pm, x, y_dtype, out, stream, ws):
    import torch
    m = x.shape[0]
    if out is None:
        dt = torch.float32 if y_dtype == TERN_F32 else torch.float16
        out = torch.empty((m, pm.n), dtype=dt, device=x.device)
    d = pm.desc()
    ws = ws if ws is not None else _workspace(d, m, x.device, stream)
    check(fn(ctypes.byref(d), _ptr(x), m, _ptr(out), y_dtype, _ptr(ws), ws.numel(), _stream(stream)))
    return out


def tern_gemv(pm, x, y_dtype=TERN_F16, out=None, stream=None, ws=None):
    return _product(load().tern_gemv, pm, x, y_dtype, out, stream, ws)


def tern_gemv_noalloc(pm, x, out, y_dtype=TERN_F16, stream=None):
    """tern_gemv with the library's fixed per-GPU workspace: the caller
    passes the output tensor `out` ([m][n], fp16 or fp32 per y_dtype); no
    device memory is allocated."""
    d = pm.desc()
    check(load().tern_gemv_noalloc(ctypes.byref(d), _ptr(x), x.shape[0], _ptr(out), y_dtype, _stream(stream)))
    return out


def tern_gemm(pm, x, y_dtype=TERN_F16, out=None, stream=None, ws=None):
    return _product(load().tern_gemm, pm, x, y_dtype, out, stream, ws)


def _arrays(mats, xs, ys):
    n = len(mats)
    descs = (tern_matrix * max(n, 1))(*[m.desc() for m in mats])
    xp = (c_void_p * max(n, 1))(*[x.data_ptr() for x in xs])
    yp = (c_void_p * max(n, 1))(*[y.data_ptr() for y in ys])
    return descs, xp, yp


def tern_gemv_batched(mats, xs, ys, y_dtype=TERN_F16, stream=None, ws=None):
    m = xs[0].shape[0] if xs else 0
    descs, xp, yp = _arrays(mats, xs, ys)
    if ws is None:
        ws = _zeroed(load().tern_batch_workspace_bytes(descs, len(mats), m), xs[0].device, stream)
    check(load().tern_gemv_batched(descs, xp, yp, len(mats), m, y_dtype, _ptr(ws), ws.numel(), _stream(stream)))
    return ys


def _event(e):
    """The HIP event handle of a torch.cuda.Event (created on first record)."""
    if e is None:
        return None
    if not e.cuda_event:
        e.record()
    return e.cuda_event


class Plan:
    """tern_plan_create / tern_plan_run / tern_plan_destroy; with `rots` (a
    list of fp16 rotation-block tensors or None per product) and rot_block,
    tern_plan_create_rotated.  The plan's workspace is a torch tensor that
    lives as long as the Plan: keep the Plan until runs queued on a stream
    other than torch's current one have finished (torch's allocator may hand
    the memory out again as soon as the Plan is gone)."""

    def __init__(self, mats, xs, ys, y_dtype=TERN_F16, rots=None, rot_block=128):
        import torch
        self.m = xs[0].shape[0] if xs else 0
        descs, xp, yp = _arrays(mats, xs, ys)
        if rots is not None:
            nbytes = load().tern_rotated_workspace_bytes(descs, len(mats), self.m)
        else:
            nbytes = load().tern_batch_workspace_bytes(descs, len(mats), self.m)
        # tern_plan_create writes every table and clears its counters itself
        # (synchronously, on the null stream): no fill is queued here, and the
        # caller's queued work on its inputs is finished first
        self.ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=xs[0].device)
        if xs:
            torch.cuda.current_stream(xs[0].device).synchronize()
        self._keep = (mats, xs, ys, rots)
        handle = c_void_p()
        if rots is not None:
            rp = (c_void_p * max(len(rots), 1))(*[None if r is None else r.data_ptr() for r in rots])
            check(load().tern_plan_create_rotated(descs, xp, rp, rot_block, yp, len(mats), self.m, y_dtype,
                                                  _ptr(self.ws), self.ws.numel(), ctypes.byref(handle)))
        else:
            check(load().tern_plan_create(descs, xp, yp, len(mats), self.m, y_dtype, _ptr(self.ws),
                                          self.ws.numel(), ctypes.byref(handle)))
        self.handle = handle

    def run(self, stream=None):
        check(load().tern_plan_run(self.handle, _stream(stream)))

    def run_events(self, before, after, stream=None):
        """run() recording two torch.cuda.Event objects (created with
        enable_timing=True) around the main decode launch."""
        check(load().tern_plan_run_events(self.handle, _stream(stream), _event(before), _event(after)))

    def launches(self):
        """Kernel launches one run() makes (tern_plan_launches)."""
        return int(load().tern_plan_launches(self.handle))

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.tern_plan_destroy(self.handle)
            self.handle = None


def tern_quantize(w, mask_bits=None, group=128, iters=15, stream=None):
    """Quantize fp16 weights w [n][k] (device tensor; torch.float16 or its
    uint16 bits) into (trits int8 [2][n][k], scales fp16 [2][n][k/group],
    offsets fp16 [n][k/group]); mask_bits: int32/uint32 device bitmap
    [n][ceil(k/group/32)] of the groups that get the second plane, or None."""
    import torch
    n, k = w.shape
    ng = k // group if group else 0
    trits = torch.empty((2, n, k), dtype=torch.int8, device=w.device)
    scales = torch.empty((2, n, ng), dtype=torch.float16, device=w.device)
    offset = torch.empty((n, ng), dtype=torch.float16, device=w.device)
    check(load().tern_quantize(_ptr(w), n, k, group, _ptr(mask_bits) if mask_bits is not None else None, iters,
                               _ptr(trits), _ptr(scales), _ptr(offset), _stream(stream)))
    return trits, scales, offset


def tern_rotate(R, x, out=None, stream=None):
    """out = x rotated by the block-diagonal R (device tensors: R fp16
    [k/block][block][block], x fp16 [m][k]); returns out (fp16 [m][k])."""
    import torch
    m, k = x.shape
    block = R.shape[-1]
    if out is None:
        out = torch.empty((m, k), dtype=torch.float16, device=x.device)
    check(load().tern_rotate(_ptr(R), block, _ptr(x), m, k, _ptr(out), _stream(stream)))
    return out


def tern_rotate_batched(Rs, xs, outs=None, stream=None):
    """Rotate several activation tensors in one launch (same block size and
    number of rows); returns the outputs."""
    import torch
    n = len(xs)
    m = xs[0].shape[0] if n else 0
    block = Rs[0].shape[-1] if n else 128
    if outs is None:
        outs = [torch.empty_like(x) for x in xs]
    rp = (c_void_p * max(n, 1))(*[r.data_ptr() for r in Rs])
    xp = (c_void_p * max(n, 1))(*[x.data_ptr() for x in xs])
    op = (c_void_p * max(n, 1))(*[o.data_ptr() for o in outs])
    kk = (c_int32 * max(n, 1))(*[x.shape[1] for x in xs])
    check(load().tern_rotate_batched(n, rp, block, xp, kk, m, op, _stream(stream)))
    return outs


# ---------------------------------------------------------------- 4-bit weights, routing, experts
def _refuse(what: str):
    raise ValueError(what)


def _tensor(t, name, dtypes, device, shape=None):
    """Checks a device tensor argument: its type, device, layout and shape."""
    if t.dtype not in dtypes:
        _refuse(f"{name} is {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
    if t.device != device:
        _refuse(f"{name} is on {t.device}, not {device}")
    if not t.is_contiguous():
        _refuse(f"{name} is not contiguous")
    if shape is not None and t.shape != shape:
        _refuse(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    return t


def _space(ws, device):
    """Checks a caller's workspace; its size and alignment the library checks."""
    if ws.get_device() != device.index or not ws.is_contiguous():
        _refuse(f"a workspace on {ws.device}, or with gaps; contiguous on {device} is wanted")


_torch = _raw_stream = _current_device = _halves = None


def _use_torch():
    """Looks torch's calls up once: a product of a few microseconds notices
    what its wrapper costs.  The stream handle comes without a Stream object
    where torch offers that."""
    global _torch, _raw_stream, _current_device, _halves
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _raw_stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _halves = (torch.float16,)
    _torch = torch
    return torch


def _elsewhere(device):
    """Whether `device` is not the current one (then the call is made again
    with it current)."""
    return device.index != _current_device()


def _fresh(shape, dtype, device, stream):
    """An uninitialised tensor for a call on `stream`.  When that is a stream
    of the caller's, it first waits for torch's current stream (where the
    memory may still be in use), and the allocator is told that it uses the
    tensor, so that the memory is not handed out again before the call is
    done."""
    import torch
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        ext = torch.cuda.ExternalStream(stream, device=t.device)
        ext.wait_stream(torch.cuda.current_stream(t.device))
        t.record_stream(ext)
    return t


def _scratch(nbytes, device, stream):
    import torch
    return _fresh(max(nbytes, 256), torch.uint8, device, stream)


def _count(v):
    """A size that the C interface's 32 bits hold."""
    return v if v < 2 ** 31 else _refuse(f"a size of {v} is too large")


def _bytes(size):
    """A workspace's size; the library's is 0 for sizes that it refuses."""
    return size or _refuse(last_error())


class _Fixed:
    """An object whose descriptor holds its tensors' addresses and sizes: each
    attribute is set once.  A tensor put in another's place would leave the
    library with the address of one that may be gone."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} is not replaced: write into the tensor, or make another {type(self).__name__}")
        self.__dict__[name] = value

    def __delattr__(self, name):
        raise AttributeError(f"{type(self).__name__}.{name} stays as long as its {type(self).__name__}")


class Q4Matrix(_Fixed):
    """4-bit weights on the device: codes uint8 [n][k/2] in tern_q4's word
    order, scale fp16 [n][k/group], zero uint8 [n][k/group] or None (8
    everywhere); or a stack of them, [count][n][...] in every array.  Keeps
    the tensors; makes no copy."""

    def __init__(self, codes, scale, zero=None):
        import torch
        if codes.dim() not in (2, 3) or scale.dim() != codes.dim() or codes.shape[:-1] != scale.shape[:-1]:
            _refuse(f"codes {tuple(codes.shape)} and scale {tuple(scale.shape)} are no 4-bit matrix")
        if codes.device.type != "cuda":
            _refuse(f"codes are on {codes.device}, not on a GPU")
        _tensor(codes, "codes", (torch.uint8,), codes.device)
        _tensor(scale, "scale", (torch.float16,), codes.device)
        if zero is not None:
            _tensor(zero, "zero", (torch.uint8,), codes.device, scale.shape)
        _use_torch()
        self.codes, self.scale, self.zero = codes, scale, zero
        self.device = codes.device
        self.n, self.k = _count(codes.shape[-2]), _count(2 * codes.shape[-1])
        self.count = codes.shape[0] if codes.dim() == 3 else 1
        ng = scale.shape[-1]
        if self.k and (ng < 1 or self.k % ng):
            _refuse(f"k={self.k} in {ng} groups")
        self.group = self.k // ng if self.k else 128
        self._desc = tern_q4(self.n, self.k, self.group, self.count, _ptr(codes), _ptr(scale), _ptr(zero))
        self._at = ctypes.addressof(self._desc)
        check(load().tern_q4_check(self._at))

    @classmethod
    def from_codes(cls, q, scale, zero=None, stream=None):
        """tern_q4_pack: from codes 0..15 of one byte each, uint8 [n][k] (or
        [count][n][k])."""
        import torch
        if q.device.type != "cuda":
            _refuse(f"q is on {q.device}, not on a GPU")
        if q.dim() not in (2, 3) or q.shape[-1] % 2:
            _refuse(f"codes of shape {tuple(q.shape)}")
        _tensor(q, "q", (torch.uint8,), q.device)
        codes = _fresh((*q.shape[:-1], q.shape[-1] // 2), torch.uint8, q.device, stream)
        self = cls(codes, scale, zero)
        with torch.cuda.device(self.device):
            ws = _scratch(256, self.device, stream)
            check(load().tern_q4_pack(_ptr(q), self._at, _ptr(ws), ws.numel(), _stream_of(self.device, stream)))
        return self

    def unpack(self, stream=None):
        """tern_q4_unpack: the codes, one byte each."""
        import torch
        q = _fresh((*self.codes.shape[:-1], self.k), torch.uint8, self.device, stream)
        with torch.cuda.device(self.device):
            check(load().tern_q4_unpack(self._at, _ptr(q), _stream_of(self.device, stream)))
        return q


def _stream_of(device, stream):
    return stream if stream is not None else _raw_stream(device.index)


def _y_type(y_dtype):
    if y_dtype == TERN_F16:
        return _torch.float16
    if y_dtype == TERN_F32:
        return _torch.float32
    _refuse(f"unknown output dtype {y_dtype}")


def tern_q4_workspace(w: Q4Matrix, m: int):
    """A workspace for tern_q4_gemm with up to m activation rows."""
    return _scratch(_bytes(load().tern_q4_workspace_bytes(w._at, _count(m))), w.device, None)


def tern_q4_gemm(w: Q4Matrix, x, y_dtype=TERN_F16, out=None, stream=None, ws=None):
    """y = x W^T (x fp16 [m][k], contiguous); returns y [m][n], fp16 or fp32
    per y_dtype, in `out` if given."""
    device = w.device
    if _elsewhere(device):
        with _torch.cuda.device(device):
            return tern_q4_gemm(w, x, y_dtype, out, stream, ws)
    _tensor(x, "x", _halves, device)
    shape = x.shape
    if len(shape) != 2 or shape[1] != w.k:
        _refuse(f"x has shape {tuple(shape)}, not [m][{w.k}]")
    m = _count(shape[0])
    kind = _y_type(y_dtype)
    if out is None:
        out = _fresh((m, w.n), kind, device, stream)
    else:
        _tensor(out, "out", (kind,), device, (m, w.n))
    if ws is None:
        ws = _scratch(load().tern_q4_workspace_bytes(w._at, m), device, stream)
    else:
        _space(ws, device)
    check(load().tern_q4_gemm(w._at, x.data_ptr(), m, out.data_ptr(), y_dtype, ws.data_ptr(), ws.nbytes,
                              _stream_of(device, stream)))
    return out


def tern_route(logits, topk, score=TERN_SCORE_SOFTMAX, bias=None, groups=1, group_best=1, keep_groups=1, renorm=True,
               scale=1.0, ids=None, weights=None, stream=None):
    """Routes tokens to experts: (ids int32 [m][topk], weights fp32
    [m][topk]) from logits fp16 or fp32 [m][experts], contiguous."""
    torch = _torch or _use_torch()
    device = logits.device
    if device.type != "cuda" or logits.dim() != 2:
        _refuse(f"logits of shape {tuple(logits.shape)} on {device}, not [m][experts] on a GPU")
    if _elsewhere(device):
        with torch.cuda.device(device):
            return tern_route(logits, topk, score, bias, groups, group_best, keep_groups, renorm, scale, ids, weights,
                              stream)
    _tensor(logits, "logits", (torch.float16, torch.float32), device)
    m, experts = _count(logits.size(0)), _count(logits.size(1))
    _count(max(topk, groups, group_best, keep_groups))
    if bias is not None:
        _tensor(bias, "bias", (torch.float32,), device, (experts,))
    if ids is None:
        ids = _fresh((m, max(topk, 0)), torch.int32, device, stream)
    else:
        _tensor(ids, "ids", (torch.int32,), device, (m, topk))
    if weights is None:
        weights = _fresh((m, max(topk, 0)), torch.float32, device, stream)
    else:
        _tensor(weights, "weights", (torch.float32,), device, (m, topk))
    r = tern_router(experts, topk, score, groups, group_best, keep_groups, 1 if renorm else 0, scale, _ptr(bias))
    check(load().tern_route(logits.data_ptr(), TERN_F32 if logits.dtype == torch.float32 else TERN_F16, m,
                            ctypes.addressof(r), ids.data_ptr(), weights.data_ptr(), _stream_of(device, stream)))
    return ids, weights


def tern_q4_experts_workspace(gate_up: Q4Matrix, down: Q4Matrix, m: int, topk: int):
    """A workspace for tern_q4_experts with up to m tokens of topk slots."""
    return _scratch(_bytes(load().tern_q4_experts_workspace_bytes(gate_up._at, down._at, _count(m), _count(topk))), down.device, None)


def tern_q4_experts(gate_up: Q4Matrix, down: Q4Matrix, x, ids, weights, y_dtype=TERN_F16, out=None, stream=None,
                    ws=None):
    """The routed experts' layer: y [m][down.n] from x fp16 [m][gate_up.k],
    ids int32 and weights fp32 [m][topk] (as tern_route returns them)."""
    torch, device = _torch, gate_up.device
    if _elsewhere(device):
        with torch.cuda.device(device):
            return tern_q4_experts(gate_up, down, x, ids, weights, y_dtype, out, stream, ws)
    _tensor(x, "x", (torch.float16,), device)
    if down.device != device:
        _refuse(f"down is on {down.device}, not {device}")
    if x.dim() != 2 or x.size(1) != gate_up.k:
        _refuse(f"x has shape {tuple(x.shape)}, not [m][{gate_up.k}]")
    m = _count(x.size(0))
    _tensor(ids, "ids", (torch.int32,), device)
    if ids.dim() != 2 or ids.size(0) != m:
        _refuse(f"ids have shape {tuple(ids.shape)}, not [{m}][topk]")
    _tensor(weights, "weights", (torch.float32,), device, ids.shape)
    topk = _count(ids.size(1))
    kind = _y_type(y_dtype)
    if out is None:
        out = _fresh((m, down.n), kind, device, stream)
    else:
        _tensor(out, "out", (kind,), device, (m, down.n))
    if ws is None:
        ws = _scratch(load().tern_q4_experts_workspace_bytes(gate_up._at, down._at, m, topk), device, stream)
    else:
        _space(ws, device)
    check(load().tern_q4_experts(gate_up._at, down._at, x.data_ptr(), m, ids.data_ptr(), weights.data_ptr(), topk,
                                 out.data_ptr(), y_dtype, ws.data_ptr(), ws.nbytes, _stream_of(device, stream)))
    return out


class Q4Experts:
    """A layer of experts with its router's settings: run() routes the tokens
    by their logits (tern_route) and applies their experts
    (tern_q4_experts)."""

    def __init__(self, gate_up: Q4Matrix, down: Q4Matrix, topk, score=TERN_SCORE_SOFTMAX, bias=None, groups=1,
                 group_best=1, keep_groups=1, renorm=True, scale=1.0):
        self.gate_up, self.down, self.topk = gate_up, down, topk
        self._route = dict(score=score, bias=bias, groups=groups, group_best=group_best, keep_groups=keep_groups,
                           renorm=renorm, scale=scale)

    def run(self, x, logits, y_dtype=TERN_F16, out=None, stream=None, ws=None):
        """y [m][down.n] for x fp16 [m][k] and logits [m][experts]."""
        if tuple(logits.shape) != (x.shape[0], self.down.count):
            _refuse(f"logits have shape {tuple(logits.shape)}, not {(x.shape[0], self.down.count)}")
        ids, weights = tern_route(logits, self.topk, stream=stream, **self._route)
        return tern_q4_experts(self.gate_up, self.down, x, ids, weights, y_dtype, out, stream, ws)


# ---------------------------------------------------------------- positions, cache, attention
def tern_rope_frequencies(rot, base=1e6, scaling=TERN_ROPE_PLAIN, factor=1.0, low=1.0, high=32.0, trained=4096):
    """(frequencies fp64 [rot/2] on the host, amplitude) of rotary positions;
    see tern_rope_frequencies in tern.h for the scalings."""
    import torch
    freq = torch.empty(_count(max(rot, 0)) // 2, dtype=torch.float64)
    amp = c_float()
    check(load().tern_rope_frequencies(rot, base, scaling, factor, low, high, trained,
                                       ctypes.cast(freq.data_ptr(), POINTER(c_double)), ctypes.byref(amp)))
    return freq, amp.value


class Rope(_Fixed):
    """tern_rotary: how a head's values turn.  freq: fp64 device tensor
    [rot/2]; norm: fp16 device tensor [dim] or None, the weights of an RMS norm
    of each head before.  Keeps the tensors."""

    def __init__(self, freq, interleaved=False, amp=1.0, norm=None, eps=1e-6):
        import torch
        if freq.device.type != "cuda" or freq.dim() != 1:
            _refuse(f"freq of shape {tuple(freq.shape)} on {freq.device}, not [rot/2] on a GPU")
        _tensor(freq, "freq", (torch.float64,), freq.device)
        if norm is not None:
            _tensor(norm, "norm", (torch.float16,), freq.device)
            if norm.dim() != 1:
                _refuse(f"norm has shape {tuple(norm.shape)}, not [dim]")
        _use_torch()
        self.freq, self.norm, self.device = freq, norm, freq.device
        self.dim = None if norm is None else norm.numel()
        self._desc = tern_rotary(2 * _count(freq.numel()), int(bool(interleaved)), _ptr(freq), amp, eps, _ptr(norm))
        self._at = ctypes.addressof(self._desc)

    def _of(self, device, dim):
        """The descriptor's address, for heads of dim elements on a device."""
        if self.device != device:
            _refuse(f"the rotary frequencies are on {self.device}, not {device}")
        if self.dim is not None and self.dim != dim:
            _refuse(f"a norm of {self.dim} elements for heads of {dim}")
        return self._at


def _heads(t, name, device, heads, dim):
    """Checks rows of heads, fp16 [m][heads][dim] whose heads follow each
    other (heads None: any number); the rows' stride."""
    if t.dtype is _halves[0] and t.device == device:
        shape = t.shape
        if len(shape) == 3:
            m, h, d = shape
            if d == dim and (heads is None or h == heads) and 0 < m < 2 ** 31 and 0 < h < 2 ** 31:
                if t.is_contiguous():
                    return h * d
                row, head, step = t.stride()
                if step == 1 and head == d and m > 1:
                    return row
    return _heads_slowly(t, name, device, heads, dim)


def _heads_slowly(t, name, device, heads, dim):
    """The same where a size is 1 or 0, and what is wrong otherwise."""
    if t.dtype != _torch.float16 or t.device != device:
        _refuse(f"{name} is {t.dtype} on {t.device}, not torch.float16 on {device}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        _refuse(f"{name} has shape {tuple(shape)}, not [m][{'heads' if heads is None else heads}][{dim}]")
    m, heads = _count(shape[0]), _count(shape[1])
    row, head, step = t.stride()
    if not m * heads * dim:
        return 0
    if (step != 1 and dim > 1) or (head != dim and heads > 1):
        _refuse(f"{name} has strides {(row, head, step)}: a row's heads have to follow each other")
    return row if m > 1 else heads * dim


def tern_rope(x, pos, rope: Rope, out=None, stream=None):
    """x fp16 [m][heads][dim] turned, row r by pos[r] (int32 [m]); in `out`
    if given, which may be x."""
    torch = _torch or _use_torch()
    device = rope.device
    if _elsewhere(device):
        with torch.cuda.device(device):
            return tern_rope(x, pos, rope, out, stream)
    shape = x.shape
    if len(shape) != 3:
        _refuse(f"x has shape {tuple(shape)}, not [m][heads][dim]")
    m, heads, dim = shape
    x_stride = _heads(x, "x", device, heads, dim)
    _tensor(pos, "pos", (torch.int32,), device, (m,))
    if out is None:
        out = _fresh((m, heads, dim), torch.float16, device, stream)
    elif out.shape != shape:
        _refuse(f"out has shape {tuple(out.shape)}, not {tuple(shape)}")
    check((_lib or load()).tern_rope(x.data_ptr(), x_stride, m, heads, _count(dim), pos.data_ptr(), rope._of(device, dim),
                                     out.data_ptr(), _heads(out, "out", device, heads, dim), _stream_of(device, stream)))
    return out


class KvCache(_Fixed):
    """tern_kv: a paged cache in 8 bits.  k, v: uint8 [pages][heads][64][dim]
    (the bytes of a (page, head) in tern_kv's order), k_scale, v_scale: fp32
    [pages][heads], 0, NaN or from 2^-36 to 2^36.  Keeps the tensors; makes no
    copy."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        if k.device.type != "cuda":
            _refuse(f"the cache is on {k.device}, not on a GPU")
        if k.dim() != 4 or k.size(2) != TERN_KV_PAGE:
            _refuse(f"k has shape {tuple(k.shape)}, not [pages][heads][{TERN_KV_PAGE}][dim]")
        device = k.device
        _tensor(k, "k", (torch.uint8,), device)
        _tensor(v, "v", (torch.uint8,), device, k.shape)
        _tensor(k_scale, "k_scale", (torch.float32,), device, k.shape[:2])
        _tensor(v_scale, "v_scale", (torch.float32,), device, k.shape[:2])
        _use_torch()
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, device
        self.pages, self.heads, _, self.dim = k.shape
        self._desc = tern_kv(_count(self.heads), _count(self.dim), _count(self.pages), _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale))
        self._at = ctypes.addressof(self._desc)
        check(load().tern_kv_check(self._at))

    @classmethod
    def empty(cls, pages, heads, dim, device="cuda"):
        """A cache of zeros (every scale 0)."""
        import torch
        code = lambda: torch.full((pages, heads, TERN_KV_PAGE, dim), 128, dtype=torch.uint8, device=device)
        scale = lambda: torch.zeros((pages, heads), dtype=torch.float32, device=device)
        return cls(code(), code(), scale(), scale())


class KvBatch(_Fixed):
    """tern_kv_batch: the sequences of a call.  len: int32 [count], tokens with
    the call's rows; pages: int32 [count][max_pages]; max_rows: rows of a
    sequence at most; start: int32 [count + 1], or None where every sequence
    has max_rows rows; max_len: bound of len for the choice of kernels (default
    what the pages hold).  Keeps the tensors, whose contents may change between
    calls; its attributes may not (another batch takes other tensors)."""

    def __init__(self, len, pages, max_rows, start=None, max_len=None):
        import torch
        device = len.device
        if device.type != "cuda" or len.dim() != 1 or pages.dim() != 2:
            _refuse(f"len {tuple(len.shape)} and pages {tuple(pages.shape)} on {device} are no batch on a GPU")
        count = len.numel()
        _tensor(len, "len", (torch.int32,), device)
        _tensor(pages, "pages", (torch.int32,), device, (count, pages.size(1)))
        if start is not None:
            _tensor(start, "start", (torch.int32,), device, (count + 1,))
        _use_torch()
        self.len, self.pages, self.start, self.device = len, pages, start, device
        self.count, self.max_rows = _count(count), _count(max_rows)
        self.max_len = _count(pages.size(1) * TERN_KV_PAGE if max_len is None else max_len)
        self._descs = {}

    def _of(self, device, rows):
        """The descriptor for so many rows (held by the caller while it is in
        use: another thread's call may clear the ones kept here)."""
        if self.device != device:
            _refuse(f"the batch is on {self.device}, not {device}")
        d = self._descs.get(rows)
        if d is None:
            if len(self._descs) >= 64:
                self._descs.clear()
            d = tern_kv_batch(self.count, _count(rows), self.max_rows, self.max_len, self.pages.size(1),
                              _ptr(self.start), _ptr(self.len), _ptr(self.pages))
            self._descs[rows] = d
        return d


def tern_kv_write(cache: KvCache, batch: KvBatch, k, v, rope=None, q=None, q_rope=None, q_out=None, stream=None):
    """Writes the rows k, v fp16 [m][heads][dim] into the cache, k turned by
    `rope` first if given.  With q (fp16 [m][q_heads][dim]) its rows are turned
    by q_rope in the same launch: returns q_out, contiguous, in `q_out` if
    given (which may be q)."""
    device, dim = cache.device, cache.dim
    if _elsewhere(device):
        with _torch.cuda.device(device):
            return tern_kv_write(cache, batch, k, v, rope, q, q_rope, q_out, stream)
    k_stride = _heads(k, "k", device, cache.heads, dim)
    v_stride = _heads(v, "v", device, cache.heads, dim)
    m = k.shape[0]
    if v.shape[0] != m:
        _refuse(f"{v.shape[0]} rows of v and {m} of k")
    q_at = q_out_at = None
    q_stride = q_heads = 0
    if q is not None:
        q_stride = _heads(q, "q", device, None, dim)
        rows, q_heads, _ = q.shape
        if rows != m:
            _refuse(f"{rows} rows of q and {m} of k")
        if q_rope is None:
            _refuse("q without q_rope")
        if q_out is None:
            q_out = _fresh((m, q_heads, dim), _torch.float16, device, stream)
        else:
            _tensor(q_out, "q_out", _halves, device, (m, q_heads, dim))
        q_at, q_out_at = q.data_ptr(), q_out.data_ptr()
    desc = batch._of(device, m)
    check((_lib or load()).tern_kv_write(cache._at, ctypes.addressof(desc), k.data_ptr(), k_stride, v.data_ptr(), v_stride,
                                         None if rope is None else rope._of(device, dim), q_at, q_stride, q_heads,
                                         None if q is None else q_rope._of(device, dim), q_out_at, _stream_of(device, stream)))
    return q_out


def tern_kv_read(cache: KvCache, batch: KvBatch, rows=None, y_dtype=TERN_F16, k=None, v=None, stream=None):
    """The values of the batch's rows (k, v) back, [m][heads][dim], in fp16 or
    fp32; in `k` and `v` if given.  rows: m (default count * max_rows, or the
    rows of k)."""
    device = cache.device
    if _elsewhere(device):
        with _torch.cuda.device(device):
            return tern_kv_read(cache, batch, rows, y_dtype, k, v, stream)
    if rows is None:
        rows = k.size(0) if k is not None else v.size(0) if v is not None else batch.count * batch.max_rows
    shape = (_count(rows), cache.heads, cache.dim)
    given = k if k is not None else v
    kind = _y_type(y_dtype) if given is None else given.dtype
    if kind not in (_torch.float16, _torch.float32):
        _refuse(f"unknown output dtype {kind}")
    k = _fresh(shape, kind, device, stream) if k is None else _tensor(k, "k", (kind,), device, shape)
    v = _fresh(shape, kind, device, stream) if v is None else _tensor(v, "v", (kind,), device, shape)
    desc = batch._of(device, rows)
    check(load().tern_kv_read(cache._at, ctypes.addressof(desc), k.data_ptr(), v.data_ptr(),
                              TERN_F32 if kind == _torch.float32 else TERN_F16, _stream_of(device, stream)))
    return k, v


def tern_kv_attention_workspace(cache: KvCache, batch: KvBatch, rows: int, q_heads: int):
    """A workspace for tern_kv_attention with up to `rows` rows of q_heads
    heads and no longer sequences than the batch's max_len."""
    desc = batch._of(cache.device, rows)
    return _scratch(_bytes(load().tern_kv_attention_workspace_bytes(cache._at, ctypes.addressof(desc), _count(q_heads))),
                    cache.device, None)


def tern_kv_attention(cache: KvCache, batch: KvBatch, q, scale=None, window=0, causal=True, out=None, stream=None,
                      ws=None):
    """Attention of the rows q fp16 [m][q_heads][dim] over the cache; returns
    y fp16 [m][q_heads][dim], in `out` if given.  scale: of the scores (default
    dim ** -0.5); window: tokens a row sees at most (0: all).  Single tokens
    beside a prompt's rows are faster in a call of their own."""
    device, dim = cache.device, cache.dim
    if _elsewhere(device):
        with _torch.cuda.device(device):
            return tern_kv_attention(cache, batch, q, scale, window, causal, out, stream, ws)
    q_stride = _heads(q, "q", device, None, dim)
    m, q_heads = q.shape[0], q.shape[1]
    if out is None:
        out = _fresh((m, q_heads, dim), _torch.float16, device, stream)
    else:
        _tensor(out, "out", _halves, device, q.shape)
    desc, lib = batch._of(device, m), _lib or load()
    at = ctypes.addressof(desc)
    if ws is None:
        ws = _scratch(lib.tern_kv_attention_workspace_bytes(cache._at, at, q_heads), device, stream)
    else:
        _space(ws, device)
    check(lib.tern_kv_attention(cache._at, at, q.data_ptr(), q_stride, q_heads, dim ** -0.5 if scale is None else scale,
                                _count(window), 1 if causal else 0, out.data_ptr(), ws.data_ptr(), ws.nbytes,
                                _stream_of(device, stream)))
    return out


def tern_kv_tile_rows(rows: int = -1) -> int:
    """The rows of attention's tiles in this thread's calls: 64 or 128 sets them,
    0 restores the rule, -1 queries; returns the setting before."""
    return load().tern_kv_tile_rows(rows)


def tern_read_probe(buf, sink, stream=None) -> None:
    """Plain streaming read of a whole device tensor (measurement aid)."""
    check(load().tern_read_probe(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), _stream(stream)))


def tern_b3_min_stages(stages: int = -2) -> int:
    """Threshold (in 64-row stages per launch) from which base-3 products at
    m <= 4 take the matrix-core stream kernel: stages >= 0 sets it, -1
    restores the default, -2 queries; returns the value in effect before."""
    return int(load().tern_b3_min_stages(stages))


def tern_bits(pm: PackedMatrix) -> dict:
    d = pm.desc()
    info, plane, storage = c_double(), c_double(), c_double()
    check(load().tern_bits(ctypes.byref(d), ctypes.byref(info), ctypes.byref(plane), ctypes.byref(storage)))
    return dict(info=info.value, plane=plane.value, storage=storage.value)
