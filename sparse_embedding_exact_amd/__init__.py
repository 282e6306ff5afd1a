"""Exact all-pairs cosine similarity of sparse embeddings on MI355X (gfx950).

Thin Python binding of the C ABI in ``include/sps.h`` (``libsps.so``).
Arguments are marshalled here; every step of the computation runs in the
library's HIP kernels. PyTorch only provides device memory and streams.

Page followed: "稀疏嵌入批量相似度计算的工程化实践" (Engineering practice of
bulk similarity for sparse embeddings): §3.1 defines the cosine over the
shared support, §5.2 the norms, §2.2 and §4.4 the item-chunk streaming with
8192-item chunks, §2.3 the full float32 output.

Typical use::

    items = sps.prepare(sps.CSR.from_host(item_csr, "cuda"), chunk_size=8192)
    queries = sps.prepare_queries(sps.CSR.from_host(query_csr, "cuda"), items)
    out = torch.empty(n_query, 8192, device="cuda")
    for c in range(items.num_chunks):
        sps.cosine_chunk(queries, items, c, out)   # out[:, :chunk_len] = S[:, chunk c]
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsps.so")

SPS_OK = 0
_STATUS = {
    0: "SPS_OK", -1: "SPS_ERR_INVALID_ARGUMENT", -2: "SPS_ERR_BAD_CSR",
    -3: "SPS_ERR_DIM_MISMATCH", -4: "SPS_ERR_WORKSPACE_TOO_SMALL", -5: "SPS_ERR_CHUNK_RANGE",
    -6: "SPS_ERR_OVERFLOW", -7: "SPS_ERR_HIP", -8: "SPS_ERR_UNSUPPORTED",
}


class SpsError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (_STATUS.get(status, status), msg))
        self.status = status


class _Csr(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("n_cols", ctypes.c_int64), ("nnz", ctypes.c_int64),
                ("indptr", ctypes.c_void_p), ("indices", ctypes.c_void_p),
                ("values", ctypes.c_void_p)]


class _Bsc(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("n_cols", ctypes.c_int64), ("nnz", ctypes.c_int64),
                ("indptr", ctypes.c_void_p), ("bptr", ctypes.c_void_p),
                ("blocks", ctypes.c_void_p), ("block_bytes", ctypes.c_int64),
                ("offsets", ctypes.c_void_p), ("offsets_bytes", ctypes.c_int64),
                ("values", ctypes.c_void_p)]


class _SliceView(ctypes.Structure):
    _fields_ = [("item_begin", ctypes.c_int64), ("slice_len", ctypes.c_int32),
                ("slice_nnz", ctypes.c_int32), ("post", ctypes.c_void_p),
                ("item_inv_norm", ctypes.c_void_p)]


class _Scores(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("n_rows", ctypes.c_int64),
                ("n_cols", ctypes.c_int64), ("ld", ctypes.c_int64), ("col_begin", ctypes.c_int64)]


class _Int8Rows(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("n_rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("ld", ctypes.c_int64)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t

# name -> (restype, argtypes); every symbol include/sps.h declares
SIGNATURES = {
    "sps_items_workspace_size": (_I32, [_I64, _I64, _I64, _I32, ctypes.POINTER(_SZ),
                                        ctypes.POINTER(_SZ)]),
    "sps_prepare": (_I32, [ctypes.POINTER(_Csr), _I32, _P, _SZ, _P, _SZ, _P,
                           ctypes.POINTER(_P)]),
    "sps_items_info": (_I32, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                              ctypes.POINTER(_I64), ctypes.POINTER(_I32), ctypes.POINTER(_I32)]),
    "sps_items_slices": (_I32, [_P, ctypes.POINTER(_I32), ctypes.POINTER(_I32),
                                ctypes.POINTER(_I64)]),
    "sps_items_slice_view": (_I32, [_P, _I64, _P, ctypes.POINTER(_SliceView)]),
    "sps_items_slice_col_ptr": (_I32, [_P, _I64, _P, _P, _P]),
    "sps_items_heavy_dims": (_I32, [_P, _P, _P, _I32, ctypes.POINTER(_I32)]),
    "sps_items_destroy": (None, [_P]),
    "sps_queries_workspace_size": (_I32, [_P, _I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    "sps_prepare_queries": (_I32, [ctypes.POINTER(_Csr), _P, _P, _SZ, _P, ctypes.POINTER(_P)]),
    "sps_queries_inv_norms": (_I32, [_P, ctypes.POINTER(_P)]),
    "sps_queries_destroy": (None, [_P]),
    "sps_cosine_chunk": (_I32, [_P, _P, _I32, _P, _I64, _P, _P]),
    "sps_cosine_chunk_static": (_I32, [_P, _P, _I32, _P, _I64, _P, _P]),
    "sps_cosine_stream": (_I32, [_P, _P, _I32, _I32, _P, _I64, _P, _P]),
    "sps_cosine_stream_host": (_I32, [_P, _P, _I32, _I32, _P, _I64, _P, _P, _I64, _P, _P, _P]),
    "sps_cosine_chunk_threshold": (_I32, [_P, _P, _I32, ctypes.c_float, _P, _I64, _P, _P, _P]),
    "sps_items_half_workspace_size": (_I32, [_P, ctypes.POINTER(_SZ)]),
    "sps_items_enable_half": (_I32, [_P, _P, _SZ, _P]),
    "sps_cosine_chunk_half": (_I32, [_P, _P, _I32, _P, _I64, _P, _P]),
    "sps_select_workspace_size": (_I32, [_I64, _I64, _I32, ctypes.POINTER(_SZ)]),
    "sps_select_chunk": (_I32, [ctypes.POINTER(_Scores), _P, _I32, _I32, _P, _P, _P, _SZ, _P]),
    "sps_beam_workspace_size": (_I32, [_I64, _I64, _I32, _I32, ctypes.POINTER(_SZ)]),
    "sps_beam_select": (_I32, [ctypes.POINTER(_Scores), _P, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "sps_beam_join": (_I32, [_P, _P, _I64, _I32, _I32, _I32, _P, _P, _P, _P]),
    "sps_reorder_states": (_I32, [_P, _I32, _P, _I64, _I64, _P]),
    "sps_distill_workspace_size": (_I32, [_I64, _I32, ctypes.POINTER(_SZ)]),
    "sps_distill_rows_workspace_size": (_I32, [_I64, _I64, _I32, ctypes.POINTER(_SZ)]),
    "sps_distill_prepare": (_I32, [_P, _P, _P, _I64, _I32, _I64, ctypes.c_float, _P, _SZ, _P,
                                   ctypes.POINTER(_P)]),
    "sps_distill_chunk": (_I32, [_P, ctypes.POINTER(_Scores), _I32, _P]),
    "sps_distill_loss": (_I32, [_P, _P, _P, _P]),
    "sps_distill_chunk_grad": (_I32, [_P, ctypes.POINTER(_Scores), _P, _P, _I32, _I64, _P]),
    "sps_distill_destroy": (None, [_P]),
    "sps_distill_rows": (_I32, [ctypes.POINTER(_Scores), _P, _P, _P, _I32, ctypes.c_float, _P, _P,
                                _P, _I32, _I64, _P, _SZ, _P]),
    "sps_cosine_grad_workspace_size": (_I32, [_I64, _P, ctypes.POINTER(_SZ)]),
    "sps_cosine_grad": (_I32, [ctypes.POINTER(_Csr), _P, _I32, ctypes.POINTER(_Scores), _I32, _I32,
                               _P, _P, _SZ, _P]),
    "sps_cosine_grad_both_workspace_size": (_I32, [_I64, _I64, ctypes.POINTER(_SZ)]),
    "sps_cosine_grad_both": (_I32, [ctypes.POINTER(_Csr), ctypes.POINTER(_Csr),
                                    ctypes.POINTER(_Scores), _P, _P, _P, _SZ, _P]),
    "sps_cosine_grad_values": (_I32, [ctypes.POINTER(_Csr), _P, _P, _P]),
    "sps_quantize_rows": (_I32, [ctypes.POINTER(_Scores), _P, _I64, _P, _P]),
    "sps_dequantize_rows": (_I32, [ctypes.POINTER(_Int8Rows), _P, _I32, _I64, _P]),
    "sps_int8_scores": (_I32, [ctypes.POINTER(_Int8Rows), ctypes.POINTER(_Int8Rows), _P, _I32, _I64,
                               _P]),
    "sps_dense_ce_workspace_size": (_I32, [ctypes.POINTER(_Scores), ctypes.POINTER(_Scores), _I32,
                                           _I32, ctypes.POINTER(_SZ)]),
    "sps_dense_ce": (_I32, [ctypes.POINTER(_Scores), ctypes.POINTER(_Scores), _P, _P, ctypes.c_float,
                            _P, _P, _P, _I64, _P, _I64, _I32, _P, _SZ, _P]),
    "sps_row_inv_norms": (_I32, [ctypes.POINTER(_Csr), _P, _P]),
    "sps_bsc_offsets_bytes": (_I32, [_I64, ctypes.POINTER(_SZ)]),
    "sps_bsc_encode_sizes": (_I32, [ctypes.POINTER(_Csr), _P, _P, _P, ctypes.POINTER(_I64)]),
    "sps_bsc_encode": (_I32, [ctypes.POINTER(_Csr), _P, _P, _I64, _P, _I64, _P]),
    "sps_bsc_decode": (_I32, [ctypes.POINTER(_Bsc), _P, _P, _P]),
    "sps_validate_csr": (_I32, [ctypes.POINTER(_Csr), _P, _P, ctypes.POINTER(_I64),
                                ctypes.POINTER(_I32)]),
    "sps_status_string": (ctypes.c_char_p, [_I32]),
    "sps_last_error_message": (ctypes.c_char_p, []),
}

_lib = None


def load_library(path: str | None = None):
    """Load libsps.so (building it with hipcc first if it is absent).

    There is no fallback: without the HIP library nothing here runs.
    """
    global _lib
    if _lib is not None and path is None:
        return _lib
    # torch ships its own HIP runtime and this library links the system one: the
    # process holds both, and torch's must initialise the GPU first
    if torch.cuda.is_available():
        torch.cuda.init()
    p = path or LIB_PATH
    if not os.path.exists(p):
        from . import _build
        _build.build()
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(st: int):
    if st != SPS_OK:
        msg = _lib.sps_last_error_message().decode(errors="replace")
        raise SpsError(st, msg)


def _stream_ptr(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _workspace(nbytes: int, device) -> tuple[torch.Tensor, int]:
    """uint8 device buffer of at least nbytes, 256-byte aligned."""
    buf = torch.empty(max(int(nbytes), 1) + 256, dtype=torch.uint8, device=device)
    p = buf.data_ptr()
    return buf, (p + 255) & ~255


# ---------------------------------------------------------------------------

@dataclass
class CSR:
    """Device CSR (int32 indptr/indices, float32 values) in torch tensors."""
    indptr: torch.Tensor
    indices: torch.Tensor
    values: torch.Tensor
    n_rows: int
    n_cols: int

    @property
    def nnz(self) -> int:
        return int(self.indices.numel())

    @classmethod
    def from_host(cls, m, device="cuda") -> "CSR":
        """From any object with numpy indptr/indices/values, n_rows, n_cols."""
        ip = torch.as_tensor(m.indptr).to(device=device, dtype=torch.int32).contiguous()
        ix = torch.as_tensor(m.indices).to(device=device, dtype=torch.int32).contiguous()
        v = torch.as_tensor(m.values).to(device=device, dtype=torch.float32).contiguous()
        return cls(ip, ix, v, int(m.n_rows), int(m.n_cols))

    def _c(self) -> _Csr:
        assert self.indptr.is_cuda and self.indices.is_cuda and self.values.is_cuda
        assert self.indptr.dtype == torch.int32 and self.indices.dtype == torch.int32
        assert self.values.dtype == torch.float32
        assert self.indptr.is_contiguous() and self.indices.is_contiguous() \
            and self.values.is_contiguous()
        assert self.indptr.numel() == self.n_rows + 1
        assert self.values.numel() == self.indices.numel()
        return _Csr(self.n_rows, self.n_cols, self.nnz, self.indptr.data_ptr(),
                    self.indices.data_ptr() if self.nnz else None,
                    self.values.data_ptr() if self.nnz else None)


@dataclass
class BSC:
    """Device Block-Sparse CSR (§3.2): the CSR's indptr and values, the per-row
    block-id varint bytes (located by bptr) and the packed 10-bit offsets."""
    indptr: torch.Tensor   # int32 [n_rows + 1]
    bptr: torch.Tensor     # int32 [n_rows + 1]
    blocks: torch.Tensor   # uint8 [bptr[-1]]
    offsets: torch.Tensor  # uint8, a multiple of 4 bytes
    values: torch.Tensor   # float32 [nnz]
    n_rows: int
    n_cols: int

    @property
    def nnz(self) -> int:
        return int(self.values.numel())

    def index_bytes(self) -> int:
        """Bytes that locate the entries: bptr, varints and offsets (indptr, as in
        the CSR, left out)."""
        return 4 * self.bptr.numel() + self.blocks.numel() + (10 * self.nnz + 7) // 8

    def _c(self) -> _Bsc:
        for t, dt in ((self.indptr, torch.int32), (self.bptr, torch.int32),
                      (self.blocks, torch.uint8), (self.offsets, torch.uint8),
                      (self.values, torch.float32)):
            assert t.is_cuda and t.dtype == dt and t.is_contiguous()
        return _Bsc(self.n_rows, self.n_cols, self.nnz, self.indptr.data_ptr(),
                    self.bptr.data_ptr(), self.blocks.data_ptr() if self.blocks.numel() else None,
                    self.blocks.numel(), self.offsets.data_ptr() if self.offsets.numel() else None,
                    self.offsets.numel(), self.values.data_ptr() if self.nnz else None)


def bsc_encode(m: CSR, stream=None) -> BSC:
    """Block-Sparse CSR of a canonical CSR (synchronises once, to size the varint
    stream; raises SpsError for a non-canonical CSR)."""
    load_library()
    dev = m.indptr.device
    c = m._c()
    bptr = torch.empty(m.n_rows + 1, dtype=torch.int32, device=dev)
    scratch = torch.empty(16, dtype=torch.int32, device=dev)
    nbytes = _I64()
    _check(_lib.sps_bsc_encode_sizes(ctypes.byref(c), bptr.data_ptr(), scratch.data_ptr(),
                                     _stream_ptr(stream), ctypes.byref(nbytes)))
    ob = _SZ()
    _check(_lib.sps_bsc_offsets_bytes(m.nnz, ctypes.byref(ob)))
    blocks = torch.empty(nbytes.value, dtype=torch.uint8, device=dev)
    offsets = torch.empty(ob.value, dtype=torch.uint8, device=dev)
    _check(_lib.sps_bsc_encode(ctypes.byref(c), bptr.data_ptr(),
                               blocks.data_ptr() if nbytes.value else None, nbytes.value,
                               offsets.data_ptr() if ob.value else None, ob.value,
                               _stream_ptr(stream)))
    return BSC(m.indptr, bptr, blocks, offsets, m.values, m.n_rows, m.n_cols)


def bsc_decode(b: BSC, stream=None, check: bool = True) -> CSR:
    """The CSR of a Block-Sparse CSR (its indptr and values shared). With check,
    synchronises and raises SpsError for a malformed encoding."""
    load_library()
    dev = b.indptr.device
    indices = torch.empty(b.nnz, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    c = b._c()
    _check(_lib.sps_bsc_decode(ctypes.byref(c), indices.data_ptr() if b.nnz else None,
                               status.data_ptr(), _stream_ptr(stream)))
    if check and int(status.item()) != 0:
        raise SpsError(-2, "malformed Block-Sparse CSR (status %d)" % int(status.item()))
    return CSR(b.indptr, indices, b.values, b.n_rows, b.n_cols)


class Items:
    """Prepared item corpus (owns its workspaces)."""

    def __init__(self, handle, persistent, scratch, src: CSR, chunk_size: int):
        self._h = handle
        self._persistent = persistent
        self._scratch = scratch
        self._src = src  # kept alive until release_inputs()
        n, d, z = _I64(), _I64(), _I64()
        cs, nc = _I32(), _I32()
        _check(_lib.sps_items_info(handle, ctypes.byref(n), ctypes.byref(d), ctypes.byref(z),
                                   ctypes.byref(cs), ctypes.byref(nc)))
        self.n_items, self.dim, self.nnz = n.value, d.value, z.value
        self.chunk_size, self.num_chunks = cs.value, nc.value
        ss, spc, ns = _I32(), _I32(), _I64()
        _check(_lib.sps_items_slices(handle, ctypes.byref(ss), ctypes.byref(spc), ctypes.byref(ns)))
        self.slice_size, self.slices_per_chunk, self.num_slices = ss.value, spc.value, ns.value

    def chunk_len(self, c: int) -> int:
        b = c * self.chunk_size
        return min(b + self.chunk_size, self.n_items) - b

    def enable_half(self, stream=None) -> None:
        """Build the fp16 postings used by cosine_chunk_half (once; needs the prepare work
        to have been enqueued on the same stream)."""
        if getattr(self, "_half", None) is not None:
            return
        n = _SZ()
        _check(_lib.sps_items_half_workspace_size(self._h, ctypes.byref(n)))
        buf, ptr = _workspace(n.value, self._persistent.device)
        _check(_lib.sps_items_enable_half(self._h, ptr, n.value, _stream_ptr(stream)))
        self._half = buf

    def release_inputs(self):
        """Drop the item CSR and prepare scratch (after the prepare work completed)."""
        torch.cuda.current_stream().synchronize()
        self._src = None
        self._scratch = None

    def slice_view(self, s: int, stream=None) -> dict:
        """Device views of slice s's inverted lists (synchronous)."""
        v = _SliceView()
        _check(_lib.sps_items_slice_view(self._h, s, _stream_ptr(stream), ctypes.byref(v)))
        dev = self._persistent.device

        def view(ptr, n, dtype, elem):
            if n == 0:
                return torch.empty(0, dtype=dtype, device=dev)
            base = self._persistent.data_ptr()
            off = ptr - base
            assert 0 <= off and off + n * elem <= self._persistent.numel()
            return self._persistent[off:off + n * elem].view(dtype)

        return {
            "item_begin": v.item_begin, "slice_len": v.slice_len, "slice_nnz": v.slice_nnz,
            # sps_posting records: int32 pairs (item id, value bits)
            "post": view(v.post, v.slice_nnz, torch.int32, 8).view(-1, 2),
            "item_inv_norm": view(v.item_inv_norm, v.slice_len, torch.float32, 4),
        }

    def slice_col_ptr(self, s: int, stream=None):
        """(col_ptr int32[dim+1], consistent: bool) of slice s, expanded from its dim index
        on the device (synchronous)."""
        dev = self._persistent.device
        cp = torch.empty(self.dim + 1, dtype=torch.int32, device=dev)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        _check(_lib.sps_items_slice_col_ptr(self._h, s, cp.data_ptr(), st.data_ptr(),
                                            _stream_ptr(stream)))
        (stream or torch.cuda.current_stream()).synchronize()
        return cp, int(st.item()) == 0

    def heavy_dims(self, stream=None) -> list:
        """The dims kept as dense rows (ascending; synchronous)."""
        buf = (_I32 * 128)()
        n = _I32()
        _check(_lib.sps_items_heavy_dims(self._h, _stream_ptr(stream), buf, 128, ctypes.byref(n)))
        return [int(buf[i]) for i in range(n.value)]

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.sps_items_destroy(h)


class Queries:
    """Prepared query batch (owns its workspace)."""

    def __init__(self, handle, ws, n_rows: int, items: Items):
        self._h = handle
        self._ws = ws
        self.n_rows = n_rows
        self.items = items
        p = _P()
        _check(_lib.sps_queries_inv_norms(handle, ctypes.byref(p)))
        off = p.value - ws.data_ptr()
        self.inv_norm = ws[off:off + 4 * n_rows].view(torch.float32) if n_rows else \
            torch.empty(0, dtype=torch.float32, device=ws.device)

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.sps_queries_destroy(h)


def items_workspace_size(n_items: int, dim: int, nnz: int, chunk_size: int) -> tuple[int, int]:
    load_library()
    p, s = _SZ(), _SZ()
    _check(_lib.sps_items_workspace_size(n_items, dim, nnz, chunk_size, ctypes.byref(p),
                                         ctypes.byref(s)))
    return p.value, s.value


def prepare(items, chunk_size: int = 8192, stream=None) -> Items:
    """Norms + per-chunk inverted lists of an item corpus (asynchronous). items is a
    CSR, or a BSC whose indices are decoded on the device first."""
    load_library()
    if isinstance(items, BSC):
        items = bsc_decode(items, stream)
    pb, sb = items_workspace_size(items.n_rows, items.n_cols, items.nnz, chunk_size)
    dev = items.indptr.device
    pbuf, pptr = _workspace(pb, dev)
    sbuf, sptr = _workspace(sb, dev)
    h = _P()
    c = items._c()
    _check(_lib.sps_prepare(ctypes.byref(c), chunk_size, pptr, pb, sptr, sb, _stream_ptr(stream),
                            ctypes.byref(h)))
    # the persistent view handed out by chunk_view is relative to the aligned base
    pview = pbuf[pptr - pbuf.data_ptr():]
    return Items(h.value, pview, sbuf, items, chunk_size)


def prepare_queries(queries: CSR, items: Items, stream=None) -> Queries:
    """Inverse norms and per-workgroup merged dim lists of a query batch (asynchronous)."""
    load_library()
    nb = _SZ()
    _check(_lib.sps_queries_workspace_size(items._h, queries.n_rows, queries.n_cols,
                                           queries.nnz, ctypes.byref(nb)))
    buf, ptr = _workspace(nb.value, queries.indptr.device)
    h = _P()
    c = queries._c()
    _check(_lib.sps_prepare_queries(ctypes.byref(c), items._h, ptr, nb.value, _stream_ptr(stream),
                                    ctypes.byref(h)))
    q = Queries(h.value, buf[ptr - buf.data_ptr():], queries.n_rows, items)
    q._src = queries
    return q


def _out_args(q: Queries, out: torch.Tensor, row_sums, dtype=torch.float32):
    assert out.is_cuda and out.dtype == dtype and out.dim() == 2
    assert out.stride(1) == 1 and out.shape[0] == q.n_rows
    ld = out.stride(0) if q.n_rows > 1 else out.shape[1]
    rs = None
    if row_sums is not None:
        assert row_sums.is_cuda and row_sums.dtype == torch.float64 and row_sums.is_contiguous()
        rs = row_sums.data_ptr()
    return ld, rs


def cosine_chunk(q: Queries, items: Items, chunk: int, out: torch.Tensor,
                 row_sums: torch.Tensor | None = None, stream=None) -> None:
    """out[:, :chunk_len] = S[:, chunk]; out is (n_query, >= chunk_len) float32, row-major."""
    ld, rs = _out_args(q, out, row_sums)
    assert out.shape[1] >= items.chunk_len(chunk)
    if row_sums is not None:
        assert row_sums.numel() >= q.n_rows
    _check(_lib.sps_cosine_chunk(q._h, items._h, chunk, out.data_ptr(), ld, rs,
                                 _stream_ptr(stream)))


def cosine_chunk_static(q: Queries, items: Items, chunk: int, out: torch.Tensor,
                        row_sums: torch.Tensor | None = None, stream=None) -> None:
    """cosine_chunk with the partial row sums in the library's static device scratch
    (no allocation; calls overlapping on one GPU race)."""
    ld, rs = _out_args(q, out, row_sums)
    assert out.shape[1] >= items.chunk_len(chunk)
    if row_sums is not None:
        assert row_sums.numel() >= q.n_rows
    _check(_lib.sps_cosine_chunk_static(q._h, items._h, chunk, out.data_ptr(), ld, rs,
                                        _stream_ptr(stream)))


def cosine_chunk_half(q: Queries, items: Items, chunk: int, out: torch.Tensor,
                      row_sums: torch.Tensor | None = None, stream=None) -> None:
    """The reduced-precision variant: out[:, :chunk_len] = fp16 scores from fp16 item
    values (|error| < 1e-3); out is (n_query, >= chunk_len) float16, row-major. Needs
    items.enable_half()."""
    ld, rs = _out_args(q, out, row_sums, torch.float16)
    assert out.shape[1] >= items.chunk_len(chunk)
    if row_sums is not None:
        assert row_sums.numel() >= q.n_rows
    _check(_lib.sps_cosine_chunk_half(q._h, items._h, chunk, out.data_ptr(), ld, rs,
                                      _stream_ptr(stream)))


def cosine_chunk_threshold(q: Queries, items: Items, chunk: int, threshold: float,
                           hits: torch.Tensor, count: torch.Tensor,
                           row_sums: torch.Tensor | None = None, stream=None) -> None:
    """Append every score >= threshold of the chunk to hits as (row, item, score bits) int32
    triples; count (one int64/uint64 device value, zeroed once by the caller) advances by the
    number of hits, including those past hits' capacity, which are dropped."""
    assert hits.is_cuda and hits.dtype == torch.int32 and hits.dim() == 2
    assert hits.shape[1] == 3 and hits.is_contiguous()
    assert count.is_cuda and count.dtype == torch.int64 and count.numel() >= 1
    rs = None
    if row_sums is not None:
        assert row_sums.is_cuda and row_sums.dtype == torch.float64 and row_sums.is_contiguous()
        assert row_sums.numel() >= q.n_rows
        rs = row_sums.data_ptr()
    _check(_lib.sps_cosine_chunk_threshold(q._h, items._h, chunk, float(threshold),
                                           hits.data_ptr() if hits.numel() else None,
                                           hits.shape[0], count.data_ptr(), rs,
                                           _stream_ptr(stream)))


def hits_to_numpy(hits: torch.Tensor, count: int):
    """(rows, items, scores) numpy arrays of the first min(count, capacity) hits."""
    h = hits[:min(int(count), hits.shape[0])].cpu().numpy()
    return h[:, 0].copy(), h[:, 1].copy(), h[:, 2].copy().view(np.float32)


def cosine_stream(q: Queries, items: Items, chunk_begin: int, chunk_end: int,
                  out: torch.Tensor, row_sums: torch.Tensor | None = None, stream=None) -> None:
    """Chunks [chunk_begin, chunk_end) in turn into the same rotating buffer `out`."""
    ld, rs = _out_args(q, out, row_sums)
    assert out.shape[1] >= min(items.chunk_size, items.n_items)
    if row_sums is not None:
        assert row_sums.numel() >= (chunk_end - chunk_begin) * q.n_rows
    _check(_lib.sps_cosine_stream(q._h, items._h, chunk_begin, chunk_end, out.data_ptr(), ld, rs,
                                  _stream_ptr(stream)))


_copy_streams: dict = {}


def _copy_stream(device) -> "torch.cuda.Stream":
    """One side stream per device for device-to-host copies (default priority)."""
    idx = torch.device(device).index
    idx = torch.cuda.current_device() if idx is None else idx
    if idx not in _copy_streams:
        _copy_streams[idx] = torch.cuda.Stream(device=idx)
    return _copy_streams[idx]


def cosine_stream_host(q: Queries, items: Items, chunk_begin: int, chunk_end: int,
                       host_out: torch.Tensor, bufs=None, row_sums: torch.Tensor | None = None,
                       stream=None, copy_stream=None) -> None:
    """Chunks [chunk_begin, chunk_end) into the pinned host matrix host_out
    (n_query x >= the range's items, float32, row-major), column 0 being item
    chunk_begin * chunk_size: scored into two alternating device buffers, each
    copied out by the copy engine on a side stream while the next is scored.
    Asynchronous in `stream` order: synchronise before reading host_out."""
    assert not host_out.is_cuda and host_out.is_pinned(), "host_out must be a pinned CPU tensor"
    assert host_out.dtype == torch.float32 and host_out.dim() == 2
    assert host_out.stride(1) == 1 and host_out.shape[0] == q.n_rows
    ld_host = host_out.stride(0) if q.n_rows > 1 else host_out.shape[1]
    if chunk_end > chunk_begin:
        span = min(chunk_end * items.chunk_size, items.n_items) - chunk_begin * items.chunk_size
        assert host_out.shape[1] >= span, "host_out narrower than the chunk range"
    s = stream if stream is not None else torch.cuda.current_stream()
    dev = s.device
    if bufs is None:
        width = max(min(items.chunk_size, items.n_items), 1)
        bufs = tuple(torch.empty(q.n_rows, width, dtype=torch.float32, device=dev)
                     for _ in range(2))
        for b in bufs:  # freed by the caller's stream order only after the copies
            b.record_stream(s)
    b0, b1 = bufs
    assert b0.is_cuda and b0.dtype == torch.float32 and b0.stride(1) == 1
    assert b1.shape == b0.shape and b1.stride() == b0.stride() and b1.dtype == b0.dtype
    assert b0.shape[0] == q.n_rows and b0.shape[1] >= min(items.chunk_size, items.n_items)
    ld_dev = b0.stride(0) if q.n_rows > 1 else b0.shape[1]
    rs = None
    if row_sums is not None:
        assert row_sums.is_cuda and row_sums.dtype == torch.float64 and row_sums.is_contiguous()
        assert row_sums.numel() >= (chunk_end - chunk_begin) * q.n_rows
        rs = row_sums.data_ptr()
    cs = copy_stream if copy_stream is not None else _copy_stream(dev)
    _check(_lib.sps_cosine_stream_host(q._h, items._h, chunk_begin, chunk_end,
                                       host_out.data_ptr(), ld_host, b0.data_ptr(),
                                       b1.data_ptr(), ld_dev, rs, int(s.cuda_stream),
                                       int(cs.cuda_stream)))


# ---------------------------------------------------------------------------
# rows of scores: selection

_SCORE_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _here(*tensors) -> int:
    """The current device's index; device tensors must be on it, since a launch goes to its
    streams."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None:
            assert t.is_cuda and t.get_device() == cur, \
                "tensors must be on the current device (torch.cuda.set_device)"
    return cur


def _parts(m) -> list:
    """The tensors of a CSR (or BSC)."""
    return [t for t in vars(m).values() if isinstance(t, torch.Tensor)]


# torch's own way to the current stream's handle, without a Stream object a call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device: int, stream) -> int:
    """The handle of `stream`, or of the device's current stream for None."""
    if stream is not None:
        return int(stream.cuda_stream)
    if _raw_stream is not None:
        return _raw_stream(device)
    return int(torch.cuda.current_stream(device).cuda_stream)


def _view(x: torch.Tensor, col_begin: int = 0) -> _Scores:
    """A 2-d tensor of scores (rows contiguous, any row stride) as a view of columns
    [col_begin, col_begin + x.shape[1])."""
    assert x.dim() == 2 and x.dtype in _SCORE_TYPES, \
        "scores must be (rows, columns) of float32, float16 or bfloat16"
    n, m = x.shape
    assert n == 0 or m <= 1 or x.stride(1) == 1, "rows must be contiguous"
    ld = x.stride(0) if n > 1 and m else m
    return _Scores(x.data_ptr() if n and m else None, _SCORE_TYPES[x.dtype], n, m, ld, col_begin)


def _rows_f32(t, n: int, what: str):
    """The address of a contiguous float32 vector of n values, None for None."""
    if t is None:
        return None
    assert t.dtype == torch.float32 and t.is_contiguous() and t.numel() == n, \
        "%s must be %d contiguous float32 values" % (what, n)
    return t.data_ptr()


def _on(stream):
    """Allocations inside belong to `stream` (the current one for None)."""
    return torch.cuda.stream(stream) if stream is not None else _NO_STREAM


class _NoStream:
    def __enter__(self):
        pass

    def __exit__(self, *a):
        pass


_NO_STREAM = _NoStream()


@functools.lru_cache(maxsize=256)
def _sized(name: str, *args) -> int:
    n = _SZ()
    _check(getattr(_lib, name)(*args, ctypes.byref(n)))
    return n.value


@dataclass
class TopRows:
    """The best k of every row, best first: scores float32 (n_rows, k) and columns int32
    (n_rows, k); -inf and -1 where a row has fewer candidates."""
    scores: torch.Tensor
    cols: torch.Tensor

    @property
    def k(self) -> int:
        return int(self.scores.shape[1])


@dataclass
class BeamStep:
    """The best k of each group of beams, best first: scores float32, the parents' rows
    int32 and the columns int32, each (groups, k); -inf, -1 and -1 in places that no
    candidate fills."""
    scores: torch.Tensor
    parents: torch.Tensor
    cols: torch.Tensor


def top_rows(n_rows: int, k: int, device="cuda") -> TopRows:
    """Room for the best k of n_rows rows (filled by select_chunk with first=True)."""
    return TopRows(torch.empty(n_rows, k, dtype=torch.float32, device=device),
                   torch.empty(n_rows, k, dtype=torch.int32, device=device))


def select_chunk(scores: torch.Tensor, top: TopRows, col_begin: int = 0,
                 offsets: torch.Tensor | None = None, first: bool = False, stream=None) -> None:
    """Join a chunk of columns (scores[:, j] being column col_begin + j) to the running
    best k of every row, by fl32(offsets[row] + score), ties to the lower column. NaN and
    -inf are no candidates. first=True starts the lists; chunks may come in any order."""
    load_library()
    dev = _here(scores, top.scores, top.cols, offsets)
    v = _view(scores, col_begin)
    n, k = v.n_rows, top.scores.shape[1]
    assert top.scores.shape == (n, k) and top.cols.shape == (n, k)
    assert top.scores.dtype == torch.float32 and top.cols.dtype == torch.int32
    assert top.scores.is_contiguous() and top.cols.is_contiguous()
    nb = _sized("sps_select_workspace_size", n, v.n_cols, k)
    with _on(stream):
        ws = torch.empty(nb, dtype=torch.uint8, device=scores.device) if nb else None
        _check(_lib.sps_select_chunk(ctypes.byref(v), _rows_f32(offsets, n, "offsets"), k,
                                     int(first), top.scores.data_ptr(), top.cols.data_ptr(),
                                     ws.data_ptr() if nb else None, nb, _stream_of(dev, stream)))


def _beam_step(groups: int, k: int, device) -> BeamStep:
    return BeamStep(torch.empty((groups, k), dtype=torch.float32, device=device),
                    torch.empty((groups, k), dtype=torch.int32, device=device),
                    torch.empty((groups, k), dtype=torch.int32, device=device))


def beam_select(scores: torch.Tensor, beam_scores: torch.Tensor | None, beams: int,
                k: int | None = None, col_begin: int = 0, stream=None) -> BeamStep:
    """One step of a beam search over whole rows: of each group of `beams` consecutive rows,
    the best k (default: beams) of (beam, column) by fl32(beam_scores[row] + score), ties to
    the lower row, then the lower column. A beam whose score is -inf takes no part."""
    load_library()
    dev = _here(scores, beam_scores)
    v = _view(scores, col_begin)
    k = beams if k is None else k
    assert beams >= 1 and v.n_rows % beams == 0, "rows must be groups of %d beams" % beams
    bs = _rows_f32(beam_scores, v.n_rows, "beam_scores")
    nb = _sized("sps_beam_workspace_size", v.n_rows, v.n_cols, beams, k)
    with _on(stream):
        out = _beam_step(v.n_rows // beams, k, scores.device)
        ws = torch.empty(nb, dtype=torch.uint8, device=scores.device) if nb else None
        _check(_lib.sps_beam_select(ctypes.byref(v), bs, beams, k, out.scores.data_ptr(),
                                    out.parents.data_ptr(), out.cols.data_ptr(),
                                    ws.data_ptr() if nb else None, nb, _stream_of(dev, stream)))
    return out


def beam_join(top: TopRows, beams: int, k: int | None = None, stream=None) -> BeamStep:
    """beam_select's step from the running lists that select_chunk kept over chunks of
    columns with the beams' scores as its offsets (equal to it where top.k >= k)."""
    load_library()
    dev = _here(top.scores, top.cols)
    n, k_in = top.scores.shape
    assert top.cols.shape == (n, k_in)
    assert top.scores.dtype == torch.float32 and top.cols.dtype == torch.int32
    assert top.scores.is_contiguous() and top.cols.is_contiguous()
    assert beams >= 1 and n % beams == 0, "rows must be groups of %d beams" % beams
    k = beams if k is None else k
    with _on(stream):
        out = _beam_step(n // beams, k, top.scores.device)
        _check(_lib.sps_beam_join(top.scores.data_ptr(), top.cols.data_ptr(), n, k_in, beams, k,
                                  out.scores.data_ptr(), out.parents.data_ptr(),
                                  out.cols.data_ptr(), _stream_of(dev, stream)))
    return out


def reorder_states(states, parents: torch.Tensor, outs=None, stream=None) -> list:
    """States follow their parents: out[j] = state[parents[j]] for every tensor of `states`
    (first dimension the beams' rows, each row contiguous, any types), zeros where parents[j]
    is no row. parents: int32, any shape (BeamStep.parents). Returns the outs (allocated if
    not given; they may share no byte with a state, the parents or each other, but lie
    beside them in one buffer: t[:, 1] for t[:, 0])."""
    load_library()
    states = list(states)
    dev = _here(parents, *states)
    assert parents.dtype == torch.int32 and parents.is_contiguous()
    n = parents.numel()
    rows = states[0].shape[0] if states else 0
    with _on(stream):
        if outs is None:
            outs = [t.new_empty((n,) + t.shape[1:]) for t in states]
        else:
            outs = list(outs)
            _here(*outs)
        assert len(outs) == len(states)
        args = []
        for t, o in zip(states, outs):
            assert t.shape[0] == rows, "states must have the same rows"
            assert o.dtype == t.dtype and o.shape[0] == n and o.shape[1:] == t.shape[1:]
            size = t.element_size()
            width = t.numel() // rows * size if rows else o.numel() // n * size if n else 0
            for x in (t, o):  # a row is one run of bytes
                assert x.is_contiguous() or x[:1].is_contiguous(), "rows must be contiguous"
            args += (t.data_ptr(), o.data_ptr(), width, t.stride(0) * size if rows > 1 else width,
                     o.stride(0) * size if n > 1 else width)
        # sps_state is five 8-byte words: the two addresses and the three sizes
        _check(_lib.sps_reorder_states((_I64 * len(args))(*args), len(states), parents.data_ptr(), n,
                                       rows, _stream_of(dev, stream)))
    return outs


def bulk_select(queries: CSR, items: CSR, k: int, chunk_size: int = 8192) -> TopRows:
    """The best k items of every query, of all of them (exact): every chunk scored and
    joined to the running lists. The score matrix is never kept; bulk_similarity's loop."""
    _here(*_parts(queries), *_parts(items))
    it = prepare(items, chunk_size)
    q = prepare_queries(queries, it)
    dev = queries.indptr.device
    top = top_rows(queries.n_rows, k, dev)
    buf = torch.empty(queries.n_rows, min(chunk_size, it.n_items), dtype=torch.float32, device=dev)
    if it.num_chunks == 0:
        select_chunk(buf, top, 0, first=True)
    for c in range(it.num_chunks):
        cosine_chunk(q, it, c, buf)
        select_chunk(buf[:, :it.chunk_len(c)], top, c * chunk_size, first=c == 0)
    return top


# ---------------------------------------------------------------------------
# rows of scores: distillation

class Distill:
    """A batch's teacher lists and the running statistics of its rows (owns its workspace)."""

    def __init__(self, handle, ws, n_rows: int, n_cols: int, device):
        self._h = handle
        self._ws = ws
        self.n_rows, self.n_cols, self.device = n_rows, n_cols, device

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h and _lib is not None:
            _lib.sps_distill_destroy(h)


def _teacher(ids: torch.Tensor, logits: torch.Tensor, teacher_lse):
    assert ids.dim() == 2 and ids.dtype == torch.int32 and ids.is_contiguous(), \
        "teacher ids must be contiguous int32 (rows, k)"
    assert logits.shape == ids.shape and logits.dtype == torch.float32 and logits.is_contiguous(), \
        "teacher logits must be contiguous float32 (rows, k)"
    n, k = ids.shape
    return n, k, _rows_f32(teacher_lse, n, "teacher_lse")


def distill_prepare(teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, n_cols: int,
                    temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
                    stream=None) -> Distill:
    """The teacher's best k of every row, for rows of n_cols scores that come in chunks:
    distill_chunk for every chunk, distill_loss, distill_chunk_grad for every chunk. ids
    outside [0, n_cols) (pad with -1), an id's repetitions in its row and logits of -inf take
    no part. With teacher_lse (the teacher's log-sum-exp of logits / temperature over all
    columns) its mass outside the list is one more class; without, the list's is all (a list
    of every column that has a score goes without: what rounding leaves of 1 would have no
    column to go to, an infinite loss). The temperature is used as the nearest float32."""
    load_library()
    cur = _here(teacher_ids, teacher_logits, teacher_lse)
    n, k, lse = _teacher(teacher_ids, teacher_logits, teacher_lse)
    nb = _sized("sps_distill_workspace_size", n, k)
    dev = teacher_ids.device
    with _on(stream):
        buf, ptr = _workspace(nb, dev)
        h = _P()
        _check(_lib.sps_distill_prepare(teacher_ids.data_ptr(), teacher_logits.data_ptr(), lse, n, k,
                                        n_cols, float(temperature), ptr, nb,
                                        _stream_of(cur, stream),
                                        ctypes.byref(h)))
    return Distill(h.value, buf, n, n_cols, dev)


def distill_chunk(d: Distill, scores: torch.Tensor, col_begin: int = 0, first: bool = False,
                  stream=None) -> None:
    """Take in the student's scores of columns [col_begin, col_begin + scores.shape[1]); every
    column once, in any order of the chunks. first=True forgets what came before."""
    dev = _here(scores, d._ws)
    v = _view(scores, col_begin)
    _check(_lib.sps_distill_chunk(d._h, ctypes.byref(v), int(first), _stream_of(dev, stream)))


def distill_loss(d: Distill, return_lse: bool = False, stream=None):
    """The loss of every row, float32 (n_rows,), once all chunks are in; with return_lse also
    the student's log-sum-exp of scores / temperature."""
    with _on(stream):
        loss = torch.empty(d.n_rows, dtype=torch.float32, device=d.device)
        lse = torch.empty_like(loss) if return_lse else None
        _check(_lib.sps_distill_loss(d._h, loss.data_ptr(), lse.data_ptr() if return_lse else None,
                                     _stream_of(_here(loss), stream)))
    return (loss, lse) if return_lse else loss


def _grad_out(scores: torch.Tensor, out):
    if out is None:
        out = torch.empty(scores.shape, dtype=scores.dtype, device=scores.device)
    assert out.shape == scores.shape and (out.stride(1) == 1 or out.shape[1] <= 1)
    assert out.dtype in (scores.dtype, torch.float32), "gradients have the scores' type or float32"
    return out, out.stride(0) if out.shape[0] > 1 else out.shape[1]


def distill_chunk_grad(d: Distill, scores: torch.Tensor, col_begin: int = 0,
                       row_weights: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """row_weights[r] * d loss_r / d scores[r, j] of a chunk, after distill_loss of the same
    scores. out: of the scores' type or float32, may be `scores` itself."""
    dev = _here(scores, row_weights, out, d._ws)
    v = _view(scores, col_begin)
    w = _rows_f32(row_weights, v.n_rows, "row_weights")
    with _on(stream):
        out, ld = _grad_out(scores, out)
        _check(_lib.sps_distill_chunk_grad(d._h, ctypes.byref(v), w, out.data_ptr(),
                                           _SCORE_TYPES[out.dtype], ld, _stream_of(dev, stream)))
    return out


def distill(scores: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
            temperature: float = 1.0, teacher_lse: torch.Tensor | None = None,
            row_weights: torch.Tensor | None = None, out: torch.Tensor | None = None,
            need_grad: bool = True, stream=None):
    """(loss of every row, gradient about the scores) of whole rows against the teacher's best
    k (distill_prepare says which entries count); the gradient is None without need_grad."""
    load_library()
    dev = _here(scores, teacher_ids, teacher_logits, teacher_lse, row_weights, out)
    v = _view(scores)
    n, k, lse = _teacher(teacher_ids, teacher_logits, teacher_lse)
    assert n == v.n_rows, "one list a row"
    w = _rows_f32(row_weights, n, "row_weights")
    nb = _sized("sps_distill_rows_workspace_size", n, v.n_cols, k)
    with _on(stream):
        loss = torch.empty(n, dtype=torch.float32, device=scores.device)
        ld = 0
        if need_grad:
            out, ld = _grad_out(scores, out)
        buf, ptr = _workspace(nb, scores.device)
        _check(_lib.sps_distill_rows(ctypes.byref(v), teacher_ids.data_ptr(),
                                     teacher_logits.data_ptr(), lse, k, float(temperature), w,
                                     loss.data_ptr(), out.data_ptr() if need_grad else None,
                                     _SCORE_TYPES[out.dtype] if need_grad else 0, ld, ptr, nb,
                                     _stream_of(dev, stream)))
    return loss, out if need_grad else None


# ---------------------------------------------------------------------------
# the gradient of the scores

def cosine_chunk_grad(rows: CSR, other: Items, chunk: int, grad: torch.Tensor, du: torch.Tensor,
                      transposed: bool = False, first: bool = False, stream=None) -> None:
    """du[e] (+)= the gradient about the unit values of the rows of a CSR from chunk `chunk`
    of the other side, `grad` being that of the scores: (rows, chunk's items), or with
    transposed (chunk's items, rows). For the items' gradient, `rows` are items and `other`
    the queries prepared as a corpus. first=True starts the sums; cosine_grad_values ends
    them."""
    load_library()
    dev = _here(*_parts(rows), other._persistent, grad, du)
    assert du.dtype == torch.float32 and du.is_contiguous() and du.numel() == rows.nnz
    v = _view(grad)
    c = rows._c()
    nb = _SZ()
    _check(_lib.sps_cosine_grad_workspace_size(rows.nnz, other._h, ctypes.byref(nb)))
    with _on(stream):
        ws = torch.empty(nb.value, dtype=torch.uint8, device=grad.device) if nb.value else None
        _check(_lib.sps_cosine_grad(ctypes.byref(c), other._h, chunk, ctypes.byref(v),
                                    int(transposed), int(first), du.data_ptr(),
                                    ws.data_ptr() if nb.value else None, nb.value,
                                    _stream_of(dev, stream)))


def cosine_grad_values(rows: CSR, du: torch.Tensor, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """The gradient about the stored values from that about the unit values (the norm's
    part taken off); out may be du itself."""
    load_library()
    dev = _here(*_parts(rows), du, out)
    assert du.dtype == torch.float32 and du.is_contiguous() and du.numel() == rows.nnz
    with _on(stream):
        if out is None:
            out = torch.empty_like(du)
        assert out.dtype == torch.float32 and out.is_contiguous() and out.numel() == rows.nnz
        c = rows._c()
        _check(_lib.sps_cosine_grad_values(ctypes.byref(c), du.data_ptr(), out.data_ptr(),
                                           _stream_of(dev, stream)))
    return out


def cosine_grad(queries: CSR, items: CSR, grad: torch.Tensor, stream=None):
    """(gradient of the queries' values, gradient of the items' values), float32 (nnz,) each,
    from the gradient of their whole score matrix (n_query, n_item): float32, float16 or
    bfloat16. The stored structure of both is fixed. Nothing is prepared: a training step's
    batch has new values each time. Nothing is checked on the device either: the gradients of
    a CSR that is not canonical are undefined."""
    load_library()
    dev = _here(*_parts(queries), *_parts(items), grad)
    v = _view(grad)
    q, i = queries._c(), items._c()
    nb = _sized("sps_cosine_grad_both_workspace_size", q.nnz, i.nnz)
    with _on(stream):
        gq = torch.empty(q.nnz, dtype=torch.float32, device=grad.device)
        gi = torch.empty(i.nnz, dtype=torch.float32, device=grad.device)
        buf, ptr = _workspace(nb, grad.device)
        _check(_lib.sps_cosine_grad_both(ctypes.byref(q), ctypes.byref(i), ctypes.byref(v),
                                         gq.data_ptr(), gi.data_ptr(), ptr, nb,
                                         _stream_of(dev, stream)))
    return gq, gi


def bulk_distill(queries: CSR, items: CSR, teacher_ids: torch.Tensor,
                 teacher_logits: torch.Tensor, temperature: float = 1.0,
                 teacher_lse: torch.Tensor | None = None,
                 row_weights: torch.Tensor | None = None, chunk_size: int = 8192):
    """One step of distilling sparse embeddings over a whole corpus: (loss of every query,
    gradient of the queries' values, gradient of the items' values) of the softmax over all
    cosines / temperature against the teacher's best k of every query (bulk_select's lists of
    another scorer, say). bulk_similarity's loop, twice: once for the sums, once for the
    gradients, with one chunk of scores kept."""
    _here(*_parts(queries), *_parts(items), teacher_ids, teacher_logits, teacher_lse, row_weights)
    it = prepare(items, chunk_size)
    q = prepare_queries(queries, it)
    qt = prepare(queries, max(min(chunk_size, queries.n_rows), 1))
    dev = queries.indptr.device
    d = distill_prepare(teacher_ids, teacher_logits, it.n_items, temperature, teacher_lse)
    buf = torch.empty(queries.n_rows, min(chunk_size, it.n_items), dtype=torch.float32, device=dev)
    gq = torch.zeros(queries.nnz, dtype=torch.float32, device=dev)
    gi = torch.zeros(items.nnz, dtype=torch.float32, device=dev)
    if it.num_chunks == 0:
        distill_chunk(d, buf, 0, first=True)
    for c in range(it.num_chunks):
        cosine_chunk(q, it, c, buf)
        distill_chunk(d, buf[:, :it.chunk_len(c)], c * chunk_size, first=c == 0)
    loss = distill_loss(d)
    # entries of each chunk of items: one copy to the host
    begins = list(range(0, it.n_items, chunk_size)) + [it.n_items]
    cuts = items.indptr[torch.tensor(begins, device=dev)].tolist()
    for c in range(it.num_chunks):
        cosine_chunk(q, it, c, buf)
        g = buf[:, :it.chunk_len(c)]
        distill_chunk_grad(d, g, c * chunk_size, row_weights, out=g)
        cosine_chunk_grad(queries, it, c, g, gq, first=c == 0)
        lo, hi = cuts[c], cuts[c + 1]
        part = CSR(items.indptr[begins[c]:begins[c + 1] + 1] - lo, items.indices[lo:hi],
                   items.values[lo:hi], it.chunk_len(c), items.n_cols)
        for j in range(qt.num_chunks):
            b = j * qt.chunk_size
            cosine_chunk_grad(part, qt, j, g[b:b + qt.chunk_len(j)], gi[lo:hi], transposed=True,
                              first=j == 0)
    return loss, cosine_grad_values(queries, gq, gq), cosine_grad_values(items, gi, gi)


# ---------------------------------------------------------------------------
# dense rows

@dataclass
class Int8Rows:
    """Dense rows in 8 bits: row r stands for values[r, :dim] * scales[r]. values: int8
    (n_rows, ld), rows on 16-byte boundaries with zeros from dim to the next multiple of 16;
    scales: float32 (n_rows,). quantize_rows makes them so; rows[a:b] is a part of the rows."""
    values: torch.Tensor
    scales: torch.Tensor
    dim: int

    @property
    def n_rows(self) -> int:
        return int(self.values.shape[0])

    def __getitem__(self, part: slice) -> "Int8Rows":
        return Int8Rows(self.values[part], self.scales[part], self.dim)

    def _c(self) -> _Int8Rows:
        v, s = self.values, self.scales
        assert v.dim() == 2 and v.dtype == torch.int8, "values must be int8 (rows, ld)"
        n, m = v.shape
        assert m <= 1 or v.stride(1) == 1, "rows must be contiguous"
        # a row's chunks of 16 bytes belong to it, the last one whole
        assert m >= (self.dim + 15) // 16 * 16, "values must hold whole 16-byte chunks of a row"
        return _Int8Rows(v.data_ptr() if n else None, _rows_f32(s, n, "scales") if n else None, n,
                         self.dim, v.stride(0) if n > 1 else (m + 15) // 16 * 16)


def quantize_rows(x: torch.Tensor, stream=None) -> Int8Rows:
    """Dense rows (n, dim) of float32, float16 or bfloat16 in 8 bits, a scale a row: the scale
    is the largest magnitude / 127, the integers the nearest of x / scale, ties to even. A row
    that holds NaN or an infinity has scale NaN."""
    load_library()
    dev = _here(x)
    v = _view(x)
    n, dim = v.n_rows, v.n_cols
    ld = (dim + 15) // 16 * 16
    with _on(stream):
        values = torch.empty((n, ld), dtype=torch.int8, device=x.device)
        scales = torch.empty(n, dtype=torch.float32, device=x.device)
        _check(_lib.sps_quantize_rows(ctypes.byref(v), values.data_ptr() if n else None, ld,
                                      scales.data_ptr() if n else None, _stream_of(dev, stream)))
    return Int8Rows(values, scales, dim)


def dequantize_rows(rows: Int8Rows, dtype: torch.dtype = torch.float32,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values (n, dim) that 8-bit rows stand for, in dtype (or out's type)."""
    load_library()
    dev = _here(rows.values, rows.scales, out)
    c = rows._c()
    with _on(stream):
        if out is None:
            out = torch.empty((rows.n_rows, rows.dim), dtype=dtype, device=rows.values.device)
        assert out.shape == (rows.n_rows, rows.dim)
        o = _view(out)
        _check(_lib.sps_dequantize_rows(ctypes.byref(c), o.data, o.dtype, o.ld,
                                        _stream_of(dev, stream)))
    return out


def int8_scores(queries: Int8Rows, items: Int8Rows, out: torch.Tensor | None = None,
                dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """The products of 8-bit rows, scaled: (n_query, n_item) scores of dtype (or of out's type).
    items[a:b] scores a chunk of the items. Without out, rows of more than 512 scores are a view
    of a buffer whose rows start on 128-byte lines, which is written a third faster."""
    load_library()
    dev = _here(queries.values, queries.scales, items.values, items.scales, out)
    q, i = queries._c(), items._c()
    with _on(stream):
        if out is None:
            m = i.n_rows
            line = 128 // dtype.itemsize if m > 512 and q.n_rows > 1 else 1
            out = torch.empty((q.n_rows, (m + line - 1) // line * line), dtype=dtype,
                              device=queries.values.device)[:, :m]
        assert out.shape == (q.n_rows, i.n_rows)
        o = _view(out)
        _check(_lib.sps_int8_scores(ctypes.byref(q), ctypes.byref(i), o.data, o.dtype, o.ld,
                                    _stream_of(dev, stream)))
    return out


def int8_select(queries: Int8Rows, items: Int8Rows, k: int, chunk_size: int = 65536) -> TopRows:
    """The best k items of every query by their 8-bit rows' scores, exact, ties to the lower
    item: every chunk scored and joined to the running lists (bulk_select's loop). Queries go
    in batches, so that a chunk's scores stay within 2 GiB. A chunk is two calls: for few
    queries a chunk_size of all the items is the fastest (one query, 2M items of 768 dims: 744
    us in chunks of 65,536, 334 in one)."""
    _here(queries.values, queries.scales, items.values, items.scales)
    n, m = queries.n_rows, items.n_rows
    dev = queries.values.device
    top = top_rows(n, k, dev)
    width = min(chunk_size, m)
    batch = max(1, min(n, (1 << 29) // max(width, 1)))
    buf = torch.empty(batch, width, dtype=torch.float32, device=dev)
    for a in range(0, n, batch):
        part = TopRows(top.scores[a:a + batch], top.cols[a:a + batch])
        q = queries[a:a + batch]
        if m == 0:
            select_chunk(buf[:q.n_rows], part, 0, first=True)
        for b in range(0, m, chunk_size):
            chunk = items[b:b + chunk_size]
            scores = int8_scores(q, chunk, buf[:q.n_rows, :chunk.n_rows])
            select_chunk(scores, part, b, first=b == 0)
    return top


def dense_cross_entropy(queries: torch.Tensor, items: torch.Tensor, targets: torch.Tensor,
                        temperature: float = 1.0, bias: torch.Tensor | None = None,
                        row_weights: torch.Tensor | None = None, need_grad=True,
                        grad_dtype: torch.dtype | None = None, stream=None):
    """(loss of every query, gradient of the queries, gradient of the items): softmax cross
    entropy of z = queries . items / temperature + bias over all items, without the logits.
    queries (n, dim) and items (m, dim): rows of one type, float32, float16 or bfloat16;
    targets: int32 (n,), outside [0, m) a row takes no part; bias: float32 (m,), a constant,
    -inf strikes an item out; row_weights: float32 (n,), the gradient about each loss.
    need_grad: True, False, "queries" or "items" (the other is None); gradients have the rows'
    type or grad_dtype=torch.float32."""
    load_library()
    dev = _here(queries, items, targets, bias, row_weights)
    q, i = _view(queries), _view(items)
    n, m, dim = q.n_rows, i.n_rows, q.n_cols
    assert items.dtype == queries.dtype, "queries and items must have one type"
    assert targets.dtype == torch.int32 and targets.is_contiguous() and targets.numel() == n, \
        "targets must be %d contiguous int32" % n
    assert need_grad in (True, False, "queries", "items"), "need_grad: True, False, queries or items"
    bp = _rows_f32(bias, m, "bias")
    w = _rows_f32(row_weights, n, "row_weights")
    gt = queries.dtype if grad_dtype is None else grad_dtype
    assert gt in (queries.dtype, torch.float32), "gradients have the rows' type or float32"
    want_q, want_i = need_grad in (True, "queries"), need_grad in (True, "items")
    nb = _SZ()
    _check(_lib.sps_dense_ce_workspace_size(ctypes.byref(q), ctypes.byref(i), int(want_q),
                                            int(want_i), ctypes.byref(nb)))
    with _on(stream):
        loss = torch.empty(n, dtype=torch.float32, device=queries.device)
        gq = torch.empty((n, dim), dtype=gt, device=queries.device) if want_q else None
        gi = torch.empty((m, dim), dtype=gt, device=queries.device) if want_i else None
        buf, ptr = _workspace(nb.value, queries.device)
        _check(_lib.sps_dense_ce(ctypes.byref(q), ctypes.byref(i), targets.data_ptr(), bp,
                                 float(temperature), w, loss.data_ptr(),
                                 gq.data_ptr() if want_q and n else None, dim,
                                 gi.data_ptr() if want_i and m else None, dim, _SCORE_TYPES[gt],
                                 ptr, nb.value, _stream_of(dev, stream)))
    return loss, gq, gi


def row_inv_norms(m: CSR, stream=None) -> torch.Tensor:
    load_library()
    out = torch.empty(m.n_rows, dtype=torch.float32, device=m.indptr.device)
    c = m._c()
    _check(_lib.sps_row_inv_norms(ctypes.byref(c), out.data_ptr() if m.n_rows else None,
                                  _stream_ptr(stream)))
    return out


def validate_csr(m: CSR, stream=None) -> tuple[bool, int, int]:
    """(ok, first_bad_row, reason); reason 1 indptr, 2 order/dup, 3 range, 4 non-finite."""
    load_library()
    scratch = torch.empty(64, dtype=torch.uint8, device=m.indptr.device)
    row, why = _I64(), _I32()
    c = m._c()
    st = _lib.sps_validate_csr(ctypes.byref(c), scratch.data_ptr(), _stream_ptr(stream),
                               ctypes.byref(row), ctypes.byref(why))
    if st == -2:
        return False, row.value, why.value
    _check(st)
    return True, -1, 0


def bulk_similarity(queries: CSR, items: CSR, chunk_size: int = 8192, out=None,
                    on_chunk=None, row_sums: bool = False):
    """Full (n_query, n_item) float32 cosine matrix, item chunk by item chunk.

    Mirrors the streaming loop of §4.4 with every step on the GPU. With
    ``out`` (a device or pinned host tensor of shape (n_query, n_item)) each
    chunk is copied there; with ``on_chunk(c, buf, sums)`` each chunk's
    device buffer is handed to the callback instead (and reused after it
    returns). Returns ``out`` (allocated on the device if neither is given).
    """
    it = prepare(items, chunk_size)
    q = prepare_queries(queries, it)
    dev = queries.indptr.device
    if out is not None and on_chunk is None and not out.is_cuda and out.is_pinned():
        # pinned host output: double-buffered, the copies overlapping the scoring
        cosine_stream_host(q, it, 0, it.num_chunks, out)
        torch.cuda.current_stream().synchronize()
        return out
    width = min(chunk_size, it.n_items)
    buf = torch.empty(queries.n_rows, max(width, 1), dtype=torch.float32, device=dev)
    sums = torch.empty(queries.n_rows, dtype=torch.float64, device=dev) if row_sums else None
    if out is None and on_chunk is None:
        out = torch.empty(queries.n_rows, it.n_items, dtype=torch.float32, device=dev)
    for c in range(it.num_chunks):
        cosine_chunk(q, it, c, buf, sums)
        n = it.chunk_len(c)
        b = c * chunk_size
        if on_chunk is not None:
            on_chunk(c, buf[:, :n], sums)
        if out is not None:
            out[:, b:b + n].copy_(buf[:, :n], non_blocking=False)
    return out
