"""B200 (sm_100a) SPECTRA outlier-split INT4 decode matvec.

Thin Python binding of the C ABI in ``include/spectra.h``: argument
marshalling only.  Every step of the path (kurtosis, split, quantisation,
packing, fused dequantise+matvec) runs in the library's CUDA kernels; PyTorch
provides device memory and streams.  There is no CPU fallback: importing
the binding loads ``libspectra.so`` on first use and raises ImportError when
it is missing.

Method: "SPECTRA: Sparse-Precision Exact Channel Tensor Reconstruction
Architecture" (Dev.to abstract re-post), abstract paragraph.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import KV, Layer, PagedQuery, Sizes, TrdcLayer

__all__ = ["SpectraError", "PackedLayer", "spectra_status_string", "spectra_version",
           "spectra_packed_sizes", "spectra_packed_sizes_compact", "spectra_pack_plan",
           "spectra_pack", "spectra_pack_compact", "spectra_unpack",
           "spectra_gemv", "spectra_gemm_small", "spectra_gemv_batched", "spectra_embed",
           "spectra_device_status",
           "pack_layer", "library", "spectra_crc32", "write_container", "Container", "KVCache",
           "spectra_attention_decode", "KVPool", "spectra_attention_paged", "spectra_kv_evict",
           "spectra_sample"]

class _Lazy:
    """Loads libspectra.so on first attribute access."""

    def __getattr__(self, name):
        return getattr(_lib.load(), name)


_L = _Lazy()


def library() -> ctypes.CDLL:
    return _lib.load()


class SpectraError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        msg = _L.spectra_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})" if where else msg)
        self.status = status


def _check(status: int, where: str):
    if status != _lib.OK:
        raise SpectraError(status, where)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def spectra_status_string(status: int) -> str:
    return _L.spectra_status_string(status).decode()


def spectra_version() -> int:
    return _L.spectra_version()


def spectra_device_status(*, stream=None) -> None:
    """Raise SpectraError if a bounded wait in a matvec kernel gave up."""
    _check(_L.spectra_device_status(_stream(stream)), "spectra_device_status")


def spectra_selftest_wait(kind: int = 0, *, stream=None) -> None:
    """Launch a kernel whose bounded wait can never be satisfied; the next
    spectra_device_status reports SPECTRA_ERR_INTERNAL."""
    _check(_L.spectra_selftest_wait(int(kind), _stream(stream)), "spectra_selftest_wait")


def _sizes(s: Sizes) -> dict:
    return {"n_pad": s.n_pad, "codes": s.codes_bytes, "scales": s.scales_bytes,
            "zeros": s.zeros_bytes, "outlier_idx": s.outlier_idx_bytes,
            "outlier_w": s.outlier_w_bytes, "k_bulk": s.k_bulk, "bulk_idx": s.bulk_idx_bytes}


def spectra_packed_sizes(n: int, k: int, n_outliers: int) -> dict:
    s = Sizes()
    _check(_L.spectra_packed_sizes(n, k, n_outliers, ctypes.byref(s)), "spectra_packed_sizes")
    return _sizes(s)


def spectra_packed_sizes_compact(n: int, k: int, n_outliers: int) -> dict:
    s = Sizes()
    _check(_L.spectra_packed_sizes_compact(n, k, n_outliers, ctypes.byref(s)),
           "spectra_packed_sizes_compact")
    return _sizes(s)


def spectra_pack_plan(w: torch.Tensor, gain: torch.Tensor | None, tau: float, *,
                      want_kappa: bool = False, stream=None):
    """Kurtosis split.  Returns (idx int32 [n_o], kappa float64 [k] or None)."""
    n, k = w.shape
    dev = w.device
    kappa = torch.empty(k, dtype=torch.float64, device=dev) if want_kappa else None
    idx = torch.empty(max(k, 1), dtype=torch.int32, device=dev)
    ws_bytes = _L.spectra_pack_plan_workspace_size(k)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    n_o = ctypes.c_int32(0)
    _check(_L.spectra_pack_plan(_ptr(w), _ptr(gain), n, k, float(tau), _ptr(kappa), _ptr(idx),
                                ctypes.byref(n_o), _ptr(ws), ws_bytes, _stream(stream)),
           "spectra_pack_plan")
    return idx[: n_o.value], kappa


@dataclass
class PackedLayer:
    """Device buffers of one packed layer plus the C view over them."""
    n: int
    k: int
    n_outliers: int
    codes: torch.Tensor        # uint8
    scales: torch.Tensor       # int16 storage of FP16 bits
    zeros: torch.Tensor        # int32 storage of u32 words
    outlier_idx: torch.Tensor  # int32
    outlier_w: torch.Tensor    # int16 storage of BF16 bits
    bulk_idx: torch.Tensor | None = None  # int32 [k_bulk]: compacted bulk only
    k_bulk: int = 0                       # bulk columns (k when masked)

    def __post_init__(self):
        if self.k_bulk == 0:
            self.k_bulk = self.k

    @property
    def compact(self) -> bool:
        return self.bulk_idx is not None

    def view(self) -> Layer:
        return Layer(self.n, self.k, self.n_outliers, _ptr(self.codes), _ptr(self.scales),
                     _ptr(self.zeros), _ptr(self.outlier_idx) if self.n_outliers else None,
                     _ptr(self.outlier_w) if self.n_outliers else None,
                     self.k_bulk, _ptr(self.bulk_idx))

    @property
    def nbytes(self) -> int:
        """Bytes a matvec streams from these buffers (codes, scales, zeros,
        outlier weights and indices, and the bulk column list)."""
        return (self.codes.numel() + 2 * self.scales.numel() + 4 * self.zeros.numel()
                + 4 * self.n_outliers + 2 * self.outlier_w.numel()
                + (4 * self.bulk_idx.numel() if self.compact else 0))


def _alloc(nbytes: int, dtype, dev):
    item = torch.empty((), dtype=dtype).element_size()
    return torch.zeros(max(nbytes // item, 1), dtype=dtype, device=dev)


def spectra_pack(w: torch.Tensor, idx: torch.Tensor, *, stream=None) -> PackedLayer:
    """Quantise and pack W given the outlier indices from spectra_pack_plan."""
    n, k = w.shape
    n_o = int(idx.numel())
    dev = w.device
    sz = spectra_packed_sizes(n, k, n_o)
    codes = _alloc(sz["codes"], torch.uint8, dev)
    scales = _alloc(sz["scales"], torch.int16, dev)
    zeros = _alloc(sz["zeros"], torch.int32, dev)
    outw = _alloc(sz["outlier_w"], torch.int16, dev)
    idx_c = idx.contiguous() if n_o else torch.zeros(1, dtype=torch.int32, device=dev)
    ws_bytes = _L.spectra_pack_workspace_size()
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    view = Layer()
    _check(_L.spectra_pack(_ptr(w), n, k, _ptr(idx_c) if n_o else None, n_o, _ptr(codes),
                           _ptr(scales), _ptr(zeros), _ptr(outw) if n_o else None, _ptr(ws),
                           ws_bytes, ctypes.byref(view), _stream(stream)), "spectra_pack")
    return PackedLayer(n, k, n_o, codes, scales, zeros, idx_c, outw)


def spectra_pack_compact(w: torch.Tensor, idx: torch.Tensor, *, stream=None) -> PackedLayer:
    """Quantise and pack W with the outlier columns removed from the bulk."""
    n, k = w.shape
    n_o = int(idx.numel())
    dev = w.device
    sz = spectra_packed_sizes_compact(n, k, n_o)
    codes = _alloc(sz["codes"], torch.uint8, dev)
    scales = _alloc(sz["scales"], torch.int16, dev)
    zeros = _alloc(sz["zeros"], torch.int32, dev)
    outw = _alloc(sz["outlier_w"], torch.int16, dev)
    bidx = torch.empty(sz["k_bulk"], dtype=torch.int32, device=dev)
    idx_c = idx.contiguous() if n_o else torch.zeros(1, dtype=torch.int32, device=dev)
    ws_bytes = _L.spectra_pack_workspace_size()
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    view = Layer()
    _check(_L.spectra_pack_compact(_ptr(w), n, k, _ptr(idx_c) if n_o else None, n_o, _ptr(codes),
                                   _ptr(scales), _ptr(zeros), _ptr(outw) if n_o else None,
                                   _ptr(bidx), _ptr(ws), ws_bytes, ctypes.byref(view),
                                   _stream(stream)), "spectra_pack_compact")
    return PackedLayer(n, k, n_o, codes, scales, zeros, idx_c, outw, bidx, sz["k_bulk"])


def pack_layer(w: torch.Tensor, gain: torch.Tensor | None, tau: float, *, compact: bool = False,
               stream=None):
    """spectra_pack_plan followed by spectra_pack (or spectra_pack_compact)."""
    idx, _ = spectra_pack_plan(w, gain, tau, stream=stream)
    if compact:
        return spectra_pack_compact(w, idx, stream=stream)
    return spectra_pack(w, idx, stream=stream)


def spectra_unpack(layer: PackedLayer, *, stream=None):
    """Canonical (codes u8 [n,kb], scales int16-bits [n,kb/32], zeros u8 [n,kb/32]),
    kb = k_bulk (k for a masked bulk)."""
    dev = layer.codes.device
    G = layer.k_bulk // 32
    codes = torch.empty((layer.n, layer.k_bulk), dtype=torch.uint8, device=dev)
    scales = torch.empty((layer.n, G), dtype=torch.int16, device=dev)
    zeros = torch.empty((layer.n, G), dtype=torch.uint8, device=dev)
    v = layer.view()
    _check(_L.spectra_unpack(ctypes.byref(v), _ptr(codes), _ptr(scales), _ptr(zeros),
                             _stream(stream)), "spectra_unpack")
    return codes, scales, zeros


_DT = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}


def spectra_gemv(layer: PackedLayer, x: torch.Tensor, y: torch.Tensor | None = None, *,
                 y_dtype=torch.float32, view: Layer | None = None, stream=None) -> torch.Tensor:
    """y = W_hat x for one BF16 vector x [k]."""
    if y is None:
        y = torch.empty(layer.n, dtype=y_dtype, device=x.device)
    v = layer.view() if view is None else view
    _check(_L.spectra_gemv(ctypes.byref(v), _ptr(x), _ptr(y), _DT[y.dtype], _stream(stream)),
           "spectra_gemv")
    return y


def spectra_gemm_small(layer: PackedLayer, x: torch.Tensor, y: torch.Tensor | None = None, *,
                       y_dtype=torch.float32, view: Layer | None = None,
                       stream=None) -> torch.Tensor:
    """y [m, n] = x [m, k] W_hat^T for 1 <= m <= 32."""
    m = x.shape[0]
    if y is None:
        y = torch.empty((m, layer.n), dtype=y_dtype, device=x.device)
    v = layer.view() if view is None else view
    _check(_L.spectra_gemm_small(ctypes.byref(v), _ptr(x), m, _ptr(y), _DT[y.dtype],
                                 _stream(stream)), "spectra_gemm_small")
    return y


def spectra_embed(table: PackedLayer, ids: torch.Tensor, out: torch.Tensor | None = None, *,
                  out_dtype=torch.bfloat16, view: Layer | None = None,
                  stream=None) -> torch.Tensor:
    """Rows ids (int32 [m]) of a packed table, dequantised: out [m, k]."""
    m = int(ids.numel())
    if out is None:
        out = torch.empty((m, table.k), dtype=out_dtype, device=ids.device)
    v = table.view() if view is None else view
    _check(_L.spectra_embed(ctypes.byref(v), _ptr(ids) if m else None, m,
                            _ptr(out) if m else None, _DT[out.dtype], _stream(stream)),
           "spectra_embed")
    return out


@dataclass
class RowTable:
    """Row-table buffers of a packed table (every row's pieces contiguous,
    for gathers only) and the view over them; the index lists are the
    layer's own."""
    layer: PackedLayer
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor
    outlier_w: torch.Tensor
    _view: Layer

    def view(self) -> Layer:
        return self._view

    @property
    def n(self) -> int:
        return self.layer.n

    @property
    def k(self) -> int:
        return self.layer.k


def spectra_row_table_from_layer(layer: PackedLayer, *, stream=None) -> RowTable:
    """Convert a packed layer (RT32) into a row table (new device buffers)."""
    v = layer.view()
    sz = Sizes()
    _check(_L.spectra_row_table_sizes(ctypes.byref(v), ctypes.byref(sz)), "spectra_row_table_sizes")
    dev = layer.codes.device
    codes = _alloc(sz.codes_bytes, torch.uint8, dev)
    scales = _alloc(sz.scales_bytes, torch.int16, dev)
    zeros = _alloc(sz.zeros_bytes, torch.int32, dev)
    outw = _alloc(max(2, sz.outlier_w_bytes), torch.int16, dev)
    out = Layer()
    _check(_L.spectra_row_table_from_layer(ctypes.byref(v), _ptr(codes), _ptr(scales), _ptr(zeros),
                                           _ptr(outw) if layer.n_outliers else None, ctypes.byref(out),
                                           _stream(stream)), "spectra_row_table_from_layer")
    return RowTable(layer, codes, scales, zeros, outw, out)


def spectra_embed_rows(table: RowTable, ids: torch.Tensor, out: torch.Tensor | None = None, *,
                       out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """spectra_embed over a row table: rows ids (int32 [m]) dequantised, out [m, k]."""
    m = int(ids.numel())
    if out is None:
        out = torch.empty((m, table.k), dtype=out_dtype, device=ids.device)
    _check(_L.spectra_embed_rows(ctypes.byref(table.view()), _ptr(ids) if m else None, m,
                                 _ptr(out) if m else None, _DT[out.dtype], _stream(stream)),
           "spectra_embed_rows")
    return out


class BatchViews:
    """Host arrays of layer views and device pointers for spectra_gemv_batched,
    built once and reused (e.g. for graph capture)."""

    def __init__(self, layers, xs, ys):
        n = len(layers)
        self.count = n
        self.layers = (Layer * n)(*[l.view() for l in layers])
        self.xs = (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
        self.ys = (ctypes.c_void_p * n)(*[y.data_ptr() for y in ys])
        dts = {y.dtype for y in ys}
        if len(dts) != 1:
            raise ValueError("all outputs of one batched call share one dtype")
        self.y_dtype = _DT[dts.pop()]
        self._keep = (list(layers), list(xs), list(ys))


def spectra_gemv_batched(layers=None, xs=None, ys=None, *, views: BatchViews | None = None,
                         stream=None) -> BatchViews:
    """Independent batch-1 matvecs ys[i] = W_i xs[i] in one launch."""
    v = views if views is not None else BatchViews(layers, xs, ys)
    _check(_L.spectra_gemv_batched(v.layers, v.xs, v.ys, v.count, v.y_dtype, _stream(stream)),
           "spectra_gemv_batched")
    return v


def spectra_gemv_chain(layers=None, xs=None, ys=None, *, views: BatchViews | None = None,
                       stages=None, workspace: torch.Tensor | None = None,
                       stream=None) -> BatchViews:
    """Dependent batch-1 matvecs ys[i] = W_i xs[i], i in order, in one launch;
    xs[i] may be an earlier ys[j].  With `stages` (a nondecreasing sequence of
    ints, one per matvec) matvec i waits only for the matvecs of earlier
    stages (spectra_gemv_chain_staged).  `workspace` (device, >=
    spectra_gemv_chain_workspace_size(layers, count) bytes) holds the launch's
    completion counter; one is allocated and kept with the views when none is
    given."""
    v = views if views is not None else BatchViews(layers, xs, ys)
    if workspace is None:
        workspace = getattr(v, "_chain_ws", None)
    if workspace is None:
        dev = v._keep[2][0].device
        nbytes = _L.spectra_gemv_chain_workspace_size(v.layers, v.count)
        if nbytes == 0:
            raise SpectraError(_lib.ERR_INVALID_ARG, "spectra_gemv_chain_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        v._chain_ws = workspace
    wsb = workspace.numel() * workspace.element_size()
    if stages is None:
        _check(_L.spectra_gemv_chain(v.layers, v.xs, v.ys, v.count, v.y_dtype, workspace.data_ptr(),
                                     wsb, _stream(stream)), "spectra_gemv_chain")
    else:
        st = (ctypes.c_int32 * len(stages))(*[int(s) for s in stages])
        if len(stages) != v.count:
            raise SpectraError(_lib.ERR_INVALID_ARG, "spectra_gemv_chain_staged: one stage per matvec")
        _check(_L.spectra_gemv_chain_staged(v.layers, v.xs, v.ys, v.count, v.y_dtype, st,
                                            workspace.data_ptr(), wsb, _stream(stream)),
               "spectra_gemv_chain_staged")
    return v


# ---------------------------------------------------------------- TRDC container

_BUFFERS = ("codes", "scales", "zeros", "outlier_idx", "outlier_w", "bulk_idx")


def spectra_crc32(data, crc: int = 0) -> int:
    """CRC-32 of a bytes-like object (the checksum stored in containers)."""
    buf = (ctypes.c_char * len(data)).from_buffer_copy(bytes(data))
    return int(_L.spectra_crc32(crc, buf, len(data)))


def _pinned(nbytes: int) -> torch.Tensor:
    return torch.empty(nbytes, dtype=torch.uint8, pin_memory=True)


def write_container(path: str, layers, names, taus=None, *, staging_bytes: int = 64 << 20,
                    stream=None) -> None:
    """Write packed layers (device buffers) into a TRDC container, streaming
    them through a pinned staging buffer of staging_bytes."""
    n = len(layers)
    views = (Layer * n)(*[l.view() for l in layers])
    cnames = (ctypes.c_char_p * n)(*[nm.encode() for nm in names])
    ctaus = (ctypes.c_double * n)(*(taus if taus is not None else [0.0] * n))
    staging = _pinned(staging_bytes)
    _check(_L.spectra_trdc_write(str(path).encode(), n, cnames, views, ctaus, _lib.MEM_DEVICE,
                                 _ptr(staging), staging_bytes, _stream(stream)),
           "spectra_trdc_write")


class Container:
    """An open TRDC container: layer records, and layers streamed into device
    buffers that this binding allocates with torch."""

    def __init__(self, path: str):
        h = ctypes.c_void_p()
        _check(_L.spectra_trdc_open(str(path).encode(), ctypes.byref(h)), "spectra_trdc_open")
        self._h = h

    def close(self):
        if self._h:
            _L.spectra_trdc_close(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __len__(self) -> int:
        return int(_L.spectra_trdc_count(self._h))

    def info(self, i: int) -> dict:
        r = TrdcLayer()
        _check(_L.spectra_trdc_info(self._h, i, ctypes.byref(r)), "spectra_trdc_info")
        return {"name": r.name.decode(), "n": r.n, "k": r.k, "n_outliers": r.n_outliers,
                "k_bulk": r.k_bulk, "tau": r.tau, "compact": bool(r.flags & 1),
                "offset": list(r.offset), "bytes": list(r.bytes), "crc32": list(r.crc32)}

    def load(self, i: int, device="cuda", *, staging: torch.Tensor | None = None,
             staging_bytes: int = 64 << 20, verify: bool = True, stream=None) -> PackedLayer:
        """Stream layer i into new device buffers; returns the PackedLayer."""
        inf = self.info(i)
        nb = dict(zip(_BUFFERS, inf["bytes"]))
        codes = _alloc(nb["codes"], torch.uint8, device)
        scales = _alloc(nb["scales"], torch.int16, device)
        zeros = _alloc(nb["zeros"], torch.int32, device)
        oidx = _alloc(max(nb["outlier_idx"], 4), torch.int32, device)
        outw = _alloc(max(nb["outlier_w"], 2), torch.int16, device)
        bidx = _alloc(nb["bulk_idx"], torch.int32, device) if inf["compact"] else None
        if staging is None:
            staging = _pinned(staging_bytes)
        view = Layer()
        _check(_L.spectra_trdc_load(self._h, i, _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(oidx),
                                    _ptr(outw), _ptr(bidx), _lib.MEM_DEVICE, _ptr(staging),
                                    staging.numel(), 1 if verify else 0, ctypes.byref(view),
                                    _stream(stream)), "spectra_trdc_load")
        return PackedLayer(inf["n"], inf["k"], inf["n_outliers"], codes, scales, zeros, oidx, outw,
                           bidx, inf["k_bulk"] if inf["compact"] else 0)


# ---------------------------------------------------------------- KV cache

class KVCache:
    """One Group-32 4-bit KV cache (K or V) in device buffers allocated here
    with torch: n_heads x capacity positions of head_dim channels."""

    def __init__(self, n_heads: int, head_dim: int, capacity: int, device="cuda"):
        cb, sb, zb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
        _check(_L.spectra_kv_sizes(n_heads, head_dim, capacity, ctypes.byref(cb), ctypes.byref(sb),
                                   ctypes.byref(zb)), "spectra_kv_sizes")
        self.n_heads, self.head_dim, self.capacity = n_heads, head_dim, capacity
        self.codes = torch.zeros(cb.value, dtype=torch.uint8, device=device)
        self.scales = torch.zeros(sb.value // 2, dtype=torch.int16, device=device)
        self.zeros = torch.zeros(zb.value // 4, dtype=torch.int32, device=device)
        self._view = KV(n_heads, head_dim, capacity, _ptr(self.codes), _ptr(self.scales),
                        _ptr(self.zeros))

    def view(self) -> KV:
        return self._view

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + 2 * self.scales.numel() + 4 * self.zeros.numel()

    def append(self, x: torch.Tensor, pos: int, *, stream=None) -> None:
        """Quantise x (BF16 [n_tok, n_heads, head_dim]) into positions pos.."""
        n_tok = x.shape[0] if x.numel() else 0
        _check(_L.spectra_kv_append(ctypes.byref(self._view), _ptr(x) if n_tok else None, n_tok, pos,
                                    _stream(stream)), "spectra_kv_append")


def spectra_attention_decode(k: KVCache, v: KVCache, q: torch.Tensor, length: int,
                             scale: float | None = None, out: torch.Tensor | None = None, *,
                             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode attention of q (BF16 [n_q_heads, head_dim]) over positions
    0..length-1 of the caches; returns float [n_q_heads, head_dim]."""
    hq, d = q.shape
    if scale is None:
        scale = 1.0 / d ** 0.5
    if out is None:
        out = torch.empty((hq, d), dtype=torch.float32, device=q.device)
    need = _L.spectra_attention_workspace_size(hq, d, length)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(_L.spectra_attention_decode(ctypes.byref(k.view()), ctypes.byref(v.view()), _ptr(q), hq,
                                       length, float(scale), _ptr(out), _ptr(workspace),
                                       workspace.numel(), _stream(stream)),
           "spectra_attention_decode")
    return out


# ---------------------------------------------------------------- paged KV pool

def _arg(t: torch.Tensor, name: str, dtype, shape, dev) -> int:
    """The pointer of a contiguous tensor of this type and shape on dev."""
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: a contiguous {dtype} tensor {list(shape)} on {dev} is wanted, "
                     f"got {t.dtype} {list(t.shape)} with strides {t.stride()} on {t.device}")


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _arg(t, name, dtype, shape, dev)


def _room(workspace: torch.Tensor, dev) -> int:
    """Bytes of a caller's workspace, which must lie on dev in one piece."""
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on {dev} is wanted, got one on {workspace.device} with "
                         f"strides {workspace.stride()}")
    return workspace.numel() * workspace.element_size()


# The current stream's handle without a Stream object around it, which costs
# more than a launch; the public call where this torch has no such entry.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(dev: torch.device, stream, call, *args, **kwargs):
    """call(*args, **kwargs) with dev as the current device and `stream` (when one
    is given) as the current stream, which allocations then belong to."""
    with torch.cuda.device(dev):
        if stream is None:
            return call(*args, **kwargs)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)


class KVPool:
    """A paged Group-32 4-bit pool of K and V that many sequences share:
    n_pages pages of page_size positions of n_heads KV heads, in device buffers
    allocated here with torch (``from_buffers`` takes existing ones).  With
    ``mass`` it also holds every entry's accumulated attention weight."""

    def __init__(self, n_heads: int, head_dim: int, page_size: int, n_pages: int, device="cuda", *,
                 mass: bool = False):
        sz = self.sizes(n_heads, head_dim, page_size, n_pages)
        dev = torch.device(device)
        new = lambda n, dtype, item: torch.zeros(n // item, dtype=dtype, device=dev)  # noqa: E731
        self._set(n_heads, head_dim, page_size, n_pages,
                  [new(sz["codes"], torch.uint8, 1), new(sz["scales"], torch.int16, 2),
                   new(sz["zeros"], torch.int32, 4)] +
                  [new(sz["codes"], torch.uint8, 1), new(sz["scales"], torch.int16, 2),
                   new(sz["zeros"], torch.int32, 4)],
                  new(sz["mass"], torch.float32, 4) if mass else None)

    @staticmethod
    def sizes(n_heads: int, head_dim: int, page_size: int, n_pages: int) -> dict:
        """Bytes of each buffer (codes, scales and zeros once for K and once for V)."""
        got = [ctypes.c_size_t() for _ in range(4)]
        _check(_L.spectra_kv_pool_sizes(n_heads, head_dim, page_size, n_pages, *map(ctypes.byref, got)),
               "spectra_kv_pool_sizes")
        return dict(zip(("codes", "scales", "zeros", "mass"), (g.value for g in got)))

    @classmethod
    def from_buffers(cls, n_heads: int, head_dim: int, page_size: int, n_pages: int, k_codes, k_scales,
                     k_zeros, v_codes, v_scales, v_zeros, mass=None) -> "KVPool":
        """A pool over existing device buffers: codes uint8, scales int16 (FP16
        bits), zeros int32, mass float32, flat, of the sizes that ``sizes`` gives."""
        sz = cls.sizes(n_heads, head_dim, page_size, n_pages)
        if not k_codes.is_cuda:
            raise ValueError(f"k_codes: a tensor on a CUDA device is wanted, got one on {k_codes.device}")
        for t, name, dtype, item in ((k_codes, "codes", torch.uint8, 1), (k_scales, "scales", torch.int16, 2),
                                     (k_zeros, "zeros", torch.int32, 4), (v_codes, "codes", torch.uint8, 1),
                                     (v_scales, "scales", torch.int16, 2), (v_zeros, "zeros", torch.int32, 4)):
            _arg(t, name, dtype, (sz[name] // item,), k_codes.device)
        _opt(mass, "mass", torch.float32, (sz["mass"] // 4,), k_codes.device)
        self = cls.__new__(cls)
        self._set(n_heads, head_dim, page_size, n_pages,
                  [k_codes, k_scales, k_zeros, v_codes, v_scales, v_zeros], mass)
        return self

    def _set(self, n_heads, head_dim, page_size, n_pages, buffers, mass):
        self.n_heads, self.head_dim, self.page_size, self.n_pages = n_heads, head_dim, page_size, n_pages
        (self.k_codes, self.k_scales, self.k_zeros, self.v_codes, self.v_scales, self.v_zeros) = buffers
        self.mass = mass
        self.device = self.k_codes.device
        self._view = _lib.KVPool(n_heads, head_dim, page_size, n_pages, *map(_ptr, buffers), _ptr(mass))
        self._ref = ctypes.byref(self._view)
        self._ws = {}  # workspace bytes of attention, by (rows, query heads)

    def view(self) -> _lib.KVPool:
        return self._view

    @property
    def nbytes(self) -> int:
        """Bytes of the quantised K and V (without the mass)."""
        return 2 * (self.k_codes.numel() + 2 * self.k_scales.numel() + 4 * self.k_zeros.numel())

    def _tokens(self, x, name):
        """(pointer, token stride) of BF16 [n_tok, n_heads, head_dim], heads contiguous."""
        h, d = self.n_heads, self.head_dim
        n = x.shape[0]
        if x.dtype is not torch.bfloat16 or x.shape[1:] != (h, d) or x.device != self.device or \
                (n > 0 and (x.stride(2) != 1 or (h > 1 and x.stride(1) != d))):
            raise ValueError(f"{name}: BF16 [n_tok, {h}, {d}] on {self.device} with contiguous heads is wanted, "
                             f"got {x.dtype} {list(x.shape)} with strides {x.stride()} on {x.device}")
        return x.data_ptr(), x.stride(0) if n > 1 else h * d

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *, stream=None) -> None:
        """Quantise k and v (BF16 [n_tok, n_heads, head_dim], the tokens any
        stride apart) into the token slots page * page_size + r (int32 [n_tok],
        distinct; negative: skipped)."""
        if stream is not None or _current_device() != self.device.index:
            return _elsewhere(self.device, stream, self.append, k, v, slots)
        n = k.shape[0]
        kp, ks = self._tokens(k, "k")
        vp, vs = self._tokens(v, "v")
        if v.shape[0] != n:
            raise ValueError("k and v hold different numbers of tokens")
        sp = _arg(slots, "slots", torch.int32, (n,), self.device)
        _check(_lib.load().spectra_kv_pool_append(self._ref, kp, vp, n, ks, vs, sp, _raw_stream(self.device.index)),
               "spectra_kv_pool_append")

    def read(self, slots: torch.Tensor, *, out_dtype=torch.bfloat16, stream=None):
        """K and V of the token slots (int32 [n]; negative: zeros), dequantised:
        two tensors [n, n_heads, head_dim]."""
        dev = self.device
        if stream is not None or _current_device() != dev.index:
            return _elsewhere(dev, stream, self.read, slots, out_dtype=out_dtype)
        n = slots.shape[0]
        sp = _arg(slots, "slots", torch.int32, (n,), dev)
        if out_dtype not in _DT:
            raise ValueError(f"out_dtype: float32 or bfloat16 is wanted, got {out_dtype}")
        k = torch.empty(n, self.n_heads, self.head_dim, dtype=out_dtype, device=dev)
        v = torch.empty_like(k)
        _check(_lib.load().spectra_kv_pool_read(self._ref, sp, n, k.data_ptr(), v.data_ptr(), _DT[out_dtype],
                                                _raw_stream(dev.index)), "spectra_kv_pool_read")
        return k, v


# A spectra_paged_query as bytes (native alignment, as the C struct).
_PAGED_QUERY = struct.Struct("@PPPiiiiiiffPPPiiP").pack
assert struct.calcsize("@PPPiiiiiiffPPPiiP") == ctypes.sizeof(PagedQuery)


def spectra_attention_paged(pool: KVPool, pages: torch.Tensor, lengths: torch.Tensor, q: torch.Tensor,
                            q_start: torch.Tensor | None = None, *, max_q: int | None = None,
                            scale: float | None = None, softcap: float = 0.0,
                            slopes: torch.Tensor | None = None, window: int = 0,
                            out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                            want_lse: bool = False, update_mass: bool = False,
                            workspace: torch.Tensor | None = None, stream=None):
    """Attention of sequences over a pool: pages int32 [n_seq, max_pages],
    lengths int32 [n_seq] (the new tokens' positions included), q BF16 [n_rows,
    n_q_heads, head_dim].  Sequence b's new tokens are the rows q_start[b] ..
    q_start[b+1]-1 (int32 [n_seq + 1]; without it, row b), at most max_q of
    them (n_rows by default).  softcap > 0 caps the scores, slopes (float
    [n_q_heads]) subtract slope * distance from them, window > 0 hides positions
    that far back and further.  Returns out [n_rows, n_q_heads, head_dim], with
    want_lse also the rows' log sums (float [n_rows, n_q_heads]); update_mass
    adds the weights to the pool's mass.  Rows outside every sequence are not
    written; out may not overlap q."""
    dev = pool.device
    if stream is not None or _current_device() != dev.index:
        return _elsewhere(dev, stream, spectra_attention_paged, pool, pages, lengths, q, q_start, max_q=max_q,
                          scale=scale, softcap=softcap, slopes=slopes, window=window, out=out, out_dtype=out_dtype,
                          want_lse=want_lse, update_mass=update_mass, workspace=workspace)
    n_seq, max_pages = pages.shape
    n_rows, hq, d = q.shape
    if d != pool.head_dim:
        raise ValueError(f"q has head_dim {d}, the pool {pool.head_dim}")
    if max_q is None:
        max_q = 1 if q_start is None else max(n_rows, 1)
    shape = (n_rows, hq, d)
    at_pages = _arg(pages, "pages", torch.int32, (n_seq, max_pages), dev)
    at_lengths = _arg(lengths, "lengths", torch.int32, (n_seq,), dev)
    at_start = 0 if q_start is None else _arg(q_start, "q_start", torch.int32, (n_seq + 1,), dev)
    at_q = _arg(q, "q", torch.bfloat16, shape, dev)
    at_slopes = 0 if slopes is None else _arg(slopes, "slopes", torch.float32, (hq,), dev)
    if (out_dtype if out is None else out.dtype) not in _DT:
        raise ValueError("out: float32 or bfloat16 is wanted")
    if out is not None:
        _arg(out, "out", out.dtype, shape, dev)
    elif out_dtype is torch.bfloat16:
        out = torch.empty_like(q)
    else:
        out = torch.empty(n_rows, hq, d, dtype=out_dtype, device=dev)
    lse = torch.empty(n_rows, hq, dtype=torch.float32, device=dev) if want_lse else None
    lib = _lib.load()
    if workspace is None:
        need = pool._ws.get((n_rows, hq))
        if need is None:
            need = pool._ws[n_rows, hq] = lib.spectra_attention_paged_workspace_size(pool._ref, n_rows, hq)
        workspace, room = torch.empty(need or 16, dtype=torch.uint8, device=dev), need
    else:
        room = _room(workspace, dev)
    x = _PAGED_QUERY(at_pages, at_lengths, at_start, n_seq, max_pages, n_rows, max_q, hq, window,
                     d ** -0.5 if scale is None else scale, softcap, at_q, at_slopes, out.data_ptr(),
                     _DT[out.dtype], 1 if update_mass else 0, lse.data_ptr() if want_lse else 0)
    _check(lib.spectra_attention_paged(pool._ref, x, workspace.data_ptr(), room, _raw_stream(dev.index)),
           "spectra_attention_paged")
    return (out, lse) if want_lse else out


def spectra_kv_evict(pool: KVPool, pages: torch.Tensor, lengths: torch.Tensor, dst_pages: torch.Tensor,
                     budget: int, recent: int, new_lengths: torch.Tensor | None = None, *,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Cut each sequence to its `budget` entries: per head the newest `recent`
    and the ones with the largest accumulated weight, moved in order to the
    fresh pages dst_pages (int32 [n_seq, >= ceil(budget / page_size)]).
    Returns the new lengths (int32 [n_seq], which may not be `lengths`)."""
    dev = pool.device
    if stream is not None or _current_device() != dev.index:
        return _elsewhere(dev, stream, spectra_kv_evict, pool, pages, lengths, dst_pages, budget, recent, new_lengths,
                          workspace=workspace)
    n_seq, max_pages = pages.shape
    dst_max = dst_pages.shape[1]
    at_pages = _arg(pages, "pages", torch.int32, (n_seq, max_pages), dev)
    at_lengths = _arg(lengths, "lengths", torch.int32, (n_seq,), dev)
    at_dst = _arg(dst_pages, "dst_pages", torch.int32, (n_seq, dst_max), dev)
    lib = _lib.load()
    if new_lengths is None:
        new_lengths = torch.empty_like(lengths)
    at_new = _arg(new_lengths, "new_lengths", torch.int32, (n_seq,), dev)
    if workspace is None:
        room = lib.spectra_kv_evict_workspace_size(pool._ref, n_seq, max_pages, budget)
        workspace = torch.empty(room or 16, dtype=torch.uint8, device=dev)
    else:
        room = _room(workspace, dev)
    _check(lib.spectra_kv_evict(pool._ref, at_pages, max_pages, at_lengths, n_seq, at_dst, dst_max, budget, recent,
                                at_new, workspace.data_ptr(), room, _raw_stream(dev.index)), "spectra_kv_evict")
    return new_lengths


# ---------------------------------------------------------------- token choice

def spectra_sample(logits: torch.Tensor, u: torch.Tensor, *, temperature: torch.Tensor | None = None,
                   top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                   min_p: torch.Tensor | None = None, stream=None):
    """Choose a token per row of logits (float [rows, vocab], rows any stride
    apart, or [vocab]) with the uniform numbers u (float [rows]); temperature,
    top_p, min_p (float) and top_k (int32) are [rows] or None.  Returns (ids
    int32 [rows], log of the chosen tokens' probabilities float [rows])."""
    dev = logits.device
    if logits.dim() == 1:
        logits = logits.unsqueeze(0)
    rows, vocab = logits.shape
    if logits.dtype is not torch.float32 or not logits.is_cuda or (rows > 0 and logits.stride(1) != 1):
        raise ValueError(f"logits: float32 rows on a CUDA device are wanted, got {logits.dtype} "
                         f"{list(logits.shape)} with strides {logits.stride()} on {dev}")
    if stream is not None or _current_device() != dev.index:
        return _elsewhere(dev, stream, spectra_sample, logits, u, temperature=temperature, top_k=top_k, top_p=top_p,
                          min_p=min_p)
    f32, one = torch.float32, (rows,)
    at_u = _arg(u, "u", f32, one, dev)
    at_t = None if temperature is None else _arg(temperature, "temperature", f32, one, dev)
    at_k = None if top_k is None else _arg(top_k, "top_k", torch.int32, one, dev)
    at_p = None if top_p is None else _arg(top_p, "top_p", f32, one, dev)
    at_m = None if min_p is None else _arg(min_p, "min_p", f32, one, dev)
    logp = torch.empty_like(u)
    ids = torch.empty(rows, dtype=torch.int32, device=dev)
    _check(_lib.load().spectra_sample(logits.data_ptr(), rows, vocab, logits.stride(0) if rows > 1 else vocab, at_u,
                                      at_t, at_k, at_p, at_m, ids.data_ptr(), logp.data_ptr(),
                                      _raw_stream(dev.index)), "spectra_sample")
    return ids, logp
