"""Python binding of libdcr.so (include/dcr.h): argument marshalling only.

Every step of encode / apply / retry runs in the library's gfx950 kernels;
this module packs descriptors into the C structs, turns torch tensors into
device pointers and the current torch stream into a hipStream_t, and raises
``DcrError`` on a nonzero status.  PyTorch provides device memory and streams.

The names follow the C-ABI: ``dcr_plan_build``, ``dcr_encode``,
``dcr_encode_retry_partial``, ``dcr_encode_retry_from_delta``, ``dcr_apply``,
``dcr_apply_overwrite_retry``, ``dcr_apply_sharded``, ``dcr_apply_overwrite_retry_sharded``, and for weights in 4
bits ``dcr_fp4_quantize``, ``dcr_fp4_dequantize``, ``dcr_fp4_matmul``, ``dcr_fp4_matmul_q``,
``dcr_fp4_matmul_grad`` (plus the small helpers around them).  One turn of training round a refit:
``dcr_experts_select``, ``dcr_experts_select_grad``, ``dcr_experts_order``, ``dcr_experts_dispatch``,
``dcr_experts_combine``, ``dcr_experts_combine_grad``, ``dcr_logprobs``, ``dcr_logprobs_grad`` and ``dcr_adamw_step`` (on
``AdamWTensors``).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdcr.so")

DCR_OK, DCR_E_INVAL, DCR_E_COVERAGE, DCR_E_FORMAT, DCR_E_VERSION, DCR_E_CAPACITY, DCR_E_HIP, DCR_E_NOMEM = \
    0, -1, -2, -3, -4, -5, -6, -7
DCR_E_TIMEOUT = -8
ROUTE_AFFINE_XOR, ROUTE_OVERWRITE, ROUTE_BLOCK_SCALED = 0, 1, 2
MODE_DELTA, MODE_RETRY = 0, 1
ENC_INDEX_LISTS = 0x100            # encode option: index-list layout for low-density records
LAYOUT_BITMAP, LAYOUT_LIST = 0, 1  # directory entry byte 15

# binary layouts of the C structs (include/dcr.h)
TENSOR_DESC = np.dtype([("numel", "<u8"), ("elem_bytes", "<u4"), ("route", "<u4"),
                        ("scale_tensor", "<i4"), ("scale_block", "<u4")])
SEGMENT = np.dtype([("tensor_id", "<u4"), ("shard_id", "<u4"), ("ndim", "<u4"), ("reserved", "<u4"),
                    ("shard_off", "<u8"), ("canon_off", "<u8"), ("extent", "<u8", (4,)),
                    ("shard_stride", "<i8", (4,)), ("canon_stride", "<i8", (4,))])
STREAM_HEADER = np.dtype([("magic", "<u4"), ("format_version", "<u2"), ("stream_kind", "<u2"),
                          ("chunk_bytes", "<u4"), ("reserved0", "<u4"), ("base_version", "<u8"),
                          ("new_version", "<u8"), ("plan_fingerprint", "<u8"), ("n_records", "<u8"),
                          ("payload_bytes", "<u8"), ("reserved1", "<u8")])
ENCODE_RESULT = np.dtype([("n_records", "<u8"), ("payload_bytes", "<u8"), ("n_changed", "<u8"),
                          ("status", "<i4"), ("n_reencoded", "<u4")])
APPLY_RESULT = np.dtype([("n_applied", "<u8"), ("n_skipped", "<u8"), ("n_invalid", "<u8"),
                         ("first_invalid", "<u8")])
assert TENSOR_DESC.itemsize == 24 and SEGMENT.itemsize == 128 and STREAM_HEADER.itemsize == 64
assert ENCODE_RESULT.itemsize == 32 and APPLY_RESULT.itemsize == 32


class PlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in (
        "n_tensors", "n_shards", "n_chunks", "n_pieces", "table_bytes", "workspace_bytes",
        "max_dir_bytes", "max_payload_bytes", "fingerprint", "canonical_bytes", "compact_stage_bytes")]


class DcrError(RuntimeError):
    def __init__(self, code: int, what: str, msg: str):
        super().__init__(f"{what} failed with {code}: {msg}")
        self.code = code


_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libdcr.so; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m bit_exact_xor_amd.build`")
    lib = ctypes.CDLL(p)
    P, U32, U64, I32 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int32
    lib.dcr_plan_build.restype = I32
    lib.dcr_plan_build.argtypes = [P, U32, P, U32, P, U64, ctypes.POINTER(P)]
    lib.dcr_plan_query.restype = I32
    lib.dcr_plan_query.argtypes = [P, ctypes.POINTER(PlanInfo)]
    lib.dcr_plan_upload.restype = I32
    lib.dcr_plan_upload.argtypes = [P, P, U64, P]
    lib.dcr_plan_destroy.restype = None
    lib.dcr_plan_destroy.argtypes = [P]
    lib.dcr_encode.restype = I32
    lib.dcr_encode.argtypes = [P, P, P, U32, U64, U64, P, P, U64, P, U64, P, P, U64, P]
    lib.dcr_encode_pipelined.restype = I32
    for fn in (lib.dcr_stream_pack, lib.dcr_stream_unpack):
        fn.restype = I32
        fn.argtypes = [P, P, P, P, P, P, U64, P, U64, P, P, U64, P]
    lib.dcr_encode_noalloc.restype = I32
    lib.dcr_encode_noalloc.argtypes = [P, P, P, U32, U64, U64, P, P, U64, P, U64, P, P]
    lib.dcr_encode_pipelined.argtypes = [P, P, P, U32, U64, U64, P, P, U64, P, U64, P, P, U64, U32, P, U64, P]
    lib.dcr_ready_wait.restype = I32
    lib.dcr_ready_wait.argtypes = [P, U32, U64, P]
    lib.dcr_encode_retry_partial.restype = I32
    lib.dcr_encode_retry_partial.argtypes = [P, P, P, P, P, U64, P, U64, U64, P, P, U64, P, U64, P, P, U64, P]
    lib.dcr_encode_retry_from_delta.restype = I32
    lib.dcr_encode_retry_from_delta.argtypes = [P, P, P, P, U64, P, U64, U32, P, P, U64, P, U64, P, P, U64, P]
    lib.dcr_apply.restype = I32
    lib.dcr_apply.argtypes = [P, P, P, P, P, P, U64, U64, U64, P, P, U64, P]
    lib.dcr_apply_sharded.restype = I32
    lib.dcr_apply_sharded.argtypes = [P, P, P, P, P, P, U64, U64, U64, P, P, U64, P]
    lib.dcr_apply_overwrite_retry_sharded.restype = I32
    lib.dcr_apply_overwrite_retry_sharded.argtypes = [P, P, P, P, P, U64, P, P, U64, P]
    lib.dcr_apply_overwrite_retry.restype = I32
    lib.dcr_apply_overwrite_retry.argtypes = [P, P, P, P, P, U64, P, P, U64, P]
    lib.dcr_fp4_quantize.restype = I32
    lib.dcr_fp4_quantize.argtypes = [P, U32, U64, P, U32, P, U64, P]
    lib.dcr_fp4_dequantize.restype = I32
    lib.dcr_fp4_dequantize.argtypes = [P, P, U32, U64, P]
    for fn in (lib.dcr_fp4_matmul, lib.dcr_fp4_matmul_grad):
        fn.restype = I32
        fn.argtypes = [P, U64, U64, P, P, U32, P, U32, U64, P, U64, P]
    lib.dcr_fp4_matmul_q.restype = I32
    lib.dcr_fp4_matmul_q.argtypes = [P, P, P, U32, P, U32, U64, P, U64, P]
    FLT = ctypes.c_float
    for name, args in (
            ("dcr_experts_select", [P, U32, U64, U64, U32, P, U32, U32, U32, U32, FLT, U32, P, P, P]),
            ("dcr_experts_select_grad", [P, U32, U64, U64, U32, P, P, U32, U32, U32, FLT, P, U64, P]),
            ("dcr_experts_order", [P, U64, U32, P, P, P, U64, P]),
            ("dcr_experts_dispatch", [P, U32, U64, U64, U64, P, U32, P, U32, U64, U64, P]),
            ("dcr_experts_combine", [P, U32, U64, U64, P, P, U64, U64, U32, P, U32, U64, P]),
            ("dcr_experts_combine_grad", [P, U32, U64, U64, U64, P, U32, U64, U64, P, P, U32, P, U32, U64, P, P]),
            ("dcr_logprobs", [P, U32, U64, U64, U64, P, U32, FLT, P, P, P, U32, P, P, P, U64, P]),
            ("dcr_logprobs_grad", [P, U32, U64, U64, U64, P, U32, FLT, P, P, P, P, P, U64, P]),
            ("dcr_adamw_plan_build", [P, U64, ctypes.POINTER(P)]), ("dcr_adamw_plan_bytes", [P, ctypes.POINTER(U64)]),
            ("dcr_adamw_plan_upload", [P, P, U64, P]), ("dcr_adamw_step", [P, P, P])):
        getattr(lib, name).restype = I32
        getattr(lib, name).argtypes = args
    lib.dcr_adamw_plan_destroy.restype = None
    lib.dcr_adamw_plan_destroy.argtypes = [P]
    lib.dcr_last_error.restype = ctypes.c_char_p
    lib.dcr_last_error.argtypes = []
    lib.dcr_set_kernel_events.restype = None
    lib.dcr_set_kernel_events.argtypes = [P, P]
    lib.dcr_format_constants.restype = U32
    lib.dcr_format_constants.argtypes = [P, U32]
    if path is None:
        _lib = lib
    return lib


def _check(rc: int, what: str) -> None:
    if rc != DCR_OK:
        raise DcrError(rc, what, load_library().dcr_last_error().decode())


def _pack(arr, dtype):
    out = np.zeros(len(arr), dtype=dtype)
    for name in dtype.names:
        if name == "reserved":
            continue
        out[name] = arr[name]
    return out


def _ptr_array(ptrs):
    arr = (ctypes.c_void_p * max(1, len(ptrs)))()
    for i, p in enumerate(ptrs):
        arr[i] = int(p) if p else None
    return arr


class PtrTable:
    """The device addresses of a fixed list of buffers (shards or canonical
    tensors), packed once into pinned host memory.  Pass it wherever a list
    of buffers is taken: calls on plans with many tensors then skip
    rebuilding the address array, and the library's copy of it to the
    workspace is an asynchronous DMA instead of a staged pageable copy.  The
    buffers are kept alive by the table; it must not outlive their storage
    moving (torch never moves a tensor's storage).  Needs a GPU runtime
    (pinned host memory); a table passed to calls captured into a HIP graph
    must outlive the graph, whose copy nodes read it at every replay."""

    def __init__(self, bufs):
        import torch
        self.bufs = list(bufs)
        n = len(self.bufs)
        self.host = torch.empty(max(1, n), dtype=torch.int64, pin_memory=True)
        if n:
            self.host.numpy()[:n] = np.array([_dptr(t) for t in self.bufs], dtype=np.uint64).view(np.int64)
        self.address = int(self.host.data_ptr())

    def __len__(self):
        return len(self.bufs)


def _ptrs(bufs):
    """A C array of device addresses for a list of buffers or a PtrTable."""
    if isinstance(bufs, PtrTable):
        return ctypes.c_void_p(bufs.address)
    return _ptr_array([_dptr(t) for t in bufs])


def _dptr(t) -> int:
    """Device pointer of a torch tensor (or an int address)."""
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return int(t.ctypes.data)
    return int(t.data_ptr())


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream or None
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else (int(stream) or None)


class Plan:
    """A built plan (host) plus its device tables once uploaded."""

    def __init__(self, handle: int, info: PlanInfo):
        self.handle = handle
        self.info = info
        self.tables = None

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.dcr_plan_destroy(h)


def dcr_plan_build(tensors, shard_bytes, segments) -> Plan:
    """Build a plan from a tensor table, shard sizes (bytes) and affine segments."""
    lib = load_library()
    T = _pack(tensors, TENSOR_DESC)
    S = _pack(segments, SEGMENT)
    sb = np.ascontiguousarray(np.asarray(shard_bytes, dtype=np.uint64))
    h = ctypes.c_void_p()
    rc = lib.dcr_plan_build(T.ctypes.data if len(T) else None, len(T), sb.ctypes.data if len(sb) else None,
                            len(sb), S.ctypes.data if len(S) else None, len(S), ctypes.byref(h))
    _check(rc, "dcr_plan_build")
    info = PlanInfo()
    _check(lib.dcr_plan_query(h, ctypes.byref(info)), "dcr_plan_query")
    return Plan(h.value, info)


def dcr_plan_upload(plan: Plan, device="cuda", stream=None) -> None:
    import torch
    plan.tables = torch.empty(max(int(plan.info.table_bytes), 16), dtype=torch.uint8, device=device)
    _check(load_library().dcr_plan_upload(plan.handle, plan.tables.data_ptr(), plan.tables.numel(),
                                          _stream(stream)), "dcr_plan_upload")


def dcr_encode(plan: Plan, old_shards, new_shards, mode, base_version, new_version,
               header, dir_buf, payload, result, workspace, stream=None) -> None:
    """Enqueue an encode; buffers are torch device tensors (or int addresses)."""
    rc = load_library().dcr_encode(
        plan.handle, _ptrs(old_shards), _ptrs(new_shards),
        mode, base_version, new_version, _dptr(header), _dptr(dir_buf), _nbytes(dir_buf), _dptr(payload),
        _nbytes(payload), _dptr(result), _dptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "dcr_encode")


LAYOUT_GAPS = 2                    # directory entry byte 15, packed streams only
MAGIC_PACKED = 0x50524344


def _transport(fn, what, plan, header, dir_buf, payload, header_out, dir_out, payload_out, result, workspace,
               stream=None):
    h = np.ascontiguousarray(np.asarray(header, dtype=np.uint8).reshape(-1)[:64])
    rc = fn(plan.handle, h.ctypes.data, _dptr(dir_buf), _dptr(payload), _dptr(header_out), _dptr(dir_out),
            _nbytes(dir_out), _dptr(payload_out), _nbytes(payload_out), _dptr(result), _dptr(workspace),
            _nbytes(workspace), _stream(stream))
    _check(rc, what)


def dcr_stream_pack(plan: Plan, header, dir_buf, payload, header_out, dir_out, payload_out, result, workspace,
                    stream=None) -> None:
    """Enqueue the transport packing of a stream (host header, device
    buffers) into the output buffers."""
    _transport(load_library().dcr_stream_pack, "dcr_stream_pack", plan, header, dir_buf, payload, header_out,
               dir_out, payload_out, result, workspace, stream)


def dcr_stream_unpack(plan: Plan, header, dir_buf, payload, header_out, dir_out, payload_out, result, workspace,
                      stream=None) -> None:
    """Enqueue the inverse of dcr_stream_pack."""
    _transport(load_library().dcr_stream_unpack, "dcr_stream_unpack", plan, header, dir_buf, payload, header_out,
               dir_out, payload_out, result, workspace, stream)


NOALLOC_SCRATCH_BYTES = 64 << 20   # DCR_NOALLOC_SCRATCH_BYTES


def dcr_encode_noalloc(plan: Plan, old_shards, new_shards, mode, base_version, new_version,
                       header, dir_buf, payload, result, stream=None) -> None:
    """Enqueue an encode that uses the library's own device scratch array as
    its workspace (no workspace argument; calls overlapping on one GPU race)."""
    rc = load_library().dcr_encode_noalloc(
        plan.handle, _ptrs(old_shards), _ptrs(new_shards),
        mode, base_version, new_version, _dptr(header), _dptr(dir_buf), _nbytes(dir_buf), _dptr(payload),
        _nbytes(payload), _dptr(result), _stream(stream))
    _check(rc, "dcr_encode_noalloc")


def ready_region_bytes(n_slices: int) -> int:
    """Bytes of a dcr_encode_pipelined watermark region for n_slices."""
    return 64 + 64 * int(n_slices)


def dcr_encode_pipelined(plan: Plan, old_shards, new_shards, mode, base_version, new_version,
                         header, dir_buf, payload, result, workspace, n_slices, ready, stream=None) -> None:
    """Enqueue a sliced encode that publishes a ready watermark after each
    slice into `ready`, a pinned host tensor of ready_region_bytes(n_slices)."""
    rc = load_library().dcr_encode_pipelined(
        plan.handle, _ptrs(old_shards), _ptrs(new_shards),
        mode, base_version, new_version, _dptr(header), _dptr(dir_buf), _nbytes(dir_buf), _dptr(payload),
        _nbytes(payload), _dptr(result), _dptr(workspace), _nbytes(workspace), n_slices, _dptr(ready),
        _nbytes(ready), _stream(stream))
    _check(rc, "dcr_encode_pipelined")


def dcr_ready_wait(ready, slice_index: int, timeout_us: int = 10_000_000) -> np.ndarray:
    """Wait until slice `slice_index` of a watermark region is published;
    returns its prefix header (64 bytes)."""
    out = np.zeros(64, dtype=np.uint8)
    rc = load_library().dcr_ready_wait(_dptr(ready), slice_index, timeout_us, out.ctypes.data)
    _check(rc, "dcr_ready_wait")
    return out


def dcr_encode_retry_partial(plan: Plan, old_shards, new_shards, delta_header: np.ndarray, delta_dir, delta_flags,
                             base_version, new_version, header, dir_buf, payload, result, workspace,
                             stream=None) -> None:
    """Enqueue a partial retry encode: a RETRY stream over the chunks that hold
    a record of the DELTA stream (host header bytes, device directory) whose
    applied flag (device bytes) is 0."""
    hdr = np.ascontiguousarray(np.asarray(delta_header, dtype=np.uint8))
    rc = load_library().dcr_encode_retry_partial(
        plan.handle, _ptrs(old_shards), _ptrs(new_shards),
        hdr.ctypes.data, _dptr(delta_dir), _nbytes(delta_dir), _dptr(delta_flags), base_version, new_version,
        _dptr(header), _dptr(dir_buf), _nbytes(dir_buf), _dptr(payload), _nbytes(payload), _dptr(result),
        _dptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "dcr_encode_retry_partial")


def dcr_encode_retry_from_delta(plan: Plan, old_shards, delta_header: np.ndarray, delta_dir, delta_payload,
                                options, header, dir_buf, payload, result, workspace, stream=None) -> None:
    """Enqueue a RETRY stream written from a DELTA stream (host header bytes,
    device directory and payload) and the old shards; options 0 or
    DCR_ENC_INDEX_LISTS."""
    hdr = np.ascontiguousarray(np.asarray(delta_header, dtype=np.uint8))
    rc = load_library().dcr_encode_retry_from_delta(
        plan.handle, _ptrs(old_shards), hdr.ctypes.data, _dptr(delta_dir), _nbytes(delta_dir),
        _dptr(delta_payload), _nbytes(delta_payload), options, _dptr(header), _dptr(dir_buf), _nbytes(dir_buf),
        _dptr(payload), _nbytes(payload), _dptr(result), _dptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "dcr_encode_retry_from_delta")


def dcr_apply(plan: Plan, canon, header: np.ndarray, dir_buf, payload, flags, first_record, n_records,
              expected_base_version, result, workspace, stream=None) -> None:
    """Enqueue an apply of records [first, first+n); header is host bytes (64)."""
    hdr = np.ascontiguousarray(np.asarray(header, dtype=np.uint8))
    rc = load_library().dcr_apply(
        plan.handle, _ptrs(canon), hdr.ctypes.data, _dptr(dir_buf), _dptr(payload),
        _dptr(flags), first_record, n_records, expected_base_version, _dptr(result), _dptr(workspace),
        _nbytes(workspace), _stream(stream))
    _check(rc, "dcr_apply")


def dcr_apply_overwrite_retry(plan: Plan, canon, header: np.ndarray, dir_buf, payload,
                              expected_base_version, result, workspace, stream=None) -> None:
    hdr = np.ascontiguousarray(np.asarray(header, dtype=np.uint8))
    rc = load_library().dcr_apply_overwrite_retry(
        plan.handle, _ptrs(canon), hdr.ctypes.data, _dptr(dir_buf), _dptr(payload),
        expected_base_version, _dptr(result), _dptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "dcr_apply_overwrite_retry")


def dcr_apply_sharded(plan: Plan, shards, header: np.ndarray, dir_buf, payload, flags, first_record, n_records,
                      expected_base_version, result, workspace, stream=None) -> None:
    """Apply records [first, first+n) into a receiver layout: `plan` is the
    receiver plan, `shards` its device shards."""
    hdr = np.ascontiguousarray(np.asarray(header, dtype=np.uint8))
    rc = load_library().dcr_apply_sharded(
        plan.handle, _ptrs(shards), hdr.ctypes.data, _dptr(dir_buf), _dptr(payload),
        _dptr(flags), first_record, n_records, expected_base_version, _dptr(result), _dptr(workspace),
        _nbytes(workspace), _stream(stream))
    _check(rc, "dcr_apply_sharded")


def dcr_apply_overwrite_retry_sharded(plan: Plan, shards, header: np.ndarray, dir_buf, payload,
                                      expected_base_version, result, workspace, stream=None) -> None:
    """Overwrite retry into a receiver layout (see dcr_apply_sharded)."""
    hdr = np.ascontiguousarray(np.asarray(header, dtype=np.uint8))
    rc = load_library().dcr_apply_overwrite_retry_sharded(
        plan.handle, _ptrs(shards), hdr.ctypes.data, _dptr(dir_buf), _dptr(payload),
        expected_base_version, _dptr(result), _dptr(workspace), _nbytes(workspace), _stream(stream))
    _check(rc, "dcr_apply_overwrite_retry_sharded")


# ------------------------------------------------------------ 4-bit weights

FP4_MX, FP4_NV = 0, 1              # DCR_FP4_*: blocks of 32 with 2^n scales / of 16 with e4m3 scales
F32, BF16 = 0, 1                   # DCR_F32, DCR_BF16
FP4_CALIBRATE = 1                  # DCR_FP4_CALIBRATE
FP4_WORKSPACE_BYTES = 64 << 20     # DCR_FP4_WORKSPACE_BYTES


class Fp4Desc(ctypes.Structure):
    """dcr_fp4_tensor."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("rows", ctypes.c_uint64), ("cols", ctypes.c_uint64), ("code_stride", ctypes.c_uint64),
                ("scale_stride", ctypes.c_uint64), ("format", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


def fp4_blocks(cols: int, fmt: int) -> int:
    """Scale blocks of a row."""
    b = 32 if fmt == FP4_MX else 16
    return -(-int(cols) // b)


class Fp4Tensor:
    """A 4-bit tensor of `rows` x `cols` elements in device memory: `codes`
    (uint8, [rows, stride], rows padded to 16 bytes where made here),
    `scales` (uint8, [rows, blocks]) and, in the NV format, `tensor_scale`
    (fp32, one element).  Buffers that are passed in are used as they are
    (any row stride); they may be canonical tensors a refit patches.  The
    tensor keeps them: new contents are copied into them."""

    def __init__(self, rows, cols, fmt=FP4_MX, device="cuda", codes=None, scales=None, tensor_scale=None):
        import torch
        rows, cols = int(rows), int(cols)
        if fmt not in (FP4_MX, FP4_NV):
            raise ValueError("fmt is FP4_MX or FP4_NV")
        width, blocks = (cols + 1) // 2, fp4_blocks(cols, fmt)
        if codes is None:
            codes = torch.zeros(rows, -(-width // 16) * 16, dtype=torch.uint8, device=device)
        if scales is None:
            scales = torch.zeros(rows, blocks, dtype=torch.uint8, device=codes.device)
        if fmt == FP4_NV and tensor_scale is None:
            tensor_scale = torch.ones(1, dtype=torch.float32, device=codes.device)
        for name, t, w in (("codes", codes, width), ("scales", scales, blocks)):
            if t.dtype != torch.uint8 or t.dim() != 2 or t.shape[0] != rows or t.shape[1] < w or \
                    (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError(f"{name}: uint8 [{rows}, >= {w}] with contiguous rows expected")
        if fmt == FP4_NV and (tensor_scale.dtype != torch.float32 or tensor_scale.numel() != 1):
            raise ValueError("tensor_scale: one fp32 element expected")
        self.index = _one_device(codes, scales, tensor_scale if fmt == FP4_NV else None)
        self.rows, self.cols, self.fmt = rows, cols, fmt
        self.codes, self.scales = codes, scales
        self.tensor_scale = tensor_scale if fmt == FP4_NV else None
        self.device = codes.device
        self.desc = Fp4Desc(codes.data_ptr(), scales.data_ptr(),
                            tensor_scale.data_ptr() if fmt == FP4_NV else None, rows, cols,
                            codes.stride(0), scales.stride(0), fmt, 0)
        self._ref = ctypes.addressof(self.desc)

    def __setattr__(self, name, value):
        # (a new buffer would leave the description with the old one's address)
        if "_ref" in self.__dict__:
            raise AttributeError(f"{name}: an Fp4Tensor keeps its buffers; copy into them or make another")
        super().__setattr__(name, value)


def fp4_workspace(device="cuda"):
    """Workspace of the 4-bit calls (one call at a time; captured graphs that
    may run together need one each)."""
    import torch
    return torch.empty(FP4_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def _one_device(first, *others):
    """Index of the GPU that all of the tensors (None: left out) are on."""
    dev = first.get_device() if not isinstance(first, Fp4Tensor) else first.index
    if dev < 0:
        raise ValueError("tensors in GPU memory expected")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on different devices: cuda:{dev} and {t.device}")
    return dev


def _wide(t, rows, cols, name):
    """(pointer, type, row stride) of a BF16 or fp32 matrix."""
    import torch
    if t.dtype is torch.bfloat16:
        ty = BF16
    elif t.dtype is torch.float32:
        ty = F32
    else:
        raise ValueError(f"{name}: bfloat16 or float32 expected, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or shape[1] != cols or \
            (cols > 1 and strides[1] != 1):
        raise ValueError(f"{name}: [{'m' if rows is None else rows}, {cols}] with contiguous rows expected, "
                         f"got {tuple(shape)} with strides {strides}")
    if shape[0] > 1 and strides[0] < cols:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), ty, strides[0]


def _whole(workspace):
    """Refuse a workspace with gaps: the library takes an address and a size."""
    if not workspace.is_contiguous():
        raise ValueError("workspace: contiguous memory expected")


def _fp4_call(torch, fn, what, device, stream, *args):
    """Call `fn` with GPU `device`, the one of its tensors, current, on
    `stream` or that GPU's current stream."""
    # (torch.cuda.current_stream() costs as much as the rest of a small call)
    raw = torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == device:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc:
        _check(rc, what)


def dcr_fp4_quantize(x, q: Fp4Tensor, options=0, workspace=None, stream=None) -> None:
    """Enqueue the quantisation of x (BF16 or fp32, [rows, cols]) into q;
    FP4_CALIBRATE (NV) first takes q's tensor scale from x, and needs a
    workspace."""
    import torch
    p, ty, stride = _wide(x, q.rows, q.cols, "x")
    if workspace is not None:
        _whole(workspace)
    dev = _one_device(q, x, workspace)
    _fp4_call(torch, load_library().dcr_fp4_quantize, "dcr_fp4_quantize", dev, stream, p, ty, stride, q._ref, options,
              workspace.data_ptr() if workspace is not None else None,
              _nbytes(workspace) if workspace is not None else 0)


def dcr_fp4_dequantize(q: Fp4Tensor, y, stream=None) -> None:
    """Enqueue reading q back into y (BF16 or fp32, [rows, cols])."""
    import torch
    p, ty, stride = _wide(y, q.rows, q.cols, "y")
    dev = _one_device(q, y)
    _fp4_call(torch, load_library().dcr_fp4_dequantize, "dcr_fp4_dequantize", dev, stream, q._ref, p, ty, stride)


def _groups(w, offsets):
    """(offsets pointer, groups, rows of a group) of a product with w."""
    if offsets is None:
        return None, 1, w.rows
    import torch
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous():
        raise ValueError("offsets: contiguous int32 [groups + 1] expected")
    g = offsets.numel() - 1
    if w.rows % g:
        raise ValueError(f"{g} groups do not divide {w.rows} rows of weights")
    return offsets.data_ptr(), g, w.rows // g


def _product(fn, what, x, w, y, offsets, workspace, stream, grad):
    import torch
    if workspace is None:
        raise ValueError("workspace: pass one made by fp4_workspace()")
    _whole(workspace)
    off, g, n = _groups(w, offsets)
    yn = "dx" if grad else "y"
    if isinstance(x, Fp4Tensor):
        if fn is not load_library().dcr_fp4_matmul_q:
            raise ValueError(f"{what}: bfloat16 rows expected, got an Fp4Tensor")
        yp, ty, ys = _wide(y, x.rows, n, yn)
        dev = _one_device(w, x.codes, y, offsets, workspace)
        _fp4_call(torch, fn, what, dev, stream, x._ref, w._ref, off, g, yp, ty, ys, workspace.data_ptr(), workspace.nbytes)
        return
    if x.dtype is not torch.bfloat16:
        raise ValueError(f"{what}: bfloat16 rows expected, got {x.dtype}")
    xp, _ty, xs = _wide(x, None, n if grad else w.cols, "dy" if grad else "x")
    m = x.shape[0]
    yp, ty, ys = _wide(y, m, w.cols if grad else n, yn)
    dev = _one_device(w, x, y, offsets, workspace)
    _fp4_call(torch, fn, what, dev, stream, xp, m, xs, w._ref, off, g, yp, ty, ys, workspace.data_ptr(), workspace.nbytes)


def dcr_fp4_matmul(x, w: Fp4Tensor, y, offsets=None, workspace=None, stream=None) -> None:
    """Enqueue y = x w^T: x BF16 [m, cols], w [n, cols] in 4 bits, y BF16 or
    fp32 [m, n].  With `offsets` (int32 [groups + 1], device) w holds `groups`
    weights stacked along its rows and rows offsets[g] .. offsets[g + 1] of x
    take weight g; the other rows of y are left as they are."""
    _product(load_library().dcr_fp4_matmul, "dcr_fp4_matmul", x, w, y, offsets, workspace, stream, False)


def dcr_fp4_matmul_q(x: Fp4Tensor, w: Fp4Tensor, y, offsets=None, workspace=None, stream=None) -> None:
    """Enqueue y = x w^T with both operands in 4 bits (FP4_MX); else as
    dcr_fp4_matmul."""
    if not isinstance(x, Fp4Tensor):
        raise ValueError("x: an Fp4Tensor expected")
    _product(load_library().dcr_fp4_matmul_q, "dcr_fp4_matmul_q", x, w, y, offsets, workspace, stream, False)


def dcr_fp4_matmul_grad(dy, w: Fp4Tensor, dx, offsets=None, workspace=None, stream=None) -> None:
    """Enqueue dx = dy w, the gradient of dcr_fp4_matmul with respect to x:
    dy BF16 [m, n], dx BF16 or fp32 [m, cols]."""
    _product(load_library().dcr_fp4_matmul_grad, "dcr_fp4_matmul_grad", dy, w, dx, offsets, workspace, stream, True)


# ------------------------------------------- one turn of training round a refit

STEP_WORKSPACE_BYTES = 4 << 20     # DCR_STEP_WORKSPACE_BYTES
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1   # DCR_SCORE_*
EXPERTS_RENORMALIZE = 1            # DCR_EXPERTS_RENORMALIZE
ADAMW_BLOCK = 32                   # DCR_ADAMW_BLOCK
ADAMW_NO_DECAY = 1                 # DCR_ADAMW_NO_DECAY


def step_workspace(device="cuda"):
    """Workspace of dcr_experts_order and dcr_logprobs (one call at a time;
    captured graphs that may run together need one each)."""
    import torch
    return torch.empty(STEP_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def _array(t, dtype, shape, name):
    """Address of a contiguous tensor of one type and shape, None of None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} {list(shape)} expected, got {t.dtype} {list(t.shape)} with strides "
                         f"{t.stride()}")
    return t.data_ptr()


def _need(t, name):
    if t is None:
        raise ValueError(f"{name}: a tensor expected")
    return t


def _step_space(workspace):
    if workspace is None:
        raise ValueError("workspace: pass one made by step_workspace()")
    _whole(workspace)


def dcr_experts_select(logits, ids, weights, bias=None, score=SCORE_SOFTMAX, groups=1, top_groups=1, renormalize=False,
                       scale=1.0, stream=None) -> None:
    """Enqueue the choice of the k best experts of each row: logits BF16 or
    fp32 [rows, experts], ids int32 [rows, k] (-1: none left), weights fp32
    [rows, k]; `bias` (fp32 [experts]) is seen by the choice alone, which is
    among the experts of the `top_groups` best of `groups` groups."""
    import torch
    rows, k = ids.shape
    p, ty, stride = _wide(logits, rows, logits.shape[-1], "logits")
    experts = logits.shape[1]
    i, w = _array(ids, torch.int32, (rows, k), "ids"), _array(weights, torch.float32, (rows, k), "weights")
    b = _array(bias, torch.float32, (experts,), "bias")
    dev = _one_device(logits, ids, weights, bias)
    _fp4_call(torch, load_library().dcr_experts_select, "dcr_experts_select", dev, stream, p, ty, stride, rows, experts, b,
              score, groups, top_groups, EXPERTS_RENORMALIZE if renormalize else 0, scale, k, i, w)


def dcr_experts_select_grad(logits, ids, dweights, dlogits, score=SCORE_SOFTMAX, renormalize=False, scale=1.0,
                            stream=None) -> None:
    """Enqueue the gradient of dcr_experts_select's weights with respect to the
    logits; dlogits has the logits' type and may be the logits."""
    import torch
    rows, k = ids.shape
    experts = logits.shape[-1]
    p, ty, stride = _wide(logits, rows, experts, "logits")
    d, dty, d_stride = _wide(dlogits, rows, experts, "dlogits")
    if dty != ty:
        raise ValueError(f"dlogits: {logits.dtype} expected, got {dlogits.dtype}")
    i, w = _array(ids, torch.int32, (rows, k), "ids"), _array(dweights, torch.float32, (rows, k), "dweights")
    dev = _one_device(logits, ids, dweights, dlogits)
    _fp4_call(torch, load_library().dcr_experts_select_grad, "dcr_experts_select_grad", dev, stream, p, ty, stride, rows,
              experts, i, w, k, score, EXPERTS_RENORMALIZE if renormalize else 0, scale, d, d_stride)


def dcr_experts_order(ids, offsets, slots, workspace, stream=None) -> None:
    """Enqueue the slots of the pairs sorted by expert (int32, like ids; -1
    without one) and the experts' offsets (int32 [experts + 1])."""
    import torch
    _step_space(workspace)
    i, s = _array(ids, torch.int32, ids.shape, "ids"), _array(slots, torch.int32, ids.shape, "slots")
    o = _array(offsets, torch.int32, offsets.shape, "offsets")
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets: [experts + 1] expected")
    dev = _one_device(ids, offsets, slots, workspace)
    _fp4_call(torch, load_library().dcr_experts_order, "dcr_experts_order", dev, stream, i, ids.numel(), offsets.numel() - 1,
              o, s, workspace.data_ptr(), workspace.nbytes)


def dcr_experts_dispatch(x, slots, y, stream=None) -> None:
    """Enqueue y[slots[t, j]] = x[t]: x [tokens, width], slots int32 [tokens, k],
    y [slots, width], each BF16 or fp32; other rows of y stay as they are."""
    import torch
    tokens, k = slots.shape
    width = x.shape[-1]
    xp, xt, xs = _wide(x, tokens, width, "x")
    yp, yt, ys = _wide(y, None, width, "y")
    s = _array(slots, torch.int32, (tokens, k), "slots")
    dev = _one_device(x, slots, y)
    _fp4_call(torch, load_library().dcr_experts_dispatch, "dcr_experts_dispatch", dev, stream, xp, xt, xs, tokens, width, s,
              k, yp, yt, ys, y.shape[0])


def dcr_experts_combine(x, slots, weights, y, stream=None) -> None:
    """Enqueue y[t] = sum over j of weights[t, j] x[slots[t, j]]; `weights`
    (fp32 [tokens, k]) None: 1, the gradient of dcr_experts_dispatch."""
    import torch
    tokens, k = slots.shape
    width = y.shape[-1]
    xp, xt, xs = _wide(x, None, width, "x")
    yp, yt, ys = _wide(y, tokens, width, "y")
    s, w = _array(slots, torch.int32, (tokens, k), "slots"), _array(weights, torch.float32, (tokens, k), "weights")
    dev = _one_device(x, slots, weights, y)
    _fp4_call(torch, load_library().dcr_experts_combine, "dcr_experts_combine", dev, stream, xp, xt, xs, x.shape[0], s, w,
              tokens, width, k, yp, yt, ys)


def dcr_experts_combine_grad(dy, x, slots, weights, dx, dweights, stream=None) -> None:
    """Enqueue dx[slots[t, j]] = weights[t, j] dy[t] (other rows stay as they
    are) and dweights[t, j] = <dy[t], x[slots[t, j]]>."""
    import torch
    tokens, k = slots.shape
    width = dy.shape[-1]
    dp, dt, ds = _wide(dy, tokens, width, "dy")
    xp, xt, xs = _wide(x, None, width, "x")
    n = x.shape[0]
    gp, gt, gs = _wide(dx, n, width, "dx")
    s, w = _array(slots, torch.int32, (tokens, k), "slots"), _array(_need(weights, "weights"), torch.float32, (tokens, k), "weights")
    dw = _array(dweights, torch.float32, (tokens, k), "dweights")
    dev = _one_device(dy, x, slots, weights, dx, dweights)
    _fp4_call(torch, load_library().dcr_experts_combine_grad, "dcr_experts_combine_grad", dev, stream, dp, dt, ds, tokens,
              width, xp, xt, xs, n, s, w, k, gp, gt, gs, dw)


def _targets(t, rows):
    """(address, bytes of an element) of target tokens."""
    import torch
    if t is None:
        return None, 4
    if t.dtype is not torch.int32 and t.dtype is not torch.int64:
        raise ValueError(f"targets: int32 or int64 expected, got {t.dtype}")
    return _array(t, t.dtype, (rows,), "targets"), t.element_size()


def dcr_logprobs(logits, targets, logp=None, lse=None, entropy=None, top_ids=None, top_values=None, scale=1.0,
                 workspace=None, stream=None) -> None:
    """Enqueue the log probabilities of `targets` (int32 or int64 [rows],
    negative: none; None without logp) under softmax(scale * logits), logits
    BF16 or fp32 [rows, vocab]; `lse` and `entropy` fp32 [rows], and the most
    probable tokens: top_ids int32, top_values fp32 [rows, top]."""
    import torch
    rows, vocab = logits.shape
    p, ty, stride = _wide(logits, rows, vocab, "logits")
    if logp is not None:
        _need(targets, "targets")
    t, tb = _targets(targets, rows)
    top = 0 if top_ids is None else top_ids.shape[-1]
    if (top_ids is None) != (top_values is None):
        raise ValueError("top_ids and top_values go together")
    f32, shape = torch.float32, (rows,)
    a, b, c = _array(logp, f32, shape, "logp"), _array(lse, f32, shape, "lse"), _array(entropy, f32, shape, "entropy")
    i, v = _array(top_ids, torch.int32, (rows, top), "top_ids"), _array(top_values, f32, (rows, top), "top_values")
    _step_space(workspace)
    dev = _one_device(logits, targets, logp, lse, entropy, top_ids, top_values, workspace)
    _fp4_call(torch, load_library().dcr_logprobs, "dcr_logprobs", dev, stream, p, ty, stride, rows, vocab, t, tb, scale, a, b,
              c, top, i, v, workspace.data_ptr(), workspace.nbytes)


def dcr_logprobs_grad(logits, targets, lse, dlogp, dlogits, entropy=None, dentropy=None, scale=1.0, stream=None) -> None:
    """Enqueue the gradient of dcr_logprobs's logp (and, with `dentropy`, its
    entropy) with respect to the logits; dlogits has the logits' type and may
    be the logits."""
    import torch
    rows, vocab = logits.shape
    p, ty, stride = _wide(logits, rows, vocab, "logits")
    d, dty, d_stride = _wide(dlogits, rows, vocab, "dlogits")
    if dty != ty:
        raise ValueError(f"dlogits: {logits.dtype} expected, got {dlogits.dtype}")
    if dentropy is not None:
        _need(entropy, "entropy")
    t, tb = _targets(_need(targets, "targets"), rows)
    f32, shape = torch.float32, (rows,)
    a, b = _array(_need(lse, "lse"), f32, shape, "lse"), _array(_need(dlogp, "dlogp"), f32, shape, "dlogp")
    c, e = _array(entropy, f32, shape, "entropy"), _array(dentropy, f32, shape, "dentropy")
    dev = _one_device(logits, targets, lse, dlogp, dlogits, entropy, dentropy)
    _fp4_call(torch, load_library().dcr_logprobs_grad, "dcr_logprobs_grad", dev, stream, p, ty, stride, rows, vocab, t, tb,
              scale, a, b, c, e, d, d_stride)


class AdamWDesc(ctypes.Structure):
    """dcr_adamw_tensor."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "m_scales", "v_scales", "copy")] + \
        [("numel", ctypes.c_uint64), ("first", ctypes.c_uint64)] + \
        [(n, ctypes.c_uint32) for n in ("param_type", "grad_type", "state_bits", "flags")]


class AdamWArgs(ctypes.Structure):
    """dcr_adamw_args."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] + \
        [("step", ctypes.c_uint64), ("live", ctypes.c_void_p), ("dither_seed", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class AdamWTensors:
    """The tensors that dcr_adamw_step updates, with their moments, and the
    plan of the step over them: addresses laid out once in device memory.

    `params` and `grads` are lists of contiguous BF16 or fp32 tensors (any
    shape).  `bits` 32: moments `m`, `v` in fp32; 8: float8_e4m3fn codes with
    uint8 `m_scales`, `v_scales` (one for each ADAMW_BLOCK elements), v by its
    square root.  Moments that are not given are made, zero.  `copies` (bf16,
    of fp32 parameters) receive the rounded parameters: the shards or canonical
    tensors that a refit compares.  `decay`: one truth value a tensor (default:
    all); `first`: the index of a tensor's first element to the dither, so
    that a shard is rounded as the whole tensor would be (default: one tensor
    behind the other).

    The buffers are kept, and the `live` tensors of captured steps; gradients are
    written into the same tensors step after step.  Steps may follow on any
    stream, one after the other; the object has to be there until they are done
    (and as long as a graph that has captured one)."""

    def __init__(self, params, grads, bits=32, copies=None, m=None, v=None, m_scales=None, v_scales=None, decay=None,
                 first=None):
        import torch
        if bits not in (8, 32):
            raise ValueError("bits is 8 or 32")
        n = len(params)
        if n == 0:
            raise ValueError("no tensors")
        types = {torch.float32: F32, torch.bfloat16: BF16}
        state = torch.float32 if bits == 32 else torch.float8_e4m3fn
        make = lambda t, ty, per: torch.zeros(-(-t.numel() // per), dtype=ty, device=t.device)  # noqa: E731
        self.bits, self.params, self.grads = bits, list(params), list(grads)
        self.live = []                   # what captured steps read
        self.copies = [None] * n if copies is None else list(copies)
        self.m = [make(p, state, 1) for p in params] if m is None else list(m)
        self.v = [make(p, state, 1) for p in params] if v is None else list(v)
        self.m_scales = self.v_scales = [None] * n
        if bits == 8:
            self.m_scales = [make(p, torch.uint8, ADAMW_BLOCK) for p in params] if m_scales is None else list(m_scales)
            self.v_scales = [make(p, torch.uint8, ADAMW_BLOCK) for p in params] if v_scales is None else list(v_scales)
        decay = [True] * n if decay is None else list(decay)
        if first is None:
            first = [0]
            for p in params:
                first.append(first[-1] + -(-p.numel() // ADAMW_BLOCK) * ADAMW_BLOCK)
            first = first[:-1]
        columns = (self.params, self.grads, self.m, self.v, self.m_scales, self.v_scales, self.copies, decay, first)
        if any(len(c) != n for c in columns):
            raise ValueError(f"{n} tensors: lists of that length expected")
        self.index = _one_device(self.params[0])
        descs = (AdamWDesc * n)()
        for i, (p, g, a, b, sa, sb, c, d, f) in enumerate(zip(*columns)):
            count = p.numel()
            for name, t, ty, size in (("params", p, None, count), ("grads", g, None, count), ("m", a, state, count),
                                      ("v", b, state, count), ("m_scales", sa, torch.uint8, -(-count // ADAMW_BLOCK)),
                                      ("v_scales", sb, torch.uint8, -(-count // ADAMW_BLOCK)),
                                      ("copies", c, torch.bfloat16, count)):
                if t is None and (name == "copies" or (bits == 32 and name.endswith("scales"))):
                    continue
                if t.numel() != size or not t.is_contiguous() or (t.dtype not in types if ty is None else t.dtype is not ty):
                    raise ValueError(f"{name}[{i}]: {size} contiguous elements of {ty or 'float32 or bfloat16'} expected, got "
                                     f"{t.dtype} {list(t.shape)}")
                if t.get_device() != self.index:
                    raise ValueError(f"tensors on different devices: cuda:{self.index} and {t.device}")
            at = lambda t: None if t is None or t.numel() == 0 else t.data_ptr()  # noqa: E731
            descs[i] = AdamWDesc(at(p), at(g), at(a), at(b), at(sa), at(sb), at(c), count, int(f), types[p.dtype],
                                 types[g.dtype], bits, 0 if d else ADAMW_NO_DECAY)
        lib = load_library()
        handle = ctypes.c_void_p()
        _check(lib.dcr_adamw_plan_build(ctypes.addressof(descs), n, ctypes.byref(handle)), "dcr_adamw_plan_build")
        self.handle = handle.value
        size = ctypes.c_uint64()
        _check(lib.dcr_adamw_plan_bytes(self.handle, ctypes.byref(size)), "dcr_adamw_plan_bytes")
        with torch.cuda.device(self.index):
            self.table = torch.empty(size.value, dtype=torch.uint8, device="cuda")
            _check(lib.dcr_adamw_plan_upload(self.handle, self.table.data_ptr(), size.value, _stream(None)),
                   "dcr_adamw_plan_upload")
            # (the first step may come on another stream)
            torch.cuda.current_stream().synchronize()

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.dcr_adamw_plan_destroy(h)


def _captures(device, stream):
    """Whether `stream`, or the GPU's current stream, is captured into a graph."""
    import torch
    with torch.cuda.device(device):
        if stream is None:
            return torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(_as_stream(stream, device)):
            return torch.cuda.is_current_stream_capturing()


def _as_stream(stream, device):
    """A torch stream of GPU `device` from one or from its handle."""
    import torch
    if isinstance(stream, torch.cuda.Stream):
        return stream
    raw = _stream(stream)
    return torch.cuda.ExternalStream(raw, device) if raw else torch.cuda.default_stream(device)


def dcr_adamw_step(tensors: AdamWTensors, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0,
                   dither=0, live=None, stream=None) -> None:
    """Enqueue step number `step` (1 upwards) of AdamW on all tensors.  `dither`:
    seed of the rounding of 8-bit moments (0: to nearest).  `live`: float64 [3]
    in device memory, the step number, lr and grad_scale that the GPU reads in
    place of those passed (for captured graphs: one that a captured step reads is kept
    by `tensors`)."""
    import torch
    if not 0 <= dither < 1 << 32:
        raise ValueError("dither: a seed below 2^32 expected")
    if live is None and not 1 <= step <= 1 << 53:
        raise ValueError("step: 1 upwards expected")
    if live is not None:
        _one_device(tensors.table, live)
        _array(live, torch.float64, (3,), "live")
    args = AdamWArgs(lr, beta1, beta2, eps, weight_decay, grad_scale, 0 if live is not None else int(step),
                     None if live is None else live.data_ptr(), dither, 0)
    _fp4_call(torch, load_library().dcr_adamw_step, "dcr_adamw_step", tensors.index, stream, tensors.handle,
              ctypes.addressof(args))
    if live is not None:
        if _captures(tensors.index, stream):
            tensors.live.append(live)
        elif stream is not None:         # (it may be gone before that stream has read it)
            live.record_stream(_as_stream(stream, tensors.index))


def dcr_set_kernel_events(start=None, stop=None) -> None:
    """Record start / stop (torch.cuda.Event, created, or raw hipEvent_t) around
    the main kernel of the following calls on this thread; None, None: off."""
    def h(e):
        if e is None:
            return None
        return int(e.cuda_event) if hasattr(e, "cuda_event") else int(e)
    load_library().dcr_set_kernel_events(h(start), h(stop))


def format_constants():
    out = (ctypes.c_uint32 * 10)()
    n = load_library().dcr_format_constants(out, 10)
    return list(out)[:n]


def _nbytes(t) -> int:
    if isinstance(t, np.ndarray):
        return int(t.nbytes)
    return int(t.numel() * t.element_size()) if hasattr(t, "numel") else 0


# ------------------------------------------------------- small conveniences

class StreamBuffers:
    """Device buffers of one stream (header, directory, payload, result)."""

    def __init__(self, plan: Plan, device="cuda", dir_bytes=None, payload_bytes=None):
        import torch
        self.header = torch.zeros(64, dtype=torch.uint8, device=device)
        self.dir = torch.empty(max(int(dir_bytes if dir_bytes is not None else plan.info.max_dir_bytes), 32),
                               dtype=torch.uint8, device=device)
        self.payload = torch.empty(max(int(payload_bytes if payload_bytes is not None
                                           else plan.info.max_payload_bytes), 16),
                                   dtype=torch.uint8, device=device)
        self.result = torch.zeros(32, dtype=torch.uint8, device=device)

    def header_host(self) -> np.ndarray:
        return self.header.cpu().numpy()

    def result_host(self):
        return np.frombuffer(self.result.cpu().numpy().tobytes(), dtype=ENCODE_RESULT)[0]

    def n_records(self) -> int:
        return int(self.result_host()["n_records"])

    def payload_bytes(self) -> int:
        return int(self.result_host()["payload_bytes"])


def workspace(plan: Plan, device="cuda", stage_bytes: int = 0):
    """Workspace of the plan's size plus an optional encode staging area."""
    import torch
    return torch.zeros(max(int(plan.info.workspace_bytes) + int(stage_bytes), 256), dtype=torch.uint8,
                       device=device)


def apply_result(t) -> np.void:
    return np.frombuffer(t.cpu().numpy().tobytes(), dtype=APPLY_RESULT)[0]
