"""Thin Python binding of librar.so (include/rar.h): argument marshalling only.

Every step of the collectives runs in the library's CUDA kernels. Torch
provides device memory (tensors) and streams; nothing here computes on data.
If the library is missing the binding raises -- there is no fallback path.
"""
import ctypes
import enum
import os
import struct
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "librar.so"
_lib = None


class Status(enum.IntEnum):
    OK = 0
    ERR_ARG = 1
    ERR_RING = 2
    ERR_ALIGN = 3
    ERR_WORKSPACE = 4
    ERR_CORESIDENCY = 5
    ERR_CUDA = 6
    ERR_TIMEOUT = 7
    ERR_ABORT = 8
    ERR_BOUNDS = 9
    ERR_CAPACITY = 10


class Dtype(enum.IntEnum):
    F32 = 0
    BF16 = 1


class Proto(enum.IntEnum):
    LL = 0
    LL128 = 1
    SIMPLE = 2


PROTO_BY_NAME = {"LL": Proto.LL, "LL128": Proto.LL128, "Simple": Proto.SIMPLE, "SIMPLE": Proto.SIMPLE}
EXPORTED = (
    "rar_workspace_bytes", "rar_workspace_init", "rar_allreduce", "rar_oneshot", "rar_get_status",
    "rar_strerror", "rar_set_spin_timeout_ns", "rar_debug_set_fault", "rar_describe_geometry",
    "rar_allreduce_static", "rar_allreduce_ex", "rar_reduce_scatter", "rar_all_gather",
    "rar_oneshot_workspace_bytes", "rar_oneshot_workspace_init", "rar_oneshot_staged",
    "rar_debug_set_ll_flag_wrap", "rar_op_workspace_init", "rar_page_tables", "rar_qk_norm_rope",
    "rar_qk_norm_rope_cached", "rar_qk_norm_rope_workspace_bytes", "rar_qk_norm_rope_backward",
    "rar_decode_attention_workspace_bytes", "rar_decode_attention", "rar_token_logprobs_workspace_bytes",
    "rar_token_logprobs", "rar_token_logprobs_backward",
)


class RarError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = Status(status)
        super().__init__(f"{what}: {self.status.name} ({strerror(self.status)})")


def library_path() -> str:
    """librar.so, or with RAR_LIBRARY=debug in the environment the debug build
    librar_debug.so (slice bounds checked on the device, RAR_ERR_BOUNDS)."""
    if os.environ.get("RAR_LIBRARY", "") == "debug":
        return os.path.join(HERE, "librar_debug.so")
    return os.path.join(HERE, _LIB_NAME)


def load_library():
    """Load librar.so (built in-tree by collective_communication_gb300/build.py)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python collective_communication_gb300/build.py` "
                           "(or __graft_entry__.build()); there is no fallback implementation")
    L = ctypes.CDLL(path)
    P, I, U64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
    L.rar_workspace_bytes.argtypes = [I, U64, I, SZ]
    L.rar_workspace_bytes.restype = SZ
    L.rar_workspace_init.argtypes = [P, SZ, I, U64, I, SZ, P]
    L.rar_workspace_init.restype = I
    L.rar_allreduce.argtypes = [P, P, I, SZ, I, I, P, U64, I, SZ, I, P, SZ, P]
    L.rar_allreduce.restype = I
    L.rar_oneshot.argtypes = [P, P, I, SZ, I, I, P]
    L.rar_oneshot.restype = I
    L.rar_get_status.argtypes = [P, P]
    L.rar_get_status.restype = I
    L.rar_strerror.argtypes = [I]
    L.rar_strerror.restype = ctypes.c_char_p
    L.rar_set_spin_timeout_ns.argtypes = [U64]
    L.rar_set_spin_timeout_ns.restype = None
    L.rar_debug_set_fault.argtypes = [I]
    L.rar_debug_set_fault.restype = None
    L.rar_describe_geometry.argtypes = [I, SZ, I, U64, I, SZ, I, P]
    L.rar_describe_geometry.restype = I
    L.rar_allreduce_static.argtypes = [P, P, I, SZ, I, I, P, U64, I, SZ, I, P]
    L.rar_allreduce_static.restype = I
    L.rar_allreduce_ex.argtypes = [P, P, I, SZ, I, I, P, I, U64, I, SZ, I, ctypes.c_uint, P, SZ, P]
    L.rar_allreduce_ex.restype = I
    L.rar_reduce_scatter.argtypes = [P, P, I, SZ, I, I, P, I, U64, I, SZ, I, ctypes.c_uint, P, SZ, P]
    L.rar_reduce_scatter.restype = I
    L.rar_all_gather.argtypes = [P, P, I, SZ, I, P, I, U64, I, SZ, I, ctypes.c_uint, P, SZ, P]
    L.rar_all_gather.restype = I
    L.rar_oneshot_workspace_bytes.argtypes = [I, SZ, I]
    L.rar_oneshot_workspace_bytes.restype = SZ
    L.rar_oneshot_workspace_init.argtypes = [P, SZ, I, SZ, I, P]
    L.rar_oneshot_workspace_init.restype = I
    L.rar_oneshot_staged.argtypes = [P, P, I, SZ, I, I, P, SZ, P]
    L.rar_oneshot_staged.restype = I
    L.rar_debug_set_ll_flag_wrap.argtypes = [ctypes.c_uint32]
    L.rar_debug_set_ll_flag_wrap.restype = I
    I64, F = ctypes.c_int64, ctypes.c_float
    L.rar_op_workspace_init.argtypes = [P, SZ, P]
    L.rar_page_tables.argtypes = [P, P, I, P, I, P, I, I, P, I64, I, P, P, P, P, I, P, P, SZ, P]
    rope = [P, I, I64, I64, P, P, P, I, I, I, P]
    heads = [I, I, I, I, F]
    L.rar_qk_norm_rope.argtypes = rope + heads + [P, I64, P, I64, P, SZ, P]
    L.rar_qk_norm_rope_cached.argtypes = rope + [P] + heads + [P, I64, P, P, I, I, P, SZ, P]
    L.rar_qk_norm_rope_backward.argtypes = rope + heads + [P, I64, P, I64, P, I64, P, I64, P, P, P, SZ, P]
    L.rar_qk_norm_rope_workspace_bytes.argtypes = [I, I]
    L.rar_decode_attention_workspace_bytes.argtypes = [I, I, I, I, I]
    L.rar_decode_attention.argtypes = [P, I64, P, P, I, I, I, I, I, I, I, I, P, I64, I, P, F, P, I64, P, P, SZ, P]
    L.rar_token_logprobs_workspace_bytes.argtypes = [I64, I]
    L.rar_token_logprobs.argtypes = [P, P, P, I, I64, I, P, P, P, P, I, P, P, P, SZ, P]
    L.rar_token_logprobs_backward.argtypes = [P, P, P, I, I64, I, P, P, P, P, P, P, P, P, SZ, P]
    for name in ("rar_qk_norm_rope_workspace_bytes", "rar_decode_attention_workspace_bytes",
                 "rar_token_logprobs_workspace_bytes"):
        getattr(L, name).restype = SZ
    for name in ("rar_op_workspace_init", "rar_page_tables", "rar_qk_norm_rope", "rar_qk_norm_rope_cached",
                 "rar_qk_norm_rope_backward", "rar_decode_attention", "rar_token_logprobs",
                 "rar_token_logprobs_backward"):
        getattr(L, name).restype = I
    _lib = L
    return L


def strerror(status) -> str:
    return load_library().rar_strerror(int(status)).decode()


def _check(st, what):
    if st != 0:
        raise RarError(st, what)


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_of(t) -> Dtype:
    import torch
    if t.dtype == torch.float32:
        return Dtype.F32
    if t.dtype == torch.bfloat16:
        return Dtype.BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptrs(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _proto(p) -> Proto:
    return PROTO_BY_NAME[p] if isinstance(p, str) else Proto(p)


def workspace_bytes(nranks: int, mask: int, proto, buff_size: int = 0) -> int:
    return int(load_library().rar_workspace_bytes(nranks, mask, int(_proto(proto)), buff_size))


class Workspace:
    """Device workspace (connector FIFOs and step counters) for one (nranks,
    channel mask, protocol, buffer size) configuration, held in a torch
    uint8 tensor and initialised through rar_workspace_init."""

    def __init__(self, nranks: int, mask: int, proto, buff_size: int = 0, device=None, stream=None):
        import torch
        self.nranks, self.mask, self.proto, self.buff_size = nranks, mask, _proto(proto), buff_size
        nbytes = workspace_bytes(nranks, mask, self.proto, buff_size)
        if nbytes == 0:
            raise RarError(Status.ERR_ARG, "rar_workspace_bytes")
        self.nbytes = nbytes
        self.tensor = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
        self.init(stream)

    @property
    def ptr(self) -> int:
        return self.tensor.data_ptr()

    def init(self, stream=None):
        _check(load_library().rar_workspace_init(self.ptr, self.nbytes, self.nranks, self.mask, int(self.proto),
                                                 self.buff_size, _stream_handle(stream)), "rar_workspace_init")


def allreduce(sendbufs: Sequence, recvbufs: Sequence, ring_order: Sequence[int], mask: int, proto,
              workspace: Workspace, buff_size: int = 0, chunk_steps: int = 4, stream=None) -> None:
    """Enqueue one ring AllReduce (sum) over len(sendbufs) virtual ranks."""
    n = len(sendbufs)
    count = sendbufs[0].numel()
    ring = (ctypes.c_int * n)(*ring_order)
    st = load_library().rar_allreduce(_ptrs(sendbufs), _ptrs(recvbufs), n, count, int(_dtype_of(sendbufs[0])), 0,
                                      ring, mask, int(_proto(proto)), buff_size, chunk_steps, workspace.ptr,
                                      workspace.nbytes, _stream_handle(stream))
    _check(st, "rar_allreduce")


FLAG_DIRECT = 1


def _ring_array(ring_orders):
    """(C array, nrings) for one ring order (a list of ranks) or one per channel."""
    rings = [list(r) for r in ring_orders] if isinstance(ring_orders[0], (list, tuple)) else [list(ring_orders)]
    flat = [int(v) for r in rings for v in r]
    return (ctypes.c_int * len(flat))(*flat), len(rings)


def allreduce_ex(sendbufs: Sequence, recvbufs: Sequence, ring_orders, mask: int, proto, workspace: Workspace,
                 buff_size: int = 0, chunk_steps: int = 4, direct: bool = False, stream=None) -> None:
    """Enqueue one ring AllReduce with one ring order (a list of ranks) or one
    per channel (a list of lists), optionally with direct all-gather writes."""
    n = len(sendbufs)
    ring_arr, nrings = _ring_array(ring_orders)
    st = load_library().rar_allreduce_ex(_ptrs(sendbufs), _ptrs(recvbufs), n, sendbufs[0].numel(),
                                         int(_dtype_of(sendbufs[0])), 0, ring_arr, nrings, mask,
                                         int(_proto(proto)), buff_size, chunk_steps, FLAG_DIRECT if direct else 0,
                                         workspace.ptr, workspace.nbytes, _stream_handle(stream))
    _check(st, "rar_allreduce_ex")


def reduce_scatter(sendbufs: Sequence, recvbufs: Sequence, ring_orders, mask: int, proto, workspace: Workspace,
                   buff_size: int = 0, chunk_steps: int = 4, stream=None) -> None:
    """Enqueue one ring ReduceScatter (sum): sendbufs[r] holds nranks blocks of
    recvbufs[r].numel() elements; recvbufs[r] receives block r reduced."""
    n = len(sendbufs)
    ring_arr, nrings = _ring_array(ring_orders)
    st = load_library().rar_reduce_scatter(_ptrs(sendbufs), _ptrs(recvbufs), n, recvbufs[0].numel(),
                                           int(_dtype_of(sendbufs[0])), 0, ring_arr, nrings, mask,
                                           int(_proto(proto)), buff_size, chunk_steps, 0,
                                           workspace.ptr, workspace.nbytes, _stream_handle(stream))
    _check(st, "rar_reduce_scatter")


def all_gather(sendbufs: Sequence, recvbufs: Sequence, ring_orders, mask: int, proto, workspace: Workspace,
               buff_size: int = 0, chunk_steps: int = 4, direct: bool = False, stream=None) -> None:
    """Enqueue one ring AllGather: recvbufs[r] (nranks blocks) receives every
    rank's sendbufs[b] as block b."""
    n = len(sendbufs)
    ring_arr, nrings = _ring_array(ring_orders)
    st = load_library().rar_all_gather(_ptrs(sendbufs), _ptrs(recvbufs), n, sendbufs[0].numel(),
                                       int(_dtype_of(sendbufs[0])), ring_arr, nrings, mask, int(_proto(proto)),
                                       buff_size, chunk_steps, FLAG_DIRECT if direct else 0,
                                       workspace.ptr, workspace.nbytes, _stream_handle(stream))
    _check(st, "rar_all_gather")


def allreduce_raw(send_ptrs, recv_ptrs, nranks, count, dtype, ring_order, mask, proto, buff_size, chunk_steps,
                  ws_ptr, ws_bytes, stream_handle) -> int:
    """Direct C-ABI call with raw pointers; returns the status code."""
    ring = (ctypes.c_int * len(ring_order))(*ring_order)
    sp = (ctypes.c_void_p * len(send_ptrs))(*send_ptrs)
    rp = (ctypes.c_void_p * len(recv_ptrs))(*recv_ptrs)
    return int(load_library().rar_allreduce(sp, rp, nranks, count, int(dtype), 0, ring, mask, int(_proto(proto)),
                                            buff_size, chunk_steps, ws_ptr, ws_bytes, stream_handle))


def oneshot(sendbufs: Sequence, recvbufs: Sequence, stream=None) -> None:
    """Enqueue one one-shot AllReduce (sum) over len(sendbufs) virtual ranks."""
    n = len(sendbufs)
    st = load_library().rar_oneshot(_ptrs(sendbufs), _ptrs(recvbufs), n, sendbufs[0].numel(),
                                    int(_dtype_of(sendbufs[0])), 0, _stream_handle(stream))
    _check(st, "rar_oneshot")


class OneShotWorkspace:
    """Device workspace of the staged one-shot (torch-allocated, 256-byte
    aligned), initialised for calls of up to max_count elements."""

    def __init__(self, nranks: int, max_count: int, dtype, device=None, stream=None):
        import torch
        if dtype in ("f32", "bf16"):
            dt = Dtype.F32 if dtype == "f32" else Dtype.BF16
        elif isinstance(dtype, torch.dtype):
            dt = Dtype.F32 if dtype == torch.float32 else Dtype.BF16 if dtype == torch.bfloat16 else None
        else:
            dt = Dtype(dtype)
        if dt is None:
            raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
        self.nbytes = int(load_library().rar_oneshot_workspace_bytes(nranks, max_count, int(dt)))
        if self.nbytes == 0:
            raise RarError(Status.ERR_ARG, "rar_oneshot_workspace_bytes")
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        base = self.buf.data_ptr()
        self._ptr = (base + 255) // 256 * 256
        self.nranks, self.max_count, self.dtype = nranks, max_count, dt
        self.init(stream)

    def init(self, stream=None):
        """(Re-)initialise: zero the counters, record the configuration."""
        _check(load_library().rar_oneshot_workspace_init(self._ptr, self.nbytes, self.nranks, self.max_count,
                                                          int(self.dtype), _stream_handle(stream)),
               "rar_oneshot_workspace_init")

    @property
    def ptr(self) -> int:
        return self._ptr


def oneshot_staged(sendbufs: Sequence, recvbufs: Sequence, workspace: OneShotWorkspace, stream=None) -> None:
    """Enqueue one staged one-shot AllReduce (sum) over len(sendbufs) ranks."""
    n = len(sendbufs)
    st = load_library().rar_oneshot_staged(_ptrs(sendbufs), _ptrs(recvbufs), n, sendbufs[0].numel(),
                                           int(_dtype_of(sendbufs[0])), 0, workspace.ptr, workspace.nbytes,
                                           _stream_handle(stream))
    _check(st, "rar_oneshot_staged")


# ---- operators of a tensor-parallel step (heads and vocabulary split over the virtual ranks) ----
# A per-rank argument is a sequence of nranks alike tensors, or one tensor whose
# first dimension is the rank.

OP_WORKSPACE_MIN_BYTES = 36864


class OpWorkspace:
    """Device workspace of the operators: the status word, arrival counters and
    scratch. One serves any of them, ordered on one stream; nbytes is the
    largest of their *_workspace_bytes (0: the minimum, enough for those
    without one)."""

    def __init__(self, nbytes: int = 0, device=None, stream=None):
        import torch
        self.nbytes = max(int(nbytes), OP_WORKSPACE_MIN_BYTES)
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        self.ptr = (self.buf.data_ptr() + 255) // 256 * 256
        self.init(stream)

    def init(self, stream=None):
        """(Re-)initialise: clear the status word and the counters."""
        _check(load_library().rar_op_workspace_init(self.ptr, self.nbytes, _stream_handle(stream)),
               "rar_op_workspace_init")


def _op_bytes(fn, *args) -> int:
    n = int(getattr(load_library(), fn)(*args))
    if n == 0:
        raise RarError(Status.ERR_ARG, fn)
    return n


def qk_norm_rope_workspace_bytes(nranks: int, head_dim: int) -> int:
    """Workspace of qk_norm_rope_backward."""
    return _op_bytes("rar_qk_norm_rope_workspace_bytes", nranks, head_dim)


def decode_attention_workspace_bytes(nranks: int, batch: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return _op_bytes("rar_decode_attention_workspace_bytes", nranks, batch, q_heads, kv_heads, head_dim)


def token_logprobs_workspace_bytes(rows: int, top: int) -> int:
    return _op_bytes("rar_token_logprobs_workspace_bytes", rows, top)


# A decode step makes these calls once a layer, so their checks are written for
# few Python operations: _op_setup binds once what each call needs of torch.
_ops = None


def _op_setup():
    global _ops, _INT32, _FLOAT32, _OP_DTYPES, _raw_stream, _current_device
    import torch
    _INT32, _FLOAT32 = torch.int32, torch.float32
    _OP_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
    if torch.cuda.is_available():
        torch.cuda.init()
        _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _ops = load_library()
    return _ops


def _op_stream(stream) -> int:
    return _raw_stream(_current_device()) if stream is None else _stream_handle(stream)


def _op_dtype(dtype) -> int:
    """The C ABI's number of an operator's dtype."""
    d = _OP_DTYPES.get(dtype)
    if d is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return d


def _refuse(what):
    raise RarError(Status.ERR_ARG, what)


_PACKS = {n: struct.Struct(f"{n}Q").pack for n in range(1, 33)}


_PACK1 = _PACKS[1]


def _pack(values):
    """nranks pointers, or 64-bit counts, as a C array."""
    n = len(values)
    return _PACKS[n](*values) if n in _PACKS else struct.pack(f"{n}Q", *values)


def _ranked(x, name, dims):
    """A per-rank argument as (C array of the ranks' pointers, shape with the
    rank first, row stride of a rank's tensor, dtype); the dimensions after a
    row's are dense."""
    if type(x) is list or type(x) is tuple:
        return _ranked_list(x, name, dims)
    full = x.shape
    n = full[0]
    if len(full) != dims + 1 or not x.is_cuda or n == 0:
        _refuse(f"{name}: {dims} dimensions a rank, in device memory")
    if not x.is_contiguous():
        return _ranked_list(x.unbind(0), name, dims)
    if dims == 3:
        width = full[2] * full[3]
    else:
        width = 1 if dims == 1 else full[2] if dims == 2 else full[2] * full[3] * full[4]
    base, step = x.data_ptr(), x.nbytes // n
    if n == 1:
        ptrs = _PACK1(base)
    elif step and n <= 32:
        ptrs = _PACKS[n](*range(base, base + n * step, step))
    else:
        ptrs = _pack((base,) * n)
    return ptrs, full, width, x.dtype


def _ranked_list(x, name, dims):
    first = x[0]
    shape, strides, dtype = first.shape, first.stride(), first.dtype
    for t in x:
        if t.shape != shape or t.stride() != strides or t.dtype is not dtype or not t.is_cuda:
            _refuse(f"{name}: the ranks' tensors are alike and in device memory")
    if len(shape) != dims:
        _refuse(f"{name}: {dims} dimensions a rank")
    width = 1
    for i in range(dims - 1, 0, -1):
        if shape[i] != 1 and strides[i] != width:
            _refuse(f"{name}: dense after its first dimension")
        width *= shape[i]
    return _pack([t.data_ptr() for t in x]), (len(x), *shape), strides[0] if shape[0] > 1 else width, dtype


def _ranked_dense(x, name, dims):
    """_ranked of tensors without gaps."""
    r = _ranked(x, name, dims)
    if type(x) is list or type(x) is tuple:
        if not all(t.is_contiguous() for t in x):
            _refuse(f"{name}: contiguous")
    elif not x.is_contiguous():
        _ranked_dense(x.unbind(0), name, dims)
    return r


def _ints(t, name, numel):
    if t.dtype is not _INT32 or t.numel() != numel or not t.is_contiguous() or not t.is_cuda:
        _refuse(f"{name}: {numel} contiguous int32 in device memory")
    return t.data_ptr()


def _floats(t, name, numel):
    if t.dtype is not _FLOAT32 or t.numel() != numel or not t.is_contiguous() or not t.is_cuda:
        _refuse(f"{name}: {numel} contiguous float32 in device memory")
    return t.data_ptr()


def _table(t, rows):
    """(pointer, row stride, columns) of a block table."""
    shape = t.shape
    if t.dtype is not _INT32 or len(shape) != 2 or shape[0] != rows or not t.is_cuda:
        _refuse("block_table: int32 [requests, max_blocks] in device memory")
    blocks = shape[1]
    if t.is_contiguous():
        return t.data_ptr(), blocks, blocks
    if blocks != 1 and t.stride(1) != 1:
        _refuse("block_table: dense rows")
    return t.data_ptr(), t.stride(0) if rows > 1 else blocks, blocks


def page_tables(lens, new_tokens, free_pages, free_count, block_table, page_size: int, num_pages: int, lens_out, starts,
                positions, slots, free_count_out, workspace: OpWorkspace, stream=None) -> None:
    """Enqueue one step's page tables and slot maps, from the requests' lengths
    (int32 tensors): new entries of block_table [requests, max_blocks] in place,
    lens_out, starts [requests + 1], positions and slots [most tokens of a
    step], free_count_out [1]."""
    lib = _ops or _op_setup()
    n, tokens, free = lens.numel(), slots.numel(), free_pages.numel()
    table, stride, blocks = _table(block_table, n)
    st = lib.rar_page_tables(
        _ints(lens, "lens", n), _ints(new_tokens, "new_tokens", n), n, _ints(free_pages, "free_pages", free), free,
        _ints(free_count, "free_count", 1), page_size, num_pages, table, stride, blocks,
        _ints(lens_out, "lens_out", n), _ints(starts, "starts", n + 1), _ints(positions, "positions", tokens),
        _ints(slots, "slots", tokens), tokens, _ints(free_count_out, "free_count_out", 1), workspace.ptr,
        workspace.nbytes, _op_stream(stream))
    if st:
        _check(st, "rar_page_tables")


def _rope_call(qkv, q_weight, k_weight, cos_sin, positions, q, kv_heads):
    """What the forms of the norm and rotation share: qkv [tokens, (q + 2 kv
    heads) * head_dim] against queries [tokens, q_heads, head_dim]."""
    n, tokens, q_heads, dim = q[1]
    dtype = qkv[3]
    if q[3] is not dtype or qkv[1] != (n, tokens, (q_heads + 2 * kv_heads) * dim):
        _refuse("qkv: [tokens, (q_heads + 2 kv_heads) head_dim], queries [tokens, q_heads, head_dim], of one dtype")
    if q_weight.dtype is not dtype or k_weight.dtype is not dtype or q_weight.numel() != dim \
            or k_weight.numel() != dim or not q_weight.is_contiguous() or not k_weight.is_contiguous() \
            or not q_weight.is_cuda or not k_weight.is_cuda:
        _refuse("weights: head_dim contiguous elements of qkv's dtype in device memory")
    max_pos, rot = cos_sin.shape
    if cos_sin.dtype is not _FLOAT32 or not cos_sin.is_contiguous() or not cos_sin.is_cuda:
        _refuse("cos_sin: contiguous float32 [max_pos, rot_dim] in device memory")
    return (qkv[0], n, tokens, qkv[2], q_weight.data_ptr(), k_weight.data_ptr(), cos_sin.data_ptr(), max_pos, rot), \
        _ints(positions, "positions", tokens), (q_heads, kv_heads, dim, _op_dtype(dtype))


def qk_norm_rope(qkv, q_weight, k_weight, cos_sin, positions, q_out, k_out, workspace: OpWorkspace, eps: float = 1e-6,
                 interleaved: bool = False, stream=None) -> None:
    """Enqueue the norm and rotation of every rank's queries and keys: q_out
    [tokens, q_heads, head_dim] and k_out [tokens, kv_heads, head_dim] a rank."""
    lib = _ops or _op_setup()
    q, k = _ranked(q_out, "q_out", 3), _ranked(k_out, "k_out", 3)
    head, pos, heads = _rope_call(_ranked(qkv, "qkv", 2), q_weight, k_weight, cos_sin, positions, q, k[1][2])
    if k[3] is not q[3] or k[1] != (*q[1][:2], heads[1], heads[2]):
        _refuse("k_out: [tokens, kv_heads, head_dim]")
    st = lib.rar_qk_norm_rope(*head, interleaved, pos, *heads, eps, q[0], q[2], k[0], k[2], workspace.ptr,
                              workspace.nbytes, _op_stream(stream))
    if st:
        _check(st, "rar_qk_norm_rope")


def qk_norm_rope_cached(qkv, q_weight, k_weight, cos_sin, positions, slots, q_out, k_cache, v_cache,
                        workspace: OpWorkspace, eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """Enqueue the norm and rotation, keys and values into the paged caches
    [num_pages, kv_heads, page_size, head_dim] a rank at slots."""
    lib = _ops or _op_setup()
    q = _ranked(q_out, "q_out", 3)
    k, v = _ranked_dense(k_cache, "k_cache", 4), _ranked_dense(v_cache, "v_cache", 4)
    n, pages, kv_heads, page, dim = k[1]
    head, pos, heads = _rope_call(_ranked(qkv, "qkv", 2), q_weight, k_weight, cos_sin, positions, q, kv_heads)
    if n != head[1] or v[1] != k[1] or k[3] is not q[3] or v[3] is not q[3] or dim != heads[2]:
        _refuse("k_cache, v_cache: [num_pages, kv_heads, page_size, head_dim]")
    st = lib.rar_qk_norm_rope_cached(*head, interleaved, pos, _ints(slots, "slots", head[2]), *heads, eps, q[0], q[2],
                                     k[0], v[0], pages, page, workspace.ptr, workspace.nbytes, _op_stream(stream))
    if st:
        _check(st, "rar_qk_norm_rope_cached")


def qk_norm_rope_backward(qkv, q_weight, k_weight, cos_sin, positions, dq, dk, dv, dqkv, dq_weight, dk_weight,
                          workspace: OpWorkspace, eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """Enqueue the gradient: dqkv (as qkv) and float32 dq_weight, dk_weight
    [head_dim] a rank from dq [tokens, q_heads, head_dim], dk and dv [tokens,
    kv_heads, head_dim]."""
    lib = _ops or _op_setup()
    q, k, v = _ranked(dq, "dq", 3), _ranked(dk, "dk", 3), _ranked(dv, "dv", 3)
    x, d = _ranked(qkv, "qkv", 2), _ranked(dqkv, "dqkv", 2)
    head, pos, heads = _rope_call(x, q_weight, k_weight, cos_sin, positions, q, k[1][2])
    if k[3] is not q[3] or v[3] is not q[3] or v[1] != k[1] or k[1] != (*q[1][:2], heads[1], heads[2]):
        _refuse("dk, dv: [tokens, kv_heads, head_dim]")
    if d[1] != x[1] or d[3] is not x[3]:
        _refuse("dqkv: as qkv")
    wq, wk = _ranked(dq_weight, "dq_weight", 1), _ranked(dk_weight, "dk_weight", 1)
    for w in (wq, wk):
        if w[1] != (head[1], heads[2]) or w[3] is not _FLOAT32 or w[2] != 1:
            _refuse("dq_weight, dk_weight: float32 [head_dim]")
    st = lib.rar_qk_norm_rope_backward(*head, interleaved, pos, *heads, eps, q[0], q[2], k[0], k[2], v[0], v[2], d[0],
                                       d[2], wq[0], wk[0], workspace.ptr, workspace.nbytes, _op_stream(stream))
    if st:
        _check(st, "rar_qk_norm_rope_backward")


def decode_attention(q, k_cache, v_cache, block_table, lens, out, lse, workspace: OpWorkspace,
                     scale: Optional[float] = None, stream=None) -> None:
    """Enqueue attention of one new token per request: q, out [batch, q_heads,
    head_dim] a rank, caches as qk_norm_rope_cached writes them, int32
    block_table [batch, max_blocks] and lens [batch]; lse float32 [batch,
    q_heads] a rank, or None. scale: head_dim ** -0.5 by default."""
    lib = _ops or _op_setup()
    x, o = _ranked(q, "q", 3), _ranked(out, "out", 3)
    k, v = _ranked_dense(k_cache, "k_cache", 4), _ranked_dense(v_cache, "v_cache", 4)
    dtype = x[3]
    n, batch, q_heads, dim = x[1]
    kn, pages, kv_heads, page, kdim = k[1]
    if kn != n or kdim != dim or v[1] != k[1] or o[1] != x[1] or k[3] is not dtype or v[3] is not dtype \
            or o[3] is not dtype:
        _refuse("q, out: [batch, q_heads, head_dim]; caches: [num_pages, kv_heads, page_size, head_dim]")
    table, stride, blocks = _table(block_table, batch)
    lse_p = None
    if lse is not None:
        e = _ranked_dense(lse, "lse", 2)
        if e[1] != (n, batch, q_heads) or e[3] is not _FLOAT32:
            _refuse("lse: float32 [batch, q_heads]")
        lse_p = e[0]
    st = lib.rar_decode_attention(
        x[0], x[2], k[0], v[0], n, batch, q_heads, kv_heads, dim, _op_dtype(dtype), pages, page, table, stride, blocks,
        _ints(lens, "lens", batch), dim ** -0.5 if scale is None else scale, o[0], o[2], lse_p, workspace.ptr,
        workspace.nbytes, _op_stream(stream))
    if st:
        _check(st, "rar_decode_attention")


def _shards(x, name):
    """(pointers, vocabulary of each shard, row strides, nranks, rows, dtype); shards may differ in width."""
    if type(x) is not list and type(x) is not tuple:
        p, (n, rows, width), stride, dtype = _ranked(x, name, 2)
        return p, _pack((width,) * n), _pack((stride,) * n), n, rows, dtype
    ones = [_ranked_list((t,), name, 2) for t in x]
    rows, dtype = ones[0][1][1], ones[0][3]
    for o in ones:
        if o[1][1] != rows or o[3] is not dtype:
            _refuse(f"{name}: [rows, vocabulary of the shard], of one dtype")
    return (b"".join([o[0] for o in ones]), _pack([o[1][2] for o in ones]), _pack([o[2] for o in ones]), len(ones), rows,
            dtype)


def token_logprobs(logits, tokens, logprob, entropy, lse, top_values, top_ids, workspace: OpWorkspace,
                   stream=None) -> None:
    """Enqueue log probabilities of int32 tokens [rows] over vocabulary shards
    logits [rows, shard] a rank: float32 logprob, entropy, lse [rows] and the top
    alternatives' float32 top_values and int32 top_ids [rows, top] (None, or top
    0: none)."""
    lib = _ops or _op_setup()
    p, vocab, strides, n, rows, dtype = _shards(logits, "logits")
    top = 0 if top_ids is None else top_ids.shape[1]
    values_p = ids_p = None
    if top:
        values_p = _floats(top_values, "top_values", rows * top)
        ids_p = _ints(top_ids, "top_ids", rows * top)
    st = lib.rar_token_logprobs(
        p, vocab, strides, n, rows, _op_dtype(dtype), _ints(tokens, "tokens", rows), _floats(logprob, "logprob", rows),
        _floats(entropy, "entropy", rows), _floats(lse, "lse", rows), top, values_p, ids_p, workspace.ptr,
        workspace.nbytes, _op_stream(stream))
    if st:
        _check(st, "rar_token_logprobs")


def token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob, grad_entropy, dlogits, workspace: OpWorkspace,
                            stream=None) -> None:
    """Enqueue the gradient with respect to the logits, from lse and entropy of
    token_logprobs and float32 gradients [rows] (grad_entropy None: no such
    term); dlogits as logits (in place is allowed)."""
    lib = _ops or _op_setup()
    p, vocab, strides, n, rows, dtype = _shards(logits, "logits")
    dp, dvocab, dstrides, dn, drows, ddtype = _shards(dlogits, "dlogits")
    if dn != n or drows != rows or ddtype is not dtype or dvocab != vocab:
        _refuse("dlogits: as logits")
    st = lib.rar_token_logprobs_backward(
        p, vocab, strides, n, rows, _op_dtype(dtype), _ints(tokens, "tokens", rows), _floats(lse, "lse", rows),
        _floats(entropy, "entropy", rows), _floats(grad_logprob, "grad_logprob", rows),
        None if grad_entropy is None else _floats(grad_entropy, "grad_entropy", rows), dp, dstrides, workspace.ptr,
        workspace.nbytes, _op_stream(stream))
    if st:
        _check(st, "rar_token_logprobs_backward")


def get_status(workspace, stream=None) -> Status:
    return Status(load_library().rar_get_status(workspace.ptr, _stream_handle(stream)))


def set_spin_timeout_ns(ns: int) -> None:
    load_library().rar_set_spin_timeout_ns(ns)


def debug_set_fault(fault: int) -> None:
    load_library().rar_debug_set_fault(fault)


def debug_set_ll_flag_wrap(flag_max: int) -> None:
    """LL flag test mode: 0 = production flags, else the wrap period (a power
    of two >= 64) with the slot cleanup."""
    _check(load_library().rar_debug_set_ll_flag_wrap(flag_max), "rar_debug_set_ll_flag_wrap")


def describe_geometry(nranks, count, dtype, mask, proto, buff_size=0, chunk_steps=4):
    """The library's own geometry for a call (host computation, no device work)."""
    import numpy as np
    c = bin(mask).count("1")
    out = np.zeros(6 + 4 * max(c, 1), np.int64)
    st = load_library().rar_describe_geometry(nranks, count, int(dtype), mask, int(_proto(proto)), buff_size,
                                              chunk_steps, out.ctypes.data_as(ctypes.c_void_p))
    _check(st, "rar_describe_geometry")
    C = int(out[4])
    return {
        "step_bytes": int(out[0]),
        "chunk_elems": int(out[1]),
        "steps_per_slice": int(out[2]),
        "slices_per_chunk": int(out[3]),
        "nchannels": C,
        "per_channel": int(out[5]),
        "channel_ids": out[6:6 + C].tolist(),
        "channels": [(int(out[6 + C + 2 * i]), int(out[6 + C + 2 * i + 1])) for i in range(C)],
        "loops": out[6 + 3 * C:6 + 4 * C].tolist(),
    }
