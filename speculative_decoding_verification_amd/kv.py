"""Key-value cache of a verification round: buffers and calls of sv_kv_*.

Argument marshalling only, as in the package's other calls: KvCache owns (or
adopts) a cache's device buffers and passes them, with the call's tensors and
the current stream of the cache's device, to the C call of the same name.
Tensors are checked for their type, shape, device and contiguity, and
SpecVerifyError is raised before anything is enqueued.

One cycle of a sequence, nothing of it decided on the host:

    kv.reserve(M)                        pages for the M rows of the round
    for each layer:
        kv.append(layer, k, v, rope=r)   the rows' keys and values
        attn.run(layer, q, out, rope=r)  attn = kv.attention(q_heads, B, M)
    sv.accept_greedy(..., out)
    kv.commit(M, out)                    keeps the accepted rows
"""

from __future__ import annotations

import ctypes
import math


def _sv():
    import speculative_decoding_verification_amd as sv
    return sv


def _bad(msg, code=-1):
    return _sv().SpecVerifyError(code, msg)


_BUFFERS = ("data", "table", "len", "refs", "free_ids", "ctl")


def kv_page_bytes(type: int, heads: int, dim: int, page: int) -> int:
    return int(_sv().lib().sv_kv_page_bytes(type, heads, dim, page))


def rope_table(n_pos: int, rot: int, base: float = 10000.0, device="cuda"):
    """[n_pos, rot / 2, 2] fp32 cos and sin of position * base^(-2 i / rot),
    taken in 64 bits (a far position's angle loses its fraction in 32)."""
    import torch
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()


class Rope:
    """Rotary embedding of the first `rot` elements of a head: mode
    SV_ROPE_PAIRS or SV_ROPE_HALVES (SV_ROPE_NONE: no rotation), table
    [n_pos, rot / 2, 2] fp32 (see rope_table) with at least width * page
    rows."""

    def __init__(self, mode: int, rot: int, table):
        import torch
        if mode != 0:
            if table is None or table.dtype != torch.float32 or not table.is_contiguous() or table.ndim != 3 or \
                    table.shape[1] * 2 != rot or table.shape[2] != 2:
                raise _bad("rope: table must be contiguous float32 [n_pos, rot / 2, 2]")
        self.table = table
        self.device = table.device if mode != 0 else None
        self.c = _sv().KvRope(mode, rot, table.shape[0] if mode != 0 else 0, table.data_ptr() if mode != 0 else None)


class KvCache:
    """A pool of pages, the tables of `seqs` sequences and their lengths on
    one device.  type: SV_KV_F16, SV_KV_BF16 or SV_KV_I8; heads and dim of
    the keys and values; `page` slots per page (32, 64, 128 or 256); `width`
    page-table entries per sequence.  buffers: a dict of existing tensors to
    adopt (data uint8, the others int32) in place of new, emptied ones."""

    def __init__(self, type: int, layers: int, heads: int, dim: int, page: int, n_pages: int, seqs: int, width: int,
                 device=None, buffers=None):
        import torch
        sv = _sv()
        self._torch, self._lib = torch, sv.lib()
        self.type, self.layers, self.heads, self.dim, self.page = type, layers, heads, dim, page
        self.n_pages, self.seqs, self.width = n_pages, seqs, width
        self.c = sv.Kv(type, layers, heads, dim, page, n_pages, seqs, width)
        need = int(self._lib.sv_kv_data_bytes(ctypes.byref(self.c)))
        if need == 0:
            raise _bad("kv: unsupported cache type or shape", sv.SV_ERR_SHAPE)
        sizes = {"data": need, "table": seqs * width, "len": seqs, "refs": n_pages, "free_ids": n_pages, "ctl": 4}
        given = buffers is not None
        if not given:
            device = torch.device("cuda" if device is None else device)
            shapes = {"table": (seqs, width)}
            buffers = {n: torch.empty(shapes.get(n, (sizes[n],)), device=device,
                                      dtype=torch.uint8 if n == "data" else torch.int32) for n in _BUFFERS}
        self.device = buffers["data"].device
        for n in _BUFFERS:
            t = buffers[n]
            if t.dtype != (torch.uint8 if n == "data" else torch.int32) or not t.is_contiguous() or \
                    t.numel() < sizes[n] or t.device != self.device or not t.is_cuda:
                raise _bad(f"kv: {n} must be a contiguous {'uint8' if n == 'data' else 'int32'} GPU tensor of at "
                           f"least {sizes[n]} elements, on the device of the others")
            setattr(self, n if n != "len" else "lens", t)
            setattr(self.c, n, t.data_ptr())
        self._ref, self._index = ctypes.byref(self.c), self.device.index
        # the handle of the current stream, without a Stream object made for
        # it (0.1 against 1.9 us, of the 6 that a call takes on the host)
        self._current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        self._struct = sv.KvBatch
        self._compact_ws = None
        if not given:
            self.init()

    # ------------------------------------------------------------- helpers
    def _call(self, fn, *args, stream=None):
        """A C call on the cache's device and its current stream."""
        torch = self._torch
        if stream is None:
            stream = self._current(self._index)
        elif hasattr(stream, "cuda_stream"):
            stream = stream.cuda_stream
        if torch.cuda.current_device() == self._index:
            rc = fn(self._ref, *args, stream)
        else:
            with torch.cuda.device(self.device):
                rc = fn(self._ref, *args, stream)
        if rc:
            raise _sv().SpecVerifyError(rc, self._lib.sv_last_error().decode())

    def _tensor(self, t, name, dtype, shape=None):
        """The data pointer of a tensor of the call, checked; None for None."""
        if t is None:
            return None
        if t.dtype != dtype or t.get_device() != self._index or not t.is_contiguous() or \
                (shape is not None and t.shape != shape):
            raise _bad(f"kv: {name} must be a contiguous {dtype} tensor on {self.device}"
                       + (f" of shape {shape}" if shape is not None else ""))
        return t.data_ptr()

    def _batch(self, B, M, seq, n_new, tree=None):
        i32 = self._torch.int32
        return self._struct(B, M, self._tensor(seq, "seq", i32, (B,)), self._tensor(n_new, "n_new", i32, (B,)),
                            self._tensor(tree, "tree", i32, (B, M)))

    def _rope(self, rope):
        if rope is None:
            return None
        if rope.device is not None and rope.device != self.device:
            raise _bad(f"kv: the rope table must be on {self.device}")
        return ctypes.byref(rope.c)

    def _places(self, seq):
        return self.seqs if seq is None else seq.numel()

    # --------------------------------------------------------------- calls
    def init(self, stream=None):
        """Empties the cache (sv_kv_init)."""
        self._call(self._lib.sv_kv_init, stream=stream)

    def reserve(self, n: int, seq=None, n_new=None, stream=None):
        """Pages for the next n slots of sequences `seq` (int32 [B]; None:
        all of them); n_new int32 [B]: each one's own count, at most n."""
        b = self._batch(self._places(seq), n, seq, n_new)
        self._call(self._lib.sv_kv_reserve, ctypes.byref(b), stream=stream)

    def append(self, layer: int, k, v, seq=None, n_new=None, tree=None, rope=None, stream=None):
        """Writes rows k, v (fp32 [B, M, heads, dim]) to the slots past each
        sequence's length; tree int32 [B, M] masks."""
        B, M = k.shape[:2]
        f32 = self._torch.float32
        shape = (B, M, self.heads, self.dim)
        b = self._batch(B, M, seq, n_new, tree)
        self._call(self._lib.sv_kv_append, layer, ctypes.byref(b), self._tensor(k, "k", f32, shape),
                   self._tensor(v, "v", f32, shape), self._rope(rope), stream=stream)

    def read(self, layer: int, k_out=None, v_out=None, seq=None, n_new=None, start=None, stream=None):
        """Reads M slots of each sequence from start (int32 [B]; None: the
        sequence's length, the new rows) on into fp32 [B, M, heads, dim]."""
        one = k_out if k_out is not None else v_out
        if one is None:
            raise _bad("kv: read needs k_out or v_out")
        B, M = one.shape[:2]
        f32 = self._torch.float32
        shape = (B, M, self.heads, self.dim)
        b = self._batch(B, M, seq, n_new)
        self._call(self._lib.sv_kv_read, layer, ctypes.byref(b), self._tensor(start, "start", self._torch.int32, (B,)),
                   self._tensor(k_out, "k_out", f32, shape), self._tensor(v_out, "v_out", f32, shape), stream=stream)

    def commit(self, M: int, accepted, seq=None, n_new=None, path=None, stream=None):
        """Ends a round of M rows: accepted int32 [B], or [B, n] with the
        counts in column 0 (the outputs of the acceptance calls; [n] for
        one sequence); path int32 [B, M]: the rows kept, or None."""
        B = self._places(seq) if path is None else path.shape[0]
        if accepted.ndim < 2 and accepted.numel() != B and B != 1:
            raise _bad(f"kv: accepted must hold {B} counts")
        if accepted.ndim > 2 or (accepted.ndim == 2 and accepted.shape[0] != B) or accepted.numel() < 1:
            raise _bad(f"kv: accepted must be [{B}] or [{B}, n]")
        stride = accepted.shape[1] if accepted.ndim == 2 else 1
        i32 = self._torch.int32
        b = self._batch(B, M, seq, n_new)
        self._call(self._lib.sv_kv_commit, ctypes.byref(b), self._tensor(accepted, "accepted", i32), stride,
                   self._tensor(path, "path", i32, (B, M)), stream=stream)

    def fork(self, src, dst, stream=None):
        """Sequences dst (int32 [n], empty ones) become copies of src."""
        n, i32 = dst.numel(), self._torch.int32
        self._call(self._lib.sv_kv_fork, self._tensor(src, "src", i32, (n,)), self._tensor(dst, "dst", i32, (n,)), n,
                   stream=stream)

    def release(self, ids, stream=None):
        """Empties sequences ids (int32 [n])."""
        self._call(self._lib.sv_kv_release, self._tensor(ids, "ids", self._torch.int32), ids.numel(), stream=stream)

    def compact(self, stream=None):
        """Moves the held pages to the lowest ids.  The workspace belongs to
        the cache."""
        need = int(self._lib.sv_kv_compact_workspace_bytes(self._ref))
        if self._compact_ws is None:
            self._compact_ws = self._torch.empty(need // 4, dtype=self._torch.int32, device=self.device)
        self._call(self._lib.sv_kv_compact, self._compact_ws.data_ptr(), need, stream=stream)

    def bookkeeping(self):
        """The tensors that say what the cache holds: table, lengths, holders,
        free pages, counts.  Copying them back undoes calls since, but for
        rows written to slots that were not committed."""
        return self.table, self.lens, self.refs, self.free_ids, self.ctl

    def status(self) -> int:
        """SV_KV_* bits set on the device since the last call; synchronises."""
        v = ctypes.c_uint32()
        with self._torch.cuda.device(self.device):
            rc = self._lib.sv_kv_status(self._ref, ctypes.byref(v))
        if rc:
            raise _sv().SpecVerifyError(rc, self._lib.sv_last_error().decode())
        return v.value

    def attention(self, q_heads: int, B: int, M: int, scale=None, window: int = 0, sinks: int = 0, max_len: int = 0,
                  chunk: int = 0) -> "Attention":
        """The attention of calls of up to B sequences of M rows, with a
        workspace of its own: calls that may run at once, in two captured
        graphs or on two streams, take one each, and a plan is kept until
        what it enqueued on a stream other than its creation's has run."""
        return Attention(self, q_heads, B, M, scale, window, sinks, max_len, chunk)


class Attention:
    """sv_kv_attention for one shape of call: see KvCache.attention."""

    def __init__(self, kv: KvCache, q_heads, B, M, scale, window, sinks, max_len, chunk):
        sv = _sv()
        self.kv, self.q_heads, self.B, self.M = kv, q_heads, B, M
        self.c = sv.KvAttn(q_heads, 1.0 / math.sqrt(kv.dim) if scale is None else scale, window, sinks, max_len,
                           chunk, None)
        b = sv.KvBatch(B, M, kv.lens.data_ptr() if B > kv.seqs else None)
        # a size of 0 is also the answer to an invalid shape: run() says which
        self._n = int(kv._lib.sv_kv_attention_workspace_bytes(kv._ref, ctypes.byref(b), ctypes.byref(self.c)))
        self._ws = None
        if self._n:
            buf = kv._torch.empty(self._n + 256, dtype=kv._torch.uint8, device=kv.device)
            self._ws = buf[(-buf.data_ptr()) % 256:]

    def run(self, layer: int, q, out=None, seq=None, n_new=None, tree=None, rope=None, ep=None, stream=None):
        """out [B, M, q_heads, dim] fp32 = attention of rows q (same shape)
        over the cache; ep: an epilogue (sv.epilogue(SV_EP_QUANT, ...)) that
        takes the next projection's input."""
        kv = self.kv
        f32 = kv._torch.float32
        shape = (self.B, self.M, self.q_heads, kv.dim)
        qp = kv._tensor(q, "q", f32)
        if q.numel() != self.B * self.M * self.q_heads * kv.dim or (out is not None and out.numel() != q.numel()):
            raise _bad(f"kv: q and out must hold {shape} values")
        b = kv._batch(self.B, self.M, seq, n_new, tree)
        self.c.rope = None if rope is None else ctypes.addressof(rope.c)
        if rope is not None and rope.device is not None and rope.device != kv.device:
            raise _bad(f"kv: the rope table must be on {kv.device}")
        kv._call(kv._lib.sv_kv_attention, layer, ctypes.byref(b), ctypes.byref(self.c), qp,
                 kv._tensor(out, "out", f32), None if ep is None else ctypes.byref(ep),
                 None if self._ws is None else self._ws.data_ptr(), self._n, stream=stream)
