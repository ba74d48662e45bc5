"""The steps of a round around the projections: the residual's addition with
the RMS norm (sv_add_norm_q8), and sampling with filters (sv_sample).

Argument marshalling only, as in the package's other calls.  Tensors are
checked for their type, shape, device and contiguity, and SpecVerifyError is
raised before anything is enqueued; a call runs on its tensors' device, on
that device's current stream unless one is given.
"""

from __future__ import annotations

_torch = _library = _raw_stream = None


def _sv():
    import speculative_decoding_verification_amd as sv
    return sv


def _lib():
    """The library; torch, which importing the package leaves out, with it,
    and its call for the handle of a device's current stream, where it has one
    that makes no Stream object."""
    global _torch, _library, _raw_stream
    if _library is None:
        import torch
        _torch, _library = torch, _sv().lib()
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return _library


def _bad(msg):
    return _sv().SpecVerifyError(-1, msg)


def _device(t, name):
    if not t.is_cuda:
        raise _bad(f"{name} must be on a GPU")
    return t.get_device()


def _tensor(t, name, dtype, index, shape):
    """The data pointer of a tensor of the call, checked; None for None."""
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != index or not t.is_contiguous() or t.shape != shape:
        raise _bad(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


def _call(fn, index, stream, *args):
    cuda = _torch.cuda
    if stream is None:
        stream = _raw_stream(index) if _raw_stream else cuda.current_stream(index).cuda_stream
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if cuda.current_device() == index:
        rc = fn(*args, stream)
    else:
        with cuda.device(index):
            rc = fn(*args, stream)
    if rc:
        raise _sv().SpecVerifyError(rc, _library.sv_last_error().decode())


def add_norm_q8(x, delta=None, gamma=None, eps=1e-6, fold=False, sum=None, y=None, q=None, d=None, s16=None,
                sumsq=None, stream=None):
    """t = x + delta (fp32 [rows, K]) to `sum` (which may be x or delta), its
    RMS norm with weight gamma [K] to y, and the int8 codes of t * gamma to q
    [rows, K], d and sumsq [rows, K / 32] and s16 [rows, K / 16].  fold: the
    norm's factor is left to the codes' consumer (act(..., sumsq_parts))."""
    fn = _lib().sv_add_norm_q8
    if x.ndim != 2:
        raise _bad("add_norm_q8: x must be [rows, K]")
    index = _device(x, "add_norm_q8: x")
    one = x.shape
    rows, K = one
    f32 = _torch.float32
    b32 = (rows, K // 32)
    _call(fn, index, stream, _tensor(x, "add_norm_q8: x", f32, index, one),
          _tensor(delta, "add_norm_q8: delta", f32, index, one), rows, K,
          _tensor(gamma, "add_norm_q8: gamma", f32, index, (K,)), eps, int(fold),
          _tensor(sum, "add_norm_q8: sum", f32, index, one), _tensor(y, "add_norm_q8: y", f32, index, one),
          _tensor(q, "add_norm_q8: q", _torch.int8, index, one), _tensor(d, "add_norm_q8: d", f32, index, b32),
          _tensor(s16, "add_norm_q8: s16", _torch.int32, index, (rows, K // 16)),
          _tensor(sumsq, "add_norm_q8: sumsq", f32, index, b32))


def sampling_params(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, device="cuda"):
    """Settings for sample(): numbers for all rows alike, or sequences with
    one for each row (numbers among them count for every row).  Returns the
    device array of sv_sampling, int32 [n, 4]."""
    import numpy as np
    import torch
    fields = [np.atleast_1d(np.asarray(v)) for v in (temperature, top_k, top_p, min_p)]
    if any(f.ndim != 1 or f.size == 0 for f in fields) or len({f.size for f in fields if f.size != 1}) > 1:
        raise _bad("sampling_params: settings must be numbers or sequences of one length")
    if fields[1].dtype.kind not in "iu" or fields[1].min() < -(1 << 31) or fields[1].max() >= 1 << 31:
        raise _bad("sampling_params: top_k must be integers of 32 bits")
    n = max(f.size for f in fields)
    out = np.zeros((n, 4), np.int32)
    for i, f in enumerate(fields):
        out[:, i] = f.astype(np.int32) if i == 1 else f.astype(np.float32).view(np.int32)
    return torch.from_numpy(out).to(device)


def sample_workspace(rows: int, V: int, device="cuda"):
    """A workspace for sample() calls of up to `rows` rows of up to V tokens;
    calls that may run at once, in two captured graphs or on two streams,
    take one each."""
    import torch
    need = int(_sv().lib().sv_sample_workspace_bytes(rows, V))
    if need == 0:
        raise _sv().SpecVerifyError(_sv().SV_ERR_SHAPE, _sv().lib().sv_last_error().decode())
    buf = torch.empty(need + 256, dtype=torch.uint8, device=device)
    return buf[(-buf.data_ptr()) % 256:][:need]


def sample(logits, params, u, tokens, workspace, probs=None, kept=None, stream=None):
    """tokens int32 [rows] sampled from logits fp32 [rows, V] (rows may lie
    apart) with the settings of sampling_params() and uniforms u fp64 [rows];
    probs, kept fp32 [rows, V]: the distribution sampled from, and the logits
    with -inf for what the filters drop.  tokens may be None (then u too)."""
    fn, torch = _lib().sv_sample, _torch
    index = _device(logits, "sample: logits")
    if logits.ndim != 2 or logits.dtype != torch.float32 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise _bad("sample: logits must be float32 [rows, V] with contiguous rows")
    rows, V = logits.shape
    i32 = torch.int32
    if params.ndim != 2 or workspace is None:
        raise _bad("sample: params must be int32 [1 or rows, 4], and a workspace is needed")
    _call(fn, index, stream, logits.data_ptr(), rows, V, logits.stride(0) if rows > 1 else V,
          _tensor(params, "sample: params", i32, index, (params.shape[0], 4)), params.shape[0],
          _tensor(u, "sample: u", torch.float64, index, (rows,)), _tensor(tokens, "sample: tokens", i32, index, (rows,)),
          _tensor(probs, "sample: probs", torch.float32, index, (rows, V)),
          _tensor(kept, "sample: kept", torch.float32, index, (rows, V)),
          _tensor(workspace, "sample: workspace", torch.uint8, index, workspace.shape), workspace.numel())
