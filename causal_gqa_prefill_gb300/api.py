"""Python entry points over the C ABI (torch supplies device memory and streams).

``attn_prefill_fwd`` mirrors the C function argument for argument; the
convenience wrapper ``attn_prefill`` allocates the outputs and derives the
sizes from the tensors. Both only marshal arguments: the attention forward
runs entirely in the CUDA library, and a status other than ATTN_OK raises.
"""

from __future__ import annotations

import math

from . import _abi


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {_abi.status_string(status)}")


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream_handle(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def attn_prefill_fwd(q, k, v, o, lse, B, L, n_q, n_kv, d_h, causal, scale, stream=None) -> int:
    """Direct call of the C entry point; returns the raw status code.

    q, k, v, o, lse are CUDA tensors or integer device addresses with the
    layouts of the C header; ``stream`` is a torch.cuda.Stream, a raw
    cudaStream_t as int, or None for torch's current stream.
    """
    lib = _abi.load()
    return int(lib.attn_prefill_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(L),
                                    int(n_q), int(n_kv), int(d_h), int(causal), float(scale),
                                    _stream_handle(stream)))


def attn_prefill_fwd_chunk(q, k, v, o, lse, B, Lq, Lk, n_q, n_kv, d_h, causal, scale,
                           stream=None) -> int:
    """Direct call of the chunked-prefill C entry point (query = last Lq of Lk
    positions); returns the raw status code."""
    lib = _abi.load()
    return int(lib.attn_prefill_fwd_chunk(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B),
                                          int(Lq), int(Lk), int(n_q), int(n_kv), int(d_h),
                                          int(causal), float(scale), _stream_handle(stream)))


def attn_prefill_fwd_fp8(q, k, v, o, lse, B, Lq, Lk, n_q, n_kv, d_h, causal, scale, q_descale,
                         k_descale, v_descale, stream=None) -> int:
    """Direct call of the e4m3 C entry point; returns the raw status code."""
    lib = _abi.load()
    return int(lib.attn_prefill_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B),
                                        int(Lq), int(Lk), int(n_q), int(n_kv), int(d_h),
                                        int(causal), float(scale), float(q_descale),
                                        float(k_descale), float(v_descale),
                                        _stream_handle(stream)))


def attn_prefill_fp8(q, k, v, *, q_descale=1.0, k_descale=1.0, v_descale=1.0, causal=True,
                     scale=None, out=None, lse=None, stream=None):
    """Attention over e4m3 CUDA tensors (torch.float8_e4m3fn) q [B,Lq,n_q,128],
    k/v [B,Lk,n_kv,128], real values = stored * descale. Returns (o bf16
    [B, Lq, n_q, 128], lse fp32 [B, n_q, Lq])."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.float8_e4m3fn:
            raise TypeError(f"{name} must be float8_e4m3fn")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, L, H, d_h] tensor")
    B, L, n_q, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] < L or k.shape[3] != d:
        raise ValueError("k and v must be [B, Lk, n_kv, d_h] with Lk >= Lq, matching q")
    Lk, n_kv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((B, L, n_q, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, n_q, L), dtype=torch.float32, device=q.device)
    st = attn_prefill_fwd_fp8(q, k, v, out, lse, B, L, Lk, n_q, n_kv, d, int(bool(causal)),
                              scale, q_descale, k_descale, v_descale, stream)
    if st != _abi.ATTN_OK:
        raise AttnError(st, "attn_prefill_fwd_fp8")
    return out, lse


def attn_decode_workspace_bytes(B, Lk, n_q, n_kv, d_h=128) -> int:
    return int(_abi.load().attn_decode_workspace_bytes(int(B), int(Lk), int(n_q), int(n_kv),
                                                       int(d_h)))


def attn_decode_fwd(q, k, v, o, lse, workspace, workspace_bytes, B, Lk, n_q, n_kv, d_h, scale,
                    stream=None) -> int:
    """Direct call of the decode C entry point; returns the raw status code."""
    lib = _abi.load()
    return int(lib.attn_decode_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(workspace),
                                   int(workspace_bytes), int(B), int(Lk), int(n_q), int(n_kv),
                                   int(d_h), float(scale), _stream_handle(stream)))


def attn_decode(q, k, v, *, scale=None, workspace=None, out=None, lse=None, stream=None):
    """One decode step: q bf16 [B, 1, n_q, 128] against the cache k/v bf16
    [B, Lk, n_kv, 128]. Returns (o bf16 [B, 1, n_q, 128], lse fp32 [B, n_q, 1]).
    ``workspace`` (a CUDA tensor of at least attn_decode_workspace_bytes
    bytes) is allocated with torch when not given."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, L, H, d_h] tensor")
    B, one, n_q, d = q.shape
    if one != 1 or k.shape != v.shape or k.shape[0] != B or k.shape[3] != d:
        raise ValueError("q must be [B, 1, n_q, d_h] and k, v [B, Lk, n_kv, d_h]")
    Lk, n_kv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = attn_decode_workspace_bytes(B, Lk, n_q, n_kv, d)
    if need < 0:
        raise AttnError(_abi.ATTN_ERR_UNSUPPORTED, "attn_decode_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, n_q, 1), dtype=torch.float32, device=q.device)
    nbytes = workspace.numel() * workspace.element_size()
    st = attn_decode_fwd(q, k, v, out, lse, workspace, nbytes, B, Lk, n_q, n_kv, d, scale, stream)
    if st != _abi.ATTN_OK:
        raise AttnError(st, "attn_decode_fwd")
    return out, lse


class _Call:
    """Where a call over tensors of ``device`` runs: makes the device current,
    ``handle`` is the raw stream."""

    __slots__ = ("torch", "device", "guard", "handle", "other")

    def __init__(self, torch, device, stream):
        self.torch = torch
        self.device = device
        self.guard = None
        self.other = None                 # the torch stream, when it is not the current one
        # (a tensor is on the device, so CUDA is up: no need to ask whether it is)
        if torch._C._cuda_getDevice() != device.index:
            self.guard = torch.cuda.device(device)
        # the handle that torch.cuda.current_stream(device).cuda_stream gives,
        # without the two objects made on the way
        self.handle = torch._C._cuda_getCurrentRawStream(device.index)
        if stream is not None:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
            if handle != self.handle:
                self.handle = handle
                self.other = (torch.cuda.ExternalStream(handle, device=device) if handle
                              else torch.cuda.default_stream(device))

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def empty(self, shape, dtype):
        """Memory for the call. On another stream than the current one it is that
        stream's (the current one may still be at work on memory of its own that
        was freed), and is not handed out again before the current stream is done
        with it either."""
        if self.other is None:
            return self.torch.empty(shape, dtype=dtype, device=self.device)
        current = self.torch.cuda.current_stream(self.device)
        with self.torch.cuda.stream(self.other):
            t = self.torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(current)
        return t

    def workspace(self, given, size, *sizes):
        """(workspace, its bytes): the one given, or one of size(*sizes) bytes."""
        if given is None:
            nbytes = size(*sizes)
            if nbytes < 0:
                raise AttnError(_abi.ATTN_ERR_UNSUPPORTED, size.__name__)
            return self.empty(nbytes, self.torch.uint8), nbytes
        if getattr(given, "device", None) != self.device:
            raise ValueError(f"workspace must be a tensor on {self.device}")
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        return given, given.nbytes


def _laid_out(index, dtype, *tensors):
    """Are all of these (None: not given) contiguous, of this dtype and on CUDA device
    ``index``? With the shapes, what a call takes: where the answer is no, the
    checks below say what is wrong. (Run for every call they are 1 of a small
    call's 25 microseconds.)"""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != index
                              or not t.is_contiguous()):
            return False
    return index >= 0


def _wrong_tensor(name, t, shape, dtype, device=None):
    """The error that says how ``t`` differs from a contiguous CUDA tensor of this
    shape (None: any size) and dtype on ``device``; None if it does not."""
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        return TypeError(f"{name} must be a {str(dtype).replace('torch.', '')} CUDA tensor")
    if device is not None and t.device != device:
        return ValueError(f"{name} is on {t.device}, the other tensors are on {device}")
    if t.dim() != len(shape) or any(a is not None and a != b for a, b in zip(shape, t.shape)):
        want = ", ".join("*" if a is None else str(a) for a in shape)
        return ValueError(f"{name} must be [{want}], not {list(t.shape)}")
    if not t.is_contiguous():
        return ValueError(f"{name} must be contiguous")
    return None


def _cuda_tensor(name, t, shape, dtype, device=None):
    """``t`` if it is a contiguous CUDA tensor of this shape (None: any size) and
    dtype, on ``device``."""
    wrong = _wrong_tensor(name, t, shape, dtype, device)
    if wrong is not None:
        raise wrong
    return t


def _heads_of(name, t, first, length, dtype, device=None):
    """The shape of the contiguous [first, length, heads, d] CUDA tensor ``t`` (None:
    any size)."""
    return _cuda_tensor(name, t, (first, length, None, None), dtype, device).shape


def attn_key_weights_workspace_bytes(B, Lq, Lk, n_q, n_kv, d_h=128) -> int:
    return int(_abi.load().attn_key_weights_workspace_bytes(int(B), int(Lq), int(Lk), int(n_q),
                                                            int(n_kv), int(d_h)))


def attn_key_weights_fwd(q, k, lse, weights, workspace, workspace_bytes, B, Lq, Lk, n_q, n_kv, d_h,
                         causal, accumulate, scale, stream=None) -> int:
    """Direct call of the key weights C entry point; returns the raw status code."""
    lib = _abi.load()
    return int(lib.attn_key_weights_fwd(_ptr(q), _ptr(k), _ptr(lse), _ptr(weights),
                                        _ptr(workspace), int(workspace_bytes), int(B), int(Lq),
                                        int(Lk), int(n_q), int(n_kv), int(d_h), int(causal),
                                        int(accumulate), float(scale), _stream_handle(stream)))


def attn_key_weights(q, k, lse, *, causal=True, scale=None, weights=None, accumulate=False,
                     workspace=None, stream=None):
    """How much attention every key received: fp32 [B, n_kv, Lk], the softmax
    weights of a prefill summed over the rows that see the key and over its
    group's query heads.

    q bf16 [B, Lq, n_q, d], k bf16 [B, Lk, n_kv, d] (d 64 or 128, rows the last
    Lq of the Lk positions), lse fp32 [B, n_q, Lq] as attn_prefill returned it
    for the same causal and scale; a row whose lse is -inf (a padded one, say)
    adds nothing, whatever its q holds. ``weights`` receives the result, or with
    ``accumulate`` is added to (chunk after chunk of one prompt: pass the part
    of the tensor's positions that exist as its own contiguous tensor)."""
    import torch

    bf16, f32 = torch.bfloat16, torch.float32
    try:
        B, Lq, n_q, d = q.shape
        _, Lk, n_kv, _ = k.shape
        index = q.get_device()
        usual = (k.shape == (B, Lk, n_kv, d) and Lk >= Lq and lse.shape == (B, n_q, Lq)
                 and (not accumulate if weights is None else weights.shape == (B, n_kv, Lk))
                 and _laid_out(index, bf16, q, k) and _laid_out(index, f32, lse, weights))
    except (AttributeError, ValueError):
        usual = False
    if not usual:
        B, Lq, n_q, d = _heads_of("q", q, None, None, bf16)
        _, Lk, n_kv, dk = _heads_of("k", k, B, None, bf16, q.device)
        if dk != d:
            raise ValueError("q and k must have the same d_h")
        if Lk < Lq:
            raise ValueError("k must hold at least as many positions as q has rows")
        _cuda_tensor("lse", lse, (B, n_q, Lq), f32, q.device)
        if weights is not None:
            _cuda_tensor("weights", weights, (B, n_kv, Lk), f32, q.device)
        elif accumulate:
            raise ValueError("accumulate needs the weights to add to")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _Call(torch, q.device, stream) as call:
        workspace, nbytes = call.workspace(workspace, attn_key_weights_workspace_bytes, B, Lq, Lk,
                                           n_q, n_kv, d)
        if weights is None:
            weights = call.empty((B, n_kv, Lk), f32)
        st = _abi.load().attn_key_weights_fwd(
            q.data_ptr(), k.data_ptr(), lse.data_ptr(), weights.data_ptr(), workspace.data_ptr(),
            nbytes, B, Lq, Lk, n_q, n_kv, d, bool(causal), bool(accumulate), scale, call.handle)
    if st != _abi.ATTN_OK:
        raise AttnError(st, "attn_key_weights_fwd")
    return weights


def attn_decode_ragged_workspace_bytes(B, C, n_q, n_kv, d_h=128, weighted=False) -> int:
    return int(_abi.load().attn_decode_ragged_workspace_bytes(
        int(B), int(C), int(n_q), int(n_kv), int(d_h), int(bool(weighted))))


def attn_decode_ragged_fwd(q, k, v, lens, weights, o, lse, workspace, workspace_bytes, B, C, n_q,
                           n_kv, d_h, scale, stream=None) -> int:
    """Direct call of the ragged decode C entry point; returns the raw status code."""
    lib = _abi.load()
    return int(lib.attn_decode_ragged_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(lens), _ptr(weights),
                                          _ptr(o), _ptr(lse), _ptr(workspace),
                                          int(workspace_bytes), int(B), int(C), int(n_q),
                                          int(n_kv), int(d_h), float(scale),
                                          _stream_handle(stream)))


def attn_decode_ragged(q, k, v, lens, *, weights=None, scale=None, workspace=None, out=None,
                       lse=None, stream=None):
    """One decode step against caches of different lengths: q bf16 [B, 1, n_q, 128],
    k/v bf16 [B, C, n_kv, 128] of which sequence b holds the first lens[b]
    positions (lens: int32 CUDA tensor [B], clamped to 0 .. C).

    Returns (o bf16 [B, 1, n_q, 128], lse fp32 [B, n_q, 1]); a sequence of
    length 0 gets o = 0 and lse = -inf. ``weights`` (fp32 [B, n_kv, C]), when
    given, is updated in place: every cached position's softmax weight, summed
    over its group's query heads, is added to it. ``workspace`` (at least
    attn_decode_ragged_workspace_bytes bytes) is allocated with torch when not
    given."""
    import torch

    bf16, f32 = torch.bfloat16, torch.float32
    try:
        B, one, n_q, d = q.shape
        _, C, n_kv, _ = k.shape
        index = q.get_device()
        usual = (one == 1 and v.shape == k.shape == (B, C, n_kv, d) and lens.shape == (B,)
                 and (weights is None or weights.shape == (B, n_kv, C))
                 and (out is None or out.shape == q.shape)
                 and (lse is None or lse.shape == (B, n_q, 1))
                 and _laid_out(index, bf16, q, k, v, out) and _laid_out(index, f32, weights, lse)
                 and _laid_out(index, torch.int32, lens))
    except (AttributeError, ValueError):
        usual = False
    if not usual:
        B, _, n_q, d = _heads_of("q", q, None, 1, bf16)
        dev = q.device
        _, C, n_kv, dk = _heads_of("k", k, B, None, bf16, dev)
        if dk != d:
            raise ValueError("q and k must have the same d_h")
        _cuda_tensor("v", v, k.shape, bf16, dev)
        _cuda_tensor("lens", lens, (B,), torch.int32, dev)
        if weights is not None:
            _cuda_tensor("weights", weights, (B, n_kv, C), f32, dev)
        if out is not None:
            _cuda_tensor("out", out, q.shape, bf16, dev)
        if lse is not None:
            _cuda_tensor("lse", lse, (B, n_q, 1), f32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _Call(torch, q.device, stream) as call:
        workspace, nbytes = call.workspace(workspace, attn_decode_ragged_workspace_bytes, B, C, n_q,
                                           n_kv, d, weights is not None)
        if out is None:
            out = call.empty(q.shape, bf16)
        if lse is None:
            lse = call.empty((B, n_q, 1), f32)
        st = _abi.load().attn_decode_ragged_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), lens.data_ptr(), _ptr(weights),
            out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), nbytes, B, C, n_q, n_kv, d, scale,
            call.handle)
    if st != _abi.ATTN_OK:
        raise AttnError(st, "attn_decode_ragged_fwd")
    return out, lse


def attn_decode_shared_workspace_bytes(B, P, C, n_q, n_kv, d_h=128) -> int:
    return int(_abi.load().attn_decode_shared_workspace_bytes(int(B), int(P), int(C), int(n_q),
                                                              int(n_kv), int(d_h)))


def attn_decode_shared_fwd(q, prefix_k, prefix_v, k, v, lens, o, lse, workspace, workspace_bytes, B,
                           P, C, n_q, n_kv, d_h, scale, stream=None) -> int:
    """Direct call of the shared-prefix decode C entry point; returns the raw status code."""
    lib = _abi.load()
    return int(lib.attn_decode_shared_fwd(_ptr(q), _ptr(prefix_k), _ptr(prefix_v), _ptr(k), _ptr(v),
                                          _ptr(lens), _ptr(o), _ptr(lse), _ptr(workspace),
                                          int(workspace_bytes), int(B), int(P), int(C), int(n_q),
                                          int(n_kv), int(d_h), float(scale),
                                          _stream_handle(stream)))


def attn_decode_shared(q, prefix_k, prefix_v, k, v, lens, *, scale=None, workspace=None, out=None,
                       lse=None, stream=None):
    """One decode step of a batch behind a shared prefix: q bf16 [B, 1, n_q, 128]
    attends to prefix_k/prefix_v bf16 [1, P, n_kv, 128], which all sequences share,
    and to the first lens[b] positions of its own k/v bf16 [B, C, n_kv, 128]
    (lens: int32 CUDA tensor [B], 0 allowed), in one softmax.

    Returns (o bf16 [B, 1, n_q, 128], lse fp32 [B, n_q, 1]). ``workspace`` (at
    least attn_decode_shared_workspace_bytes bytes) is allocated with torch when
    not given."""
    import torch

    bf16, f32 = torch.bfloat16, torch.float32
    try:
        B, one, n_q, d = q.shape
        _, C, n_kv, _ = k.shape
        P = prefix_k.shape[1]
        index = q.get_device()
        usual = (one == 1 and prefix_v.shape == prefix_k.shape == (1, P, n_kv, d)
                 and v.shape == k.shape == (B, C, n_kv, d) and lens.shape == (B,)
                 and (out is None or out.shape == q.shape)
                 and (lse is None or lse.shape == (B, n_q, 1))
                 and _laid_out(index, bf16, q, prefix_k, prefix_v, k, v, out)
                 and _laid_out(index, f32, lse) and _laid_out(index, torch.int32, lens))
    except (AttributeError, ValueError, IndexError):
        usual = False
    if not usual:
        B, _, n_q, d = _heads_of("q", q, None, 1, bf16)
        dev = q.device
        _, P, n_kv, dp = _heads_of("prefix_k", prefix_k, 1, None, bf16, dev)
        _cuda_tensor("prefix_v", prefix_v, prefix_k.shape, bf16, dev)
        _, C, own_kv, dk = _heads_of("k", k, B, None, bf16, dev)
        if dk != d or dp != d or own_kv != n_kv:
            raise ValueError("q, prefix_k and k must agree on d_h, the caches on their heads")
        _cuda_tensor("v", v, k.shape, bf16, dev)
        _cuda_tensor("lens", lens, (B,), torch.int32, dev)
        if out is not None:
            _cuda_tensor("out", out, q.shape, bf16, dev)
        if lse is not None:
            _cuda_tensor("lse", lse, (B, n_q, 1), f32, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _Call(torch, q.device, stream) as call:
        workspace, nbytes = call.workspace(workspace, attn_decode_shared_workspace_bytes, B, P, C,
                                           n_q, n_kv, d)
        if out is None:
            out = call.empty(q.shape, bf16)
        if lse is None:
            lse = call.empty((B, n_q, 1), f32)
        st = _abi.load().attn_decode_shared_fwd(
            q.data_ptr(), prefix_k.data_ptr(), prefix_v.data_ptr(), k.data_ptr(), v.data_ptr(),
            lens.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), nbytes, B, P, C,
            n_q, n_kv, d, scale, call.handle)
    if st != _abi.ATTN_OK:
        raise AttnError(st, "attn_decode_shared_fwd")
    return out, lse


def attn_cache_evict(k, v, weights, lens, k_out, v_out, weights_out, lens_out, index, B, C, C_out,
                     budget, recent, n_kv, d_h, elem_bytes, stream=None) -> int:
    """Direct call of the eviction C entry point; returns the raw status code."""
    lib = _abi.load()
    return int(lib.attn_cache_evict(_ptr(k), _ptr(v), _ptr(weights), _ptr(lens), _ptr(k_out),
                                    _ptr(v_out), _ptr(weights_out), _ptr(lens_out), _ptr(index),
                                    int(B), int(C), int(C_out), int(budget), int(recent),
                                    int(n_kv), int(d_h), int(elem_bytes),
                                    _stream_handle(stream)))


def attn_evict(k, v, weights, lens, budget, recent=0, *, capacity=None, k_out=None, v_out=None,
               weights_out=None, lens_out=None, index=None, stream=None):
    """Brings caches down to ``budget`` positions per sequence and K/V head: the
    last ``recent`` ones and, of those before them, the ones of largest
    accumulated weight (ties to the lowest position); shorter caches are kept
    whole.

    k, v: bf16 or float8_e4m3fn [B, C, n_kv, d_h], d_h 64 or 128; weights fp32
    [B, n_kv, C] (as attn_key_weights and attn_decode_ragged accumulate it);
    lens int32 [B]. Returns (k_out, v_out [B, capacity, n_kv, d_h], weights_out
    [B, n_kv, capacity], lens_out [B], index int32 [B, n_kv, budget]): kept
    positions in order, weights_out zero and index -1 past lens_out. Rows of
    k_out and v_out past lens_out are left as they were (unspecified when
    allocated here). ``capacity`` (that of k_out when given, else ``budget``) is
    the room of the new caches. Outputs must not overlap the inputs."""
    import torch

    kind = getattr(k, "dtype", None)
    if kind is not torch.bfloat16 and kind is not torch.float8_e4m3fn:
        raise TypeError("k must be a bfloat16 or float8_e4m3fn CUDA tensor")
    f32, i32 = torch.float32, torch.int32
    budget, recent = int(budget), int(recent)
    if budget < 1 or not 0 <= recent <= budget:
        raise ValueError("budget must be at least 1 and recent between 0 and budget")
    if capacity is None:
        capacity = budget if getattr(k_out, "ndim", 0) != 4 else k_out.shape[1]
    if capacity < budget:
        raise ValueError("the new capacity must hold the budget")
    try:
        B, C, n_kv, d = k.shape
        dev, device = k.get_device(), k.device
        usual = (v.shape == k.shape and weights.shape == (B, n_kv, C) and lens.shape == (B,)
                 and (k_out is None or k_out.shape == (B, capacity, n_kv, d))
                 and (v_out is None or v_out.shape == (B, capacity, n_kv, d))
                 and (weights_out is None or weights_out.shape == (B, n_kv, capacity))
                 and (lens_out is None or lens_out.shape == (B,))
                 and (index is None or index.shape == (B, n_kv, budget))
                 and _laid_out(dev, kind, k, v, k_out, v_out)
                 and _laid_out(dev, f32, weights, weights_out)
                 and _laid_out(dev, i32, lens, lens_out, index))
    except (AttributeError, ValueError):
        usual = False
    if not usual:
        B, C, n_kv, d = _heads_of("k", k, None, None, kind)
        device = k.device
        _cuda_tensor("v", v, k.shape, kind, device)
        _cuda_tensor("weights", weights, (B, n_kv, C), f32, device)
        _cuda_tensor("lens", lens, (B,), i32, device)
        for name, t, shape, dtype in (("k_out", k_out, (B, capacity, n_kv, d), kind),
                                      ("v_out", v_out, (B, capacity, n_kv, d), kind),
                                      ("weights_out", weights_out, (B, n_kv, capacity), f32),
                                      ("lens_out", lens_out, (B,), i32),
                                      ("index", index, (B, n_kv, budget), i32)):
            if t is not None:
                _cuda_tensor(name, t, shape, dtype, device)
    with _Call(torch, device, stream) as call:
        if k_out is None:
            k_out = call.empty((B, capacity, n_kv, d), kind)
        if v_out is None:
            v_out = call.empty((B, capacity, n_kv, d), kind)
        if weights_out is None:
            weights_out = call.empty((B, n_kv, capacity), f32)
        if lens_out is None:
            lens_out = call.empty((B,), i32)
        if index is None:
            index = call.empty((B, n_kv, budget), i32)
        st = _abi.load().attn_cache_evict(
            k.data_ptr(), v.data_ptr(), weights.data_ptr(), lens.data_ptr(), k_out.data_ptr(),
            v_out.data_ptr(), weights_out.data_ptr(), lens_out.data_ptr(), index.data_ptr(),
            B, C, capacity, budget, recent, n_kv, d, k.element_size(), call.handle)
    if st != _abi.ATTN_OK:
        raise AttnError(st, "attn_cache_evict")
    return k_out, v_out, weights_out, lens_out, index


def attn_prefill_bwd_workspace_bytes(B, L, n_q, n_kv, d_h=128) -> int:
    return int(_abi.load().attn_prefill_bwd_workspace_bytes(int(B), int(L), int(n_q), int(n_kv),
                                                            int(d_h)))


def attn_prefill_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, B, L, n_q,
                     n_kv, d_h, causal, scale, stream=None) -> int:
    """Direct call of the backward C entry point; returns the raw status code."""
    lib = _abi.load()
    return int(lib.attn_prefill_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                    _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                                    int(workspace_bytes), int(B), int(L), int(n_q), int(n_kv),
                                    int(d_h), int(causal), float(scale), _stream_handle(stream)))


def attn_prefill_backward(q, k, v, o, lse, dout, *, causal=True, scale=None, workspace=None,
                          dq=None, dk=None, dv=None, stream=None):
    """Gradients (dq, dk, dv) of attn_prefill for the upstream gradient ``dout``.

    q, o, dout: bf16 CUDA tensors [B, L, n_q, d_h]; k, v: [B, L, n_kv, d_h], d_h 64 or 128;
    lse: the forward's fp32 [B, n_q, L]. Outputs are allocated unless passed
    in; ``workspace`` (at least attn_prefill_bwd_workspace_bytes bytes) is
    allocated with torch when not given."""
    import torch

    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, L, H, d_h] tensor")
    B, L, n_q, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] != L or k.shape[3] != d:
        raise ValueError("k and v must be [B, L, n_kv, d_h] matching q")
    if o.shape != q.shape or dout.shape != q.shape:
        raise ValueError("o and dout must be shaped like q")
    n_kv = k.shape[2]
    if (not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32 or not lse.is_cuda
            or tuple(lse.shape) != (B, n_q, L) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 CUDA tensor [B, n_q, L]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = attn_prefill_bwd_workspace_bytes(B, L, n_q, n_kv, d)
    if need < 0:
        raise AttnError(_abi.ATTN_ERR_UNSUPPORTED, "attn_prefill_bwd_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    nbytes = workspace.numel() * workspace.element_size()
    st = attn_prefill_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, nbytes, B, L, n_q, n_kv,
                          d, int(bool(causal)), scale, stream)
    if st != _abi.ATTN_OK:
        raise AttnError(st, "attn_prefill_bwd")
    return dq, dk, dv


def attn_device_check(stream=None) -> int:
    """Synchronise the stream and report device-side timeouts (raw status)."""
    return int(_abi.load().attn_device_check(_stream_handle(stream)))


def attn_prefill_host_staging_bytes(B, Lq, Lk, n_q, n_kv, d_h=128) -> int:
    return int(_abi.load().attn_prefill_host_staging_bytes(int(B), int(Lq), int(Lk), int(n_q),
                                                           int(n_kv), int(d_h)))


def attn_prefill_fwd_host(q, k, v, o, lse, staging, staging_bytes, B, Lq, Lk, n_q, n_kv, d_h,
                          causal, scale, stream=None) -> int:
    """Direct call of the host-buffer C entry point (q, k, v, o, lse host
    tensors or addresses; staging a device buffer); returns the raw status."""
    lib = _abi.load()
    return int(lib.attn_prefill_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                         _ptr(staging), int(staging_bytes), int(B), int(Lq),
                                         int(Lk), int(n_q), int(n_kv), int(d_h), int(causal),
                                         float(scale), _stream_handle(stream)))


def attn_selftest_wait_timeout(spin_cycles: int, stream=None) -> int:
    """Enqueue the wait-limit diagnostic kernel (raw status of the launch)."""
    return int(_abi.load().attn_selftest_wait_timeout(int(spin_cycles), _stream_handle(stream)))


def attn_selftest_wait_timeout_noalloc(spin_cycles: int, stream=None) -> int:
    """The wait-limit diagnostic reporting into the allocation-free entry
    point's fixed status word (raw status of the launch)."""
    return int(_abi.load().attn_selftest_wait_timeout_noalloc(int(spin_cycles),
                                                             _stream_handle(stream)))


def attn_prefill_grid_size(B, L, n_q, n_kv, d_h, causal=True) -> int:
    return int(_abi.load().attn_prefill_grid_size(int(B), int(L), int(n_q), int(n_kv), int(d_h),
                                                  int(bool(causal))))


def attn_prefill(q, k, v, *, causal: bool = True, scale: float | None = None, out=None, lse=None,
                 stream=None):
    """O, LSE = attention(q, k, v) for bf16 CUDA tensors q [B,Lq,n_q,d], k/v [B,Lk,n_kv,d].

    Lk = Lq is ordinary prefill; Lk > Lq is a chunk whose rows are the last Lq
    positions of the key range (chunked prefill). Returns (o bf16
    [B, Lq, n_q, d], lse fp32 [B, n_q, Lq]). ``scale`` defaults to 1/sqrt(d).
    Outputs may be passed in (``out``, ``lse``) to avoid allocation. The call
    is asynchronous on ``stream`` (default: current).
    """
    import torch

    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, L, H, d_h] tensor")
    B, L, n_q, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[1] < L or k.shape[3] != d:
        raise ValueError("k and v must be [B, Lk, n_kv, d_h] with Lk >= Lq, matching q")
    Lk, n_kv = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise ValueError("out must be a contiguous bf16 tensor shaped like q")
    if lse is None:
        lse = torch.empty((B, n_q, L), dtype=torch.float32, device=q.device)
    elif tuple(lse.shape) != (B, n_q, L) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, n_q, L] tensor")
    if Lk == L:
        st = attn_prefill_fwd(q, k, v, out, lse, B, L, n_q, n_kv, d, int(bool(causal)), scale,
                              stream)
    else:
        st = attn_prefill_fwd_chunk(q, k, v, out, lse, B, L, Lk, n_q, n_kv, d,
                                    int(bool(causal)), scale, stream)
    if st != _abi.ATTN_OK:
        raise AttnError(st, "attn_prefill_fwd" if Lk == L else "attn_prefill_fwd_chunk")
    return out, lse
