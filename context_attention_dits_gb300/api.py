"""Python binding of the C ABI with the same names (argument marshalling only).

Every call takes CUDA torch tensors, checks shapes and dtypes, and passes raw
device pointers, sizes and the current torch stream to libcpattn.so. All
computation happens in the library's kernels; PyTorch only supplies device
memory and the stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import CP_BF16, CP_F32, CP_LAP_FUSED, CP_LAP_STEPWISE, CpError, check, lib

_DT = {torch.bfloat16: CP_BF16, torch.float32: CP_F32}
_MODES = {"fused": CP_LAP_FUSED, "stepwise": CP_LAP_STEPWISE}


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}: q/k/v must be bfloat16 or float32")
    return _DT[t.dtype]


def _cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")


def _mode(mode) -> int:
    return _MODES[mode] if isinstance(mode, str) else int(mode)


def cp_block_attn_fwd(q, k, v, out, lse, scale: float, stream=None):
    """Block attention of q [B,Sq,H,D] against k, v [B,Skv,H,D] -> out [B,Sq,H,D] f32, lse [B,H,Sq] f32.

    q, k, v may be views with a batch stride (the inner [S, H, D] must be dense);
    out likewise; lse must be dense.
    """
    _cuda(q, k, v, out, lse)
    B, Sq, H, D = q.shape
    Skv = k.shape[1]
    if k.shape != (B, Skv, H, D) or v.shape != k.shape or out.shape != (B, Sq, H, D) or lse.shape != (B, H, Sq):
        raise ValueError("shape mismatch")
    if q.dtype != k.dtype or q.dtype != v.dtype or out.dtype != torch.float32 or lse.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; out and lse must be float32")
    for t in (q, k, v, out):
        if t.stride()[1:] != (H * D, D, 1):
            raise ValueError("the [S, H, D] part of each tensor must be dense")
    if not lse.is_contiguous():
        raise ValueError("lse must be dense")
    st = lib().cp_block_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                 B, H, Sq, Skv, D, float(scale), q.stride(0), k.stride(0), out.stride(0),
                                 _dt(q), _stream(stream))
    check(st, "cp_block_attn_fwd")


def cp_lse_merge(out_acc, lse_acc, out_blk, lse_blk, stream=None):
    """In place: (out_acc, lse_acc) <- merge((out_acc, lse_acc), (out_blk, lse_blk)); all float32 dense."""
    _cuda(out_acc, lse_acc, out_blk, lse_blk)
    B, S, H, D = out_acc.shape
    if out_blk.shape != out_acc.shape or lse_acc.shape != (B, H, S) or lse_blk.shape != (B, H, S):
        raise ValueError("shape mismatch")
    for t in (out_acc, lse_acc, out_blk, lse_blk):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError("merge operands must be dense float32")
    st = lib().cp_lse_merge(out_acc.data_ptr(), lse_acc.data_ptr(), out_blk.data_ptr(), lse_blk.data_ptr(),
                            B, H, S, D, _stream(stream))
    check(st, "cp_lse_merge")


def cp_ulysses_seq2head(x_in, x_out, stream=None):
    """[U, B, S/U, H, D] -> [U, B, S, H/U, D] (any dtype, dense)."""
    _cuda(x_in, x_out)
    U, B, Sl, H, D = x_in.shape
    if x_out.shape != (U, B, Sl * U, H // U, D) or x_out.dtype != x_in.dtype:
        raise ValueError("shape/dtype mismatch")
    if not (x_in.is_contiguous() and x_out.is_contiguous()):
        raise ValueError("tensors must be dense")
    st = lib().cp_ulysses_seq2head(x_in.data_ptr(), x_out.data_ptr(), U, B, Sl * U, H, D, x_in.element_size(),
                                   _stream(stream))
    check(st, "cp_ulysses_seq2head")


def cp_ulysses_head2seq(x_in, x_out, stream=None):
    """[U, B, S, H/U, D] -> [U, B, S/U, H, D] (any dtype, dense)."""
    _cuda(x_in, x_out)
    U, B, S, Hg, D = x_in.shape
    if x_out.shape != (U, B, S // U, Hg * U, D) or x_out.dtype != x_in.dtype:
        raise ValueError("shape/dtype mismatch")
    if not (x_in.is_contiguous() and x_out.is_contiguous()):
        raise ValueError("tensors must be dense")
    st = lib().cp_ulysses_head2seq(x_in.data_ptr(), x_out.data_ptr(), U, B, S, Hg * U, D, x_in.element_size(),
                                   _stream(stream))
    check(st, "cp_ulysses_head2seq")


def _anything(name, x_in, x_out, U, B, S, H, D, stream):
    _cuda(x_in, x_out)
    n = B * S * H * D
    if x_in.numel() != n or x_out.numel() != n or x_out.dtype != x_in.dtype:
        raise ValueError("both buffers must hold B*S*H*D elements of one dtype")
    if not (x_in.is_contiguous() and x_out.is_contiguous()):
        raise ValueError("buffers must be dense")
    st = getattr(lib(), name)(x_in.data_ptr(), x_out.data_ptr(), U, B, S, H, D, x_in.element_size(),
                              _stream(stream))
    check(st, name)


def cp_ulysses_anything_seq2head(x_in, x_out, U, B, S, H, D, stream=None):
    """Ragged regroup: rank blocks [B, S_u, H, D] back to back -> head-group blocks [B, S, H_g, D]
    back to back (balanced splits of S and H into U; any dtype; flat dense buffers)."""
    _anything("cp_ulysses_anything_seq2head", x_in, x_out, U, B, S, H, D, stream)


def cp_ulysses_anything_head2seq(x_in, x_out, U, B, S, H, D, stream=None):
    """Inverse of cp_ulysses_anything_seq2head."""
    _anything("cp_ulysses_anything_head2seq", x_in, x_out, U, B, S, H, D, stream)


def cp_attention_validate(B, H, S, D, ring_degree=1, ulysses_degree=1, uneven_ok=False, dtype=torch.bfloat16) -> int:
    """Status code cp_attention_fwd would return on validation (0 = ok). Host only."""
    return lib().cp_attention_validate(B, H, S, D, ring_degree, ulysses_degree, int(bool(uneven_ok)), _DT[dtype])


def cp_ring_shard_table(S: int, n: int, uneven_ok: bool = False):
    """[(offset, length)] of the n ring shards. Host only."""
    off = (ctypes.c_int * n)()
    ln = (ctypes.c_int * n)()
    check(lib().cp_ring_shard_table(S, n, int(bool(uneven_ok)), off, ln), "cp_ring_shard_table")
    return [(off[i], ln[i]) for i in range(n)]


def cp_attention_workspace_size(B, H, S, D, ring_degree=1, ulysses_degree=1, dtype=torch.bfloat16,
                                mode="fused") -> int:
    return int(lib().cp_attention_workspace_size(B, H, S, D, ring_degree, ulysses_degree, _DT[dtype], _mode(mode)))


def cp_attention_launch_count(B, H, S, D, ring_degree=1, ulysses_degree=1, dtype=torch.bfloat16,
                              mode="fused") -> int:
    return int(lib().cp_attention_launch_count(B, H, S, D, ring_degree, ulysses_degree, _DT[dtype], _mode(mode)))


def cp_attention_fwd(q, k, v, out, lse, scale: float, ring_degree: int = 1, ulysses_degree: int = 1,
                     uneven_ok: bool = False, workspace=None, mode="fused", stream=None, key_mask=None):
    """Context-parallel attention over global q, k, v [B,S,H,D] -> out [B,S,H,D] f32, lse [B,H,S] f32.

    workspace: a CUDA uint8 tensor of at least cp_attention_workspace_size(...)
    bytes; allocated here through torch when None. key_mask: optional CUDA
    bool/uint8 tensor [B, S] (True/nonzero = the key takes part); calls
    cp_attention_fwd_masked.
    """
    _cuda(q, k, v, out, lse)
    B, S, H, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or out.shape != q.shape or lse.shape != (B, H, S):
        raise ValueError("shape mismatch")
    if q.dtype != k.dtype or q.dtype != v.dtype or out.dtype != torch.float32 or lse.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; out and lse must be float32")
    for t in (q, k, v, out, lse):
        if not t.is_contiguous():
            raise ValueError("tensors must be dense")
    m = _mode(mode)
    need = cp_attention_workspace_size(B, H, S, D, ring_degree, ulysses_degree, q.dtype, m)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if key_mask is not None:
        _cuda(key_mask)
        if key_mask.shape != (B, S) or key_mask.dtype not in (torch.bool, torch.uint8) or not key_mask.is_contiguous():
            raise ValueError("key_mask must be a dense bool or uint8 tensor [B, S]")
        st = lib().cp_attention_fwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), key_mask.data_ptr(),
                                           out.data_ptr(), lse.data_ptr(), B, H, S, D, float(scale), ring_degree,
                                           ulysses_degree, int(bool(uneven_ok)), ws_ptr, ws_bytes, _dt(q), m,
                                           _stream(stream))
        check(st, "cp_attention_fwd_masked")
        return
    st = lib().cp_attention_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                B, H, S, D, float(scale), ring_degree, ulysses_degree, int(bool(uneven_ok)),
                                ws_ptr, ws_bytes, _dt(q), m, _stream(stream))
    check(st, "cp_attention_fwd")


def cp_attention_host_buffer_size(B, H, S, D, ring_degree=1, ulysses_degree=1, dtype=torch.bfloat16,
                                  mode="fused") -> int:
    return int(lib().cp_attention_host_buffer_size(B, H, S, D, ring_degree, ulysses_degree, _DT[dtype], _mode(mode)))


def cp_attention_fwd_host(q, k, v, out, lse, scale: float, ring_degree: int = 1, ulysses_degree: int = 1,
                          uneven_ok: bool = False, dev_buffer=None, mode="fused", head_chunks: int = 5,
                          stream=None):
    """cp_attention_fwd over host (CPU, ideally pinned) tensors q, k, v [B,S,H,D], out [B,S,H,D] f32 and
    lse [B,H,S] f32, with transfers overlapping compute over head chunks. dev_buffer: a CUDA uint8 tensor
    of at least cp_attention_host_buffer_size(...) bytes (allocated here through torch when None).
    Returns without waiting; the results are in out, lse once `stream` reaches this point."""
    for t in (q, k, v, out, lse):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v, out, lse must be dense host tensors")
    B, S, H, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or out.shape != (B, S, H, D) or lse.shape != (B, H, S):
        raise ValueError("shape mismatch")
    if k.dtype != q.dtype or v.dtype != q.dtype or out.dtype != torch.float32 or lse.dtype != torch.float32:
        raise ValueError("dtype mismatch")
    need = cp_attention_host_buffer_size(B, H, S, D, ring_degree, ulysses_degree, q.dtype, mode)
    if dev_buffer is None:
        dev_buffer = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    _cuda(dev_buffer)
    st = lib().cp_attention_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                     B, H, S, D, float(scale), ring_degree, ulysses_degree, int(bool(uneven_ok)),
                                     dev_buffer.data_ptr(), dev_buffer.numel(), _dt(q), _mode(mode), head_chunks,
                                     _stream(stream))
    check(st, "cp_attention_fwd_host")
    return dev_buffer


def cp_attention_fwd_no_alloc(q, k, v, out, lse, scale: float, ring_degree: int = 1, ulysses_degree: int = 1,
                              uneven_ok: bool = False, mode="fused", stream=None):
    """cp_attention_fwd with the library's built-in 64 MiB device workspace (no allocation).

    For callers that cannot allocate device memory. All calls share the
    built-in workspace: calls that overlap on the GPU race.
    """
    _cuda(q, k, v, out, lse)
    B, S, H, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or out.shape != q.shape or lse.shape != (B, H, S):
        raise ValueError("shape mismatch")
    if q.dtype != k.dtype or q.dtype != v.dtype or out.dtype != torch.float32 or lse.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; out and lse must be float32")
    for t in (q, k, v, out, lse):
        if not t.is_contiguous():
            raise ValueError("tensors must be dense")
    st = lib().cp_attention_fwd_no_alloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                         B, H, S, D, float(scale), ring_degree, ulysses_degree, int(bool(uneven_ok)),
                                         _dt(q), _mode(mode), _stream(stream))
    check(st, "cp_attention_fwd_no_alloc")


def cp_attention_bwd_workspace_size(B, H, S, D, ring_degree=1, ulysses_degree=1, dtype=torch.bfloat16) -> int:
    return int(lib().cp_attention_bwd_workspace_size(B, H, S, D, ring_degree, ulysses_degree, _DT[dtype]))


def cp_attention_bwd_launch_count(B, H, S, D, ring_degree=1, ulysses_degree=1, dtype=torch.bfloat16) -> int:
    return int(lib().cp_attention_bwd_launch_count(B, H, S, D, ring_degree, ulysses_degree, _DT[dtype]))


def cp_attention_bwd(q, k, v, out, dout, lse, dq, dk, dv, scale: float, ring_degree: int = 1,
                     ulysses_degree: int = 1, uneven_ok: bool = False, workspace=None, stream=None):
    """Backward of cp_attention_fwd: q, k, v, dout [B,S,H,D] (one dtype), out [B,S,H,D] f32 and
    lse [B,H,S] f32 from the forward -> dq, dk, dv [B,S,H,D] f32 (written).

    Ring, Ulysses, unified, and Ulysses Anything (uneven_ok with ulysses_degree > 1); Ring
    Anything is inference only and raises. workspace: a CUDA uint8 tensor of at least
    cp_attention_bwd_workspace_size(...) bytes; allocated here through torch when None.
    """
    _cuda(q, k, v, out, dout, lse, dq, dk, dv)
    B, S, H, D = q.shape
    for t in (k, v, dout, out, dq, dk, dv):
        if t.shape != q.shape:
            raise ValueError("shape mismatch")
    if lse.shape != (B, H, S):
        raise ValueError("lse must be [B, H, S]")
    if k.dtype != q.dtype or v.dtype != q.dtype or dout.dtype != q.dtype:
        raise TypeError("q, k, v and dout must share a dtype")
    for t in (out, lse, dq, dk, dv):
        if t.dtype != torch.float32:
            raise TypeError("out, lse, dq, dk and dv must be float32")
    for t in (q, k, v, out, dout, lse, dq, dk, dv):
        if not t.is_contiguous():
            raise ValueError("tensors must be dense")
    need = cp_attention_bwd_workspace_size(B, H, S, D, ring_degree, ulysses_degree, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _cuda(workspace)
    st = lib().cp_attention_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), dout.data_ptr(),
                                lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, D,
                                float(scale), ring_degree, ulysses_degree, int(bool(uneven_ok)),
                                workspace.data_ptr(), workspace.numel(), _dt(q), _stream(stream))
    check(st, "cp_attention_bwd")


# ---------------------------------------------------------------------------
# attention with a score rule, and the paged cache
# ---------------------------------------------------------------------------
# A call's host time is a large part of a short one's, so the wrappers below look each thing up once, and take the
# current stream's handle by torch's own accessor where there is one (0.1 us; a torch.cuda.Stream object costs 3 us,
# as much as the launch of a kernel).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _index(t) -> int:
    """The CUDA device of the call's first tensor."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must live on a CUDA device")
    return index


def _dense_on(index, *ts):
    for t in ts:
        if t.get_device() != index:
            raise ValueError(f"a tensor is on {t.device}, the first one on cuda:{index}: all must live on one device")
        if not t.is_contiguous():
            raise ValueError("tensors must be dense")


def _call(fn, args, need, workspace, after, index, stream):
    """fn(*args, workspace, its bytes, *after, stream) on `stream` (None: the current one of the tensors' device),
    where a workspace of `need` bytes is allocated if the caller gave none; need None: the call takes no workspace."""
    if stream is not None or torch.cuda.current_device() != index:
        if stream is None:
            place = torch.cuda.device(index)
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=index)
            if stream.device.index != index:
                raise ValueError(f"the stream is of {stream.device}, the tensors are on cuda:{index}")
            place = torch.cuda.stream(stream)
        with place:
            return _call(fn, args, need, workspace, after, index, None)
    if need is None:
        status = fn(*args, *after, _raw_stream(index))
    elif workspace is not None:
        _dense_on(index, workspace)
        status = fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), *after, _raw_stream(index))
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=index)
        status = fn(*args, workspace.data_ptr(), need, *after, _raw_stream(index))
    else:
        status = fn(*args, None, 0, *after, _raw_stream(index))
    if status:
        raise CpError(status, fn.__name__)


def _i32(name, t, shape):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}")


def _slopes(slopes, H, index):
    if slopes.dtype != torch.float32 or slopes.shape != (H,):
        raise ValueError("slopes must be float32 [H]")
    _dense_on(index, slopes)
    return slopes.data_ptr()


def _score_rule(B, H, Sq, Skv, index, softcap, slopes, causal, prefix_lens, q_docs, kv_docs, q_pos0, kv_pos0):
    r = _lib.ScoreRule(float(softcap), None, bool(causal), None, None, None, int(q_pos0), int(kv_pos0))
    if slopes is not None:
        r.slopes = _slopes(slopes, H, index)
    # an empty tensor has no address; no row reads it
    if prefix_lens is not None:
        _i32("prefix_lens", prefix_lens, (B,))
        _dense_on(index, prefix_lens)
        r.prefix_lens = prefix_lens.data_ptr() or 256
    if q_docs is not None or kv_docs is not None:
        if q_docs is None or kv_docs is None:
            raise ValueError("q_docs and kv_docs come together")
        _i32("q_docs", q_docs, (B, Sq))
        _i32("kv_docs", kv_docs, (B, Skv))
        _dense_on(index, q_docs, kv_docs)
        r.q_docs, r.kv_docs = q_docs.data_ptr() or 256, kv_docs.data_ptr() or 256
    return ctypes.byref(r)


def cp_scored_attn_validate(B, H, Hkv, Sq, Skv, D, scale=1.0, softcap=0.0, causal=False, prefix=False,
                            dtype=torch.bfloat16, q_pos0=0, kv_pos0=0) -> int:
    """Status code of cp_scored_attn_fwd's checks of sizes and rule (0 = ok). Host only."""
    r = _lib.ScoreRule(softcap=float(softcap), causal=int(bool(causal)), prefix_lens=256 if prefix else None,
                       q_pos0=int(q_pos0), kv_pos0=int(kv_pos0))
    return lib().cp_scored_attn_validate(B, H, Hkv, Sq, Skv, D, float(scale), ctypes.byref(r), _DT[dtype])


def cp_scored_attn_workspace_size(B, H, Sq, Skv, docs=False) -> int:
    return int(lib().cp_scored_attn_workspace_size(B, H, Sq, Skv, int(bool(docs))))


def cp_scored_attn_bwd_workspace_size(B, H, Sq, Skv, docs=False) -> int:
    return int(lib().cp_scored_attn_bwd_workspace_size(B, H, Sq, Skv, int(bool(docs))))


def cp_scored_attn_fwd(q, k, v, out, lse, scale: float, softcap: float = 0.0, slopes=None, causal: bool = False,
                       prefix_lens=None, q_docs=None, kv_docs=None, q_pos0: int = 0, kv_pos0: int = 0, workspace=None,
                       stream=None):
    """Attention of q [B,Sq,H,D] over k, v [B,Skv,Hkv,D] (H a multiple of Hkv) with a score rule ->
    out [B,Sq,H,D] (float32 or q's dtype), lse [B,H,Sq] f32.

    Scores scale * q.k are capped to softcap * tanh(x / softcap) (softcap > 0), lose slopes[h] * distance
    (slopes: float32 [H]), and take part iff causal is off, the key's position is not after the query's, or it is
    below prefix_lens[b] (int32 [B]), and iff q_docs and kv_docs (int32 [B,Sq], [B,Skv]; negative: padding) agree.
    Row 0 of q and of k has the position q_pos0 and kv_pos0. workspace: a CUDA tensor of at least
    cp_scored_attn_workspace_size(...) bytes; allocated here through torch when None.
    """
    index, dtype = _index(q), q.dtype
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, Sq, H, D], k and v [B, Skv, Hkv, D]")
    B, Sq, H, D = q.shape
    _, Skv, Hkv, _ = k.shape
    if k.shape != (B, Skv, Hkv, D) or v.shape != k.shape or out.shape != q.shape or lse.shape != (B, H, Sq):
        raise ValueError("shape mismatch")
    if k.dtype != dtype or v.dtype != dtype or lse.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; lse must be float32")
    if out.dtype != dtype and out.dtype != torch.float32:
        raise TypeError(f"out must be float32 or {dtype}")
    _dense_on(index, q, k, v, out, lse)
    rule = _score_rule(B, H, Sq, Skv, index, softcap, slopes, causal, prefix_lens, q_docs, kv_docs, q_pos0, kv_pos0)
    L = lib()
    _call(L.cp_scored_attn_fwd, (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Hkv, Sq,
                                 Skv, D, float(scale), rule),
          0 if q_docs is None else L.cp_scored_attn_workspace_size(B, H, Sq, Skv, 1), workspace,
          (_dt(q), _DT[out.dtype]), index, stream)


def cp_scored_attn_bwd(q, k, v, out, dout, lse, dq, dk, dv, scale: float, softcap: float = 0.0, slopes=None,
                       causal: bool = False, prefix_lens=None, q_docs=None, kv_docs=None, q_pos0: int = 0,
                       kv_pos0: int = 0, workspace=None, stream=None):
    """Backward of cp_scored_attn_fwd: dout [B,Sq,H,D] (q's dtype), out (float32 or q's dtype) and lse from the
    forward -> dq [B,Sq,H,D], dk, dv [B,Skv,Hkv,D] (all float32 or all q's dtype; written).

    For a block of a ring, out and lse are the row's results over all blocks, and the blocks' gradients add up.
    workspace: a CUDA tensor of at least cp_scored_attn_bwd_workspace_size(...) bytes; allocated here when None.
    """
    index, dtype = _index(q), q.dtype
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, Sq, H, D], k and v [B, Skv, Hkv, D]")
    qs, ks = q.shape, k.shape
    B, Sq, H, D = qs
    _, Skv, Hkv, _ = ks
    if ks != (B, Skv, Hkv, D) or v.shape != ks or dk.shape != ks or dv.shape != ks or lse.shape != (B, H, Sq):
        raise ValueError("shape mismatch")
    if out.shape != qs or dout.shape != qs or dq.shape != qs:
        raise ValueError("shape mismatch")
    if k.dtype != dtype or v.dtype != dtype or dout.dtype != dtype or lse.dtype != torch.float32:
        raise TypeError("q, k, v and dout must share a dtype; lse must be float32")
    gtype = dq.dtype
    if dk.dtype != gtype or dv.dtype != gtype:
        raise TypeError("dq, dk and dv must share a dtype")
    for t in (out.dtype, gtype):
        if t != dtype and t != torch.float32:
            raise TypeError(f"out and the gradients must be float32 or {dtype}")
    _dense_on(index, q, k, v, out, dout, lse, dq, dk, dv)
    rule = _score_rule(B, H, Sq, Skv, index, softcap, slopes, causal, prefix_lens, q_docs, kv_docs, q_pos0, kv_pos0)
    L = lib()
    _call(L.cp_scored_attn_bwd, (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), dout.data_ptr(),
                                 lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Hkv, Sq, Skv, D,
                                 float(scale), rule),
          L.cp_scored_attn_bwd_workspace_size(B, H, Sq, Skv, q_docs is not None), workspace,
          (_dt(q), _DT[out.dtype], _DT[gtype]), index, stream)


def _paged_shapes(k_cache, v_cache, block_table, seq_lens, B, Hkv, D, dtype):
    """(num_pages, page_size, max_pages)"""
    if k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, Hkv, D], block_table [B, max_pages]")
    pages, page, heads, width = k_cache.shape
    if heads != Hkv or width != D or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, Hkv, D]")
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError("the caches must have the dtype of the other tensors")
    rows, most = block_table.shape
    if rows != B or seq_lens.shape != (B,):
        raise ValueError("block_table must be [B, max_pages], seq_lens [B]")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    return pages, page, most


def cp_paged_kv_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, new_lens=None, stream=None):
    """Writes new tokens k_new, v_new [B,T,Hkv,D] into the pages of k_cache, v_cache [num_pages,page,Hkv,D].

    Token t of sequence b (t < new_lens[b]; all T when new_lens is None) goes to position seq_lens[b] + t: row
    position % page of page block_table[b, position // page]. seq_lens (int32 [B], the lengths before the call) is not
    changed. A position or page out of range is skipped and reported by cp_check_device_status.
    """
    index, dtype = _index(k_new), k_new.dtype
    if k_new.dim() != 4 or v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must be [B, T, Hkv, D]")
    if v_new.dtype != dtype:
        raise TypeError("k_new and v_new must share a dtype")
    B, T, Hkv, D = k_new.shape
    pages, page, most = _paged_shapes(k_cache, v_cache, block_table, seq_lens, B, Hkv, D, dtype)
    _dense_on(index, k_new, v_new, k_cache, v_cache, block_table, seq_lens)
    news = None
    if new_lens is not None:
        _i32("new_lens", new_lens, (B,))
        _dense_on(index, new_lens)
        news = new_lens.data_ptr()
    _call(lib().cp_paged_kv_append, (k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                     block_table.data_ptr() or 256, seq_lens.data_ptr(), news, B, T, Hkv, D, pages,
                                     page, most, _dt(k_new)), None, None, (), index, stream)


def cp_paged_attn_workspace_size(B, H, Hkv, D, dtype=torch.bfloat16, page_size=None, max_pages=None) -> int:
    """Workspace bytes of cp_paged_attn_decode for any table, or for tables of max_pages pages of page_size rows (0
    where such a call needs none)."""
    if page_size is None or max_pages is None:
        return int(lib().cp_paged_attn_workspace_size(B, H, Hkv, D, _DT[dtype]))
    return int(lib().cp_paged_attn_workspace_size_for(B, H, Hkv, D, page_size, max_pages, _DT[dtype]))


def cp_paged_attn_decode(q, k_cache, v_cache, block_table, seq_lens, out, lse, scale: float, softcap: float = 0.0,
                         slopes=None, workspace=None, stream=None):
    """Attention of one new token per sequence, q [B,H,D], over its seq_lens[b] tokens in the paged cache (the new
    one among them, the last) -> out [B,H,D] (float32 or q's dtype), lse [B,H] f32.

    softcap and slopes as in cp_scored_attn_fwd, the query's position being seq_lens[b] - 1. A sequence of length 0
    gets out 0, lse -inf. workspace: a CUDA tensor of at least cp_paged_attn_workspace_size(...) bytes, one for each
    call that may run at the same time; allocated here through torch when None.
    """
    index, dtype = _index(q), q.dtype
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B, H, D], the caches [num_pages, page_size, Hkv, D]")
    B, H, D = q.shape
    Hkv = k_cache.shape[2]
    if out.shape != q.shape or lse.shape != (B, H):
        raise ValueError("shape mismatch")
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    if out.dtype != dtype and out.dtype != torch.float32:
        raise TypeError(f"out must be float32 or {dtype}")
    pages, page, most = _paged_shapes(k_cache, v_cache, block_table, seq_lens, B, Hkv, D, dtype)
    _dense_on(index, q, k_cache, v_cache, block_table, seq_lens, out, lse)
    L, dt = lib(), _dt(q)
    _call(L.cp_paged_attn_decode, (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                   seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, Hkv, D, pages, page, most,
                                   float(scale), float(softcap), None if slopes is None else _slopes(slopes, H, index)),
          L.cp_paged_attn_workspace_size_for(B, H, Hkv, D, page, most, dt), workspace, (dt, _DT[out.dtype]), index, stream)


def cp_check_device_status(stream=None) -> int:
    """Synchronizes the stream; returns 0, CP_ERR_TIMEOUT if a kernel's bounded wait expired, or CP_ERR_INVALID_ARG
    if a paged-cache kernel met a page index or a sequence length out of range."""
    return int(lib().cp_check_device_status(_stream(stream)))


def cp_debug_bounded_wait_probe(timeout_us: int, stream=None):
    check(lib().cp_debug_bounded_wait_probe(int(timeout_us), _stream(stream)), "cp_debug_bounded_wait_probe")


def cp_status_string(status: int) -> str:
    return _lib.status_string(status)


def cp_version() -> int:
    return int(lib().cp_version())


__all__ = [
    "CpError", "cp_block_attn_fwd", "cp_lse_merge", "cp_ulysses_seq2head", "cp_ulysses_head2seq",
    "cp_ulysses_anything_seq2head", "cp_ulysses_anything_head2seq",
    "cp_attention_validate", "cp_ring_shard_table", "cp_attention_workspace_size", "cp_attention_launch_count",
    "cp_attention_bwd", "cp_attention_bwd_workspace_size", "cp_attention_bwd_launch_count",
    "cp_attention_fwd", "cp_attention_fwd_no_alloc", "cp_attention_fwd_host", "cp_attention_host_buffer_size", "cp_check_device_status", "cp_debug_bounded_wait_probe",
    "cp_scored_attn_validate", "cp_scored_attn_workspace_size", "cp_scored_attn_bwd_workspace_size",
    "cp_scored_attn_fwd", "cp_scored_attn_bwd", "cp_paged_kv_append", "cp_paged_attn_workspace_size",
    "cp_paged_attn_decode", "cp_status_string", "cp_version",
]
