"""The per-layer path as a sequence of libkq calls.

Torch supplies device memory and the stream; every step runs in the
library's kernels. H_G is released as soon as BiIP has used it: the column
sweep never reads it, so the extra dout x dout memory lives only through the
preprocessing.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import numpy as np

from . import (KQ_BIIP_INPUT, KQ_BIIP_INVERSE, KQ_BIIP_OUTPUT, KQ_BIIP_SCALE, KQ_SCORE_KRONQ, KQError,
               KQ_EINVAL, KQ_ENOTPD, CacheBatch, KVCache, Rot, _need, accumulate_cov, accumulate_xcov, biip_rotate,
               biip_transform, cache_append, cache_attention, cache_attention_workspace, cholesky_inv,
               decode_matvec_group, decode_workspace, gptaq_target, make_rot, obs_quantize, sensitivity)

ALL_SIDES = KQ_BIIP_INPUT | KQ_BIIP_OUTPUT | KQ_BIIP_SCALE


@dataclass
class DeviceRot:
    """A rotation spec resident on the device (the tensors back the C struct)."""
    signs: object
    q: object
    rot: Rot


def upload_rot(signs: np.ndarray, q: np.ndarray, device) -> DeviceRot:
    import torch
    s = torch.from_numpy(np.ascontiguousarray(signs, dtype=np.int8)).to(device)
    qq = torch.from_numpy(np.ascontiguousarray(q, dtype=np.float64)).to(device)
    return DeviceRot(s, qq, make_rot(s, qq))


def covariance(a, *, out=None, chunk_rows: Optional[int] = None, stream=None):
    """H = A^T A / N for bf16 A [N, d] on the device (one call, or chunked with beta = 1)."""
    import torch
    n, d = a.shape
    h = torch.empty((d, d), dtype=torch.float32, device=a.device) if out is None else out
    if chunk_rows is None or chunk_rows >= n:
        accumulate_cov(a, h, 1.0 / n, 0.0, stream=stream)
        return h
    for i, r0 in enumerate(range(0, n, chunk_rows)):
        accumulate_cov(a[r0:r0 + chunk_rows], h, 1.0 / n, 0.0 if i == 0 else 1.0, stream=stream)
    return h


def drift_moment(xt, x, h_x, *, out=None, stream=None):
    """D = (Xt - X)^T X / N from the full-precision inputs Xt and the quantized-model inputs X
    (bf16 [N, d], the same tokens) and H_X = X^T X / N: one cross-moment call with beta = -1."""
    import torch
    n, d = x.shape
    dm = torch.empty((d, d), dtype=torch.float32, device=x.device) if out is None else out
    accumulate_xcov(xt, x, dm, 1.0 / n, -1.0, c_in=h_x, stream=stream)
    return dm


@dataclass
class LayerOut:
    w2: object          # rotated weight W'' (float64), overwritten by the dequantised W^''
    hx2: object         # H_X'' (float32), overwritten by R
    s_x: object
    s_g: object
    codes: object
    scales: object
    zeros: object
    info: object
    w_hat: Optional[object] = None


def quantize_layer(w, h_x, h_g, rot_in: DeviceRot, rot_out: DeviceRot, *, bits: int, group: int, block: int,
                   damp: float, flags: int = ALL_SIDES, keep_inputs: bool = True, unrotate: bool = True,
                   check_info: bool = True, preround=None, d_x=None, stream=None) -> LayerOut:
    """BiIP -> damped Cholesky factor of the inverse -> OBS sweep (-> un-rotation).

    ``h_x`` / ``h_g`` are the raw covariances; with ``keep_inputs`` they are
    copied first (the library transforms them in place). ``d_x`` (the drift moment of
    ``drift_moment``) selects the GPTAQ base quantizer: D'' by the input-side map, then the
    drift correction of W'' before the sweep."""
    import torch
    dev = w.device
    dout, din = w.shape
    hx = h_x.clone() if keep_inputs else h_x
    hg = None
    if flags & KQ_BIIP_OUTPUT:
        hg = h_g.clone() if keep_inputs else h_g
    w2 = torch.empty((dout, din), dtype=torch.float64, device=dev)
    s_x = torch.empty(din, dtype=torch.float64, device=dev)
    s_g = torch.empty(dout, dtype=torch.float64, device=dev)
    biip_rotate(w, w2, hx, hg, rot_in.rot if flags & KQ_BIIP_INPUT else None,
                rot_out.rot if flags & KQ_BIIP_OUTPUT else None, flags, s_x, s_g, stream=stream)
    del hg  # H_G'' is not needed by anything after BiIP
    d2 = None
    if d_x is not None:
        d2 = d_x.clone() if keep_inputs else d_x
        if flags & KQ_BIIP_INPUT:
            biip_transform(d2, rot_in.rot, s_x, stream=stream)
    info = torch.zeros(1, dtype=torch.int32, device=dev)
    cholesky_inv(hx, damp, info, stream=stream)
    if check_info:
        bad = int(info.item())
        if bad:
            raise KQError(KQ_ENOTPD, f"damped H_X'' is not positive definite at index {bad - 1}")
    if d2 is not None:
        info_t = torch.zeros(1, dtype=torch.int32, device=dev)
        gptaq_target(w2, d2, hx, info=info_t, stream=stream)
        del d2
        if check_info and int(info_t.item()):
            raise KQError(KQ_EINVAL, "the drift correction produced non-finite weights "
                                     "(the drift moment holds a NaN or Inf)")
    ng = din // group if group else 1
    codes = torch.empty((dout, din), dtype=torch.uint8, device=dev)
    scales = torch.empty((dout, ng), dtype=torch.float32, device=dev)
    zeros = torch.empty((dout, ng), dtype=torch.uint8, device=dev)
    obs_quantize(w2, hx, bits, group, block, codes, scales, zeros, preround, stream=stream)
    out = LayerOut(w2, hx, s_x, s_g, codes, scales, zeros, info)
    if unrotate:
        w_hat = torch.empty((dout, din), dtype=torch.float64, device=dev)
        biip_rotate(w2, w_hat, None, None, rot_in.rot if flags & KQ_BIIP_INPUT else None,
                    rot_out.rot if flags & KQ_BIIP_OUTPUT else None, flags | KQ_BIIP_INVERSE, s_x, s_g,
                    stream=stream)
        out.w_hat = w_hat
    return out


def score(h_x, h_g, mode: int = KQ_SCORE_KRONQ, stream=None) -> float:
    import torch
    s = torch.empty(1, dtype=torch.float64, device=h_x.device)
    sensitivity(h_x, h_g, s, mode, stream=stream)
    return float(s.item())


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device=None):
    """Rotation table for cache_append: float32 [positions, rot_dim], row p holding cos then sin of
    p base^(-2j / rot_dim), j < rot_dim / 2, computed in float64 (far positions lose their angle in float32)."""
    import torch
    j = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    angle = torch.outer(torch.arange(positions, dtype=torch.float64, device=device), base ** (-2.0 * j / rot_dim))
    return torch.cat((angle.cos(), angle.sin()), 1).to(torch.float32)


def attention_step(x, qkv, o, cache: KVCache, batch: CacheBatch, heads: int, *, bits: int, group: int, s_x, rot_in,
                   o_s_x, o_rot_in, q_norm=None, k_norm=None, eps: float = 1e-6, rope=None, interleaved: bool = False,
                   scale: Optional[float] = None, window: int = 0, info=None, ws=None, stream=None):
    """The attention half of a decoder block on quantized weights, for the new tokens x (float32 [rows, d], at most
    KQ_DECODE_MAX_TOKENS): q, k and v by one decode group call, norm, rotation and append to the 8-bit cache,
    attention over it, the o projection.

    ``qkv``: the three layers as decode_matvec_group takes them, (packed, scales, zeros, s_g, rot_out, y), y float32
    [rows, heads * head_dim] and twice [rows, kv_heads * head_dim]; ``o``: one such layer, din = heads * head_dim.
    ``s_x`` and ``rot_in`` belong to q, k and v, ``o_s_x`` and ``o_rot_in`` to o. Returns o's y. The values in
    qkv's q are replaced by the rotated queries. ``ws`` (from ``attention_step_workspace``) and the layers' y make
    the step free of allocations, so that it can be captured into a graph."""
    import torch
    rows, dim = x.shape[0], cache.head_dim
    y_q, y_k, y_v = (layer[5] for layer in qkv)
    _need(y_q.shape == (rows, heads * dim) and y_k.shape == y_v.shape == (rows, cache.kv_heads * dim),
          "attention_step: the layers' y do not match heads, kv_heads and head_dim")
    if ws is None:
        with torch.cuda.stream(stream):      # memory of the stream that uses it (None: the current one)
            ws = attention_step_workspace(x, qkv, o, cache, batch, heads)
    q = y_q.view(rows, heads, dim)
    decode_matvec_group(qkv, bits, group, s_x, rot_in, x, ws=ws.qkv, stream=stream)
    cache_append(cache, batch, q, y_k.view(rows, cache.kv_heads, dim), y_v.view(rows, cache.kv_heads, dim), q,
                 q_norm=q_norm, k_norm=k_norm, eps=eps, rope=rope, interleaved=interleaved, info=info, stream=stream)
    cache_attention(cache, batch, q, ws.attn.view(rows, heads, dim), scale=scale, window=window, info=info,
                    ws=ws.scratch, stream=stream)
    decode_matvec_group([o], bits, group, o_s_x, o_rot_in, ws.attn, ws=ws.o, stream=stream)
    return o[5]


@dataclass
class StepWorkspace:
    """Buffers of attention_step; steps that share them must not overlap."""
    qkv: object         # decode scratch of the q, k, v call
    o: object           # and of the o call
    attn: object        # the attention's output, float32 [rows, heads * head_dim]
    scratch: object     # cache_attention's workspace


def attention_step_workspace(x, qkv, o, cache: KVCache, batch: CacheBatch, heads: int) -> StepWorkspace:
    """The buffers attention_step needs for inputs like these."""
    import torch
    rows, dev = x.shape[0], x.device
    wide = heads * cache.head_dim
    attn = torch.empty((rows, wide), dtype=torch.float32, device=dev)
    return StepWorkspace(decode_workspace(sum(layer[5].shape[1] for layer in qkv), x.shape[1], rows, dev),
                         decode_workspace(o[5].shape[1], wide, rows, dev), attn,
                         cache_attention_workspace(cache, batch, attn.view(rows, heads, cache.head_dim)))
