"""Python binding of libmoe (include/moe.h): argument marshalling only.

Every function has the name of the C entry point it calls and forwards torch tensors as
raw device pointers plus sizes; every step of the layer runs in the library's own CUDA
kernels.  PyTorch is used for device memory and streams only.  If libmoe.so has not been
built, the first call raises: there is no CPU or PyTorch fallback.
"""
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_BF16, MOE_E4M3, MOE_W4 = 0, 1, 2
MOE_FEW_MAX_TOKENS = 32   # tokens of one few-token call (moe_route_hidden, moe_layer_few)
MOE_W_TILED = 0x100   # ORed into a grouped GEMM dtype: weights in the tile layout of moe_pack_weights
MOE_EPI_NONE, MOE_EPI_SWIGLU = 0, 1
MOE_DEV_BAD_EXPERT, MOE_DEV_VERIFY_MISMATCH, MOE_DEV_PIPELINE_TIMEOUT, MOE_DEV_OVERFLOW = 1, 2, 4, 8
STATUS = {0: "MOE_OK", 1: "MOE_ERR_ARG", 2: "MOE_ERR_WORKSPACE", 3: "MOE_ERR_UNSUPPORTED", 4: "MOE_ERR_CUDA"}

_P, _I, _Z, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong


class MoeError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


class LayerDesc(ctypes.Structure):
    _fields_ = [("T", _I), ("H", _I), ("I", _I), ("E", _I), ("K", _I), ("dtype", _I), ("has_shared", _I),
                ("weight_in_down", _I), ("max_tokens", _I), ("fuse_combine", _I), ("combine_fq_format", _I),
                ("dispatch_fq_format", _I), ("gemm_pairs", _I), ("weight_tiles", _I)]


class LayerWeights(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("w13", "w13_scales", "w2", "w2_scales", "shared_w13", "shared_w13_scales",
                                  "shared_w2", "shared_w2_scales")]


class FewDesc(ctypes.Structure):
    _fields_ = [("T", _I), ("H", _I), ("I", _I), ("E", _I), ("K", _I), ("dtype", _I), ("has_shared", _I),
                ("weight_tiles", _I), ("group", _I), ("zeros", _I)]


class FewWeights(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("w13", "w13_scales", "w2", "w2_scales", "shared_w13", "shared_w13_scales", "shared_w2",
                                  "shared_w2_scales", "w_router", "router_bias")]


class LayerViews(ctypes.Structure):
    _fields_ = [("xp", _P), ("xp_scales", _P), ("hs", _P), ("hs_scales", _P), ("y", _P), ("cu_seqlens", _P),
                ("src_row", _P), ("inv_map", _P), ("shared_map", _P), ("row_weights", _P), ("cap", _I),
                ("masked_m", _P), ("counters", _P)]


# C signatures (restype int = moe_status_t unless noted)
_SIGS = {
    "moe_abi_version": ([], _I),
    "moe_status_string": ([_I], ctypes.c_char_p),
    "moe_route_topk": ([_P, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_permute_workspace_bytes": ([_I, _I, _I, _I], _Z),
    "moe_permute": ([_P, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _Z, _P, _P], _I),
    "moe_permute_noalloc_max_scratch_bytes": ([], _Z),
    "moe_permute_noalloc": ([_P, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P], _I),
    "moe_permute_ex": ([_P, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _Z, _P, _P, _I, _P, _P, _P], _I),
    "moe_permute_batched_workspace_bytes": ([_I, _I, _I, _I], _Z),
    "moe_permute_batched": ([_P, _I, _I, _I, _I, _I, _P, _I, _I, _P, _P, _P, _P, _P, _P, _P, _Z, _P, _P, _I, _P,
                             _P, _P], _I),
    "moe_amax_bf16": ([_P, _Z, _P, _P], _I),
    "moe_quantize_act_fp8": ([_P, _I, _I, _P, _P, _P], _I),
    "moe_quantize_weight_fp8": ([_P, _I, _I, _I, _P, _P, _P], _I),
    "moe_grouped_gemm": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P], _I),
    "moe_grouped_gemm_ex": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P], _I),
    "moe_grouped_gemm_pairs": ([_P, _P, _I, _I, _I, _I, _P, _I, _P, _I, _P, _P, _P, _P], _I),
    "moe_pack_weights": ([_P, _I, _I, _I, _I, _P, _P], _I),
    "moe_grouped_gemm_batched": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P],
                                 _I),
    "moe_grouped_gemm_combine": ([_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, _P, _I,
                                  _I, _P, _P, _P, _P, _P, _P], _I),
    "moe_combine": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "moe_combine_verify": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    "moe_combine_amax": ([_P, _P, _P, _I, _I, _I, _P, _P], _I),
    "moe_fq_scale_from_amax": ([_P, _P, _P], _I),
    "moe_combine_nvfp4": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "moe_fq4_scale_from_amax": ([_P, _P, _P], _I),
    "moe_layer_workspace_bytes": ([ctypes.POINTER(LayerDesc)], _Z),
    "moe_layer_views": ([ctypes.POINTER(LayerDesc), _P, ctypes.POINTER(LayerViews)], _I),
    "moe_layer_forward": ([ctypes.POINTER(LayerDesc), ctypes.POINTER(LayerWeights), _P, _P, _P, _P, _P, _P, _P,
                           _P, _P, _Z, _P, _P], _I),
    "moe_quantize_weight_w4": ([_P, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_w4_packed_bytes": ([_I, _I, _I, _I], _Z),
    "moe_pack_w4": ([_P, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "moe_linear_w4_workspace_bytes": ([_I, _I, _I], _Z),
    "moe_linear_w4": ([_P, _I, _I, _L, _P, _I, _I, _I, _P, _P, _I, _L, _P, _Z, _P, _P], _I),
    "moe_route_hidden_workspace_bytes": ([], _Z),
    "moe_route_hidden": ([_P, _I, _I, _P, _P, _I, _I, _P, _P, _P, _P, _P, _Z, _P], _I),
    "moe_layer_few_workspace_bytes": ([ctypes.POINTER(FewDesc)], _Z),
    "moe_rmsnorm": ([_P, _I, _I, _L, _P, _I, ctypes.c_float, _P, _I, _P, _P, _P, _P, _P, _P], _I),
    "moe_linear_e4m3_workspace_bytes": ([_I, _I, _I], _Z),
    "moe_linear_e4m3": ([_P, _P, _I, _I, _P, _P, _I, _P, _P, _I, _L, _P, _Z, _P, _P], _I),
    "moe_permute_e4m3": ([_P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P, _P, _P, _P], _I),
    "moe_layer_forward_e4m3": ([ctypes.POINTER(LayerDesc), ctypes.POINTER(LayerWeights), _P, _P, _P, _P, _P, _P, _P,
                                _P, _P, _Z, _P, _P], _I),
    "moe_layer_few": ([ctypes.POINTER(FewDesc), ctypes.POINTER(FewWeights), _P, _P, _P, _P, _P, _P, _P, _Z, _P, _P],
                      _I),
}

_lib = None


def lib():
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m combine_moe_route_softmax_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # the current stream's handle without a Stream object around it (3 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn, code):
    if code != 0:
        raise MoeError(fn, code)


def _dev(t):
    assert t.is_cuda and t.is_contiguous(), "expected a contiguous CUDA tensor"
    return t


# ----------------------------------------------------------------------------- calls
def moe_route_topk(logits, K, num_tokens=None, topk_idx=None, topk_w=None, stream=None):
    _dev(logits)
    T, E = logits.shape
    if topk_idx is None:
        topk_idx = torch.empty(T, K, dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty(T, K, dtype=torch.float32, device=logits.device)
    _check("moe_route_topk", lib().moe_route_topk(_ptr(logits), T, E, K, _ptr(num_tokens), _ptr(topk_idx),
                                                  _ptr(topk_w), _stream(stream)))
    return topk_idx, topk_w


def moe_permute_workspace_bytes(T, K, E, with_shared):
    return lib().moe_permute_workspace_bytes(T, K, E, int(with_shared))


def _fmt(name):
    """Fake-quant format name -> the C code (0 E4M3, 1 NVFP4)."""
    if name not in ("e4m3", "nvfp4"):
        raise ValueError("fake-quant format is 'e4m3' or 'nvfp4'")
    return int(name == "nvfp4")


def moe_permute(topk_idx, E, x, with_shared=False, out_dtype=MOE_BF16, ws=None, dev_status=None, stream=None,
                dispatch_scale=None, topk_w=None, dispatch_format="e4m3"):
    """Returns dict(xp, xp_scales, cu_seqlens, src_row, inv_map, shared_map, row_weights).
    dispatch_scale / topk_w select moe_permute_ex (dispatch fake-quant in dispatch_format
    "e4m3" or "nvfp4" / row weights)."""
    _dev(topk_idx)
    _dev(x)
    T, K = topk_idx.shape
    H = x.shape[1]
    dev = x.device
    cap = T * K + (T if with_shared else 0)
    nseg = E + int(with_shared)
    fp8 = out_dtype == MOE_E4M3
    xp = torch.empty(cap, H, dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
    xps = torch.empty(cap, H // 128, dtype=torch.float32, device=dev) if fp8 else None
    cu = torch.empty(nseg + 1, dtype=torch.int32, device=dev)
    src = torch.empty(cap, dtype=torch.int32, device=dev)
    inv = torch.empty(T, K, dtype=torch.int32, device=dev)
    smap = torch.empty(T, dtype=torch.int32, device=dev) if with_shared else None
    nbytes = moe_permute_workspace_bytes(T, K, E, with_shared)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    roww = None
    if dispatch_scale is None and topk_w is None:
        _check("moe_permute", lib().moe_permute(
            _ptr(topk_idx), T, K, E, int(with_shared), _ptr(x), H, out_dtype, _ptr(xp), _ptr(xps), _ptr(cu),
            _ptr(src), _ptr(inv), _ptr(smap), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
            _stream(stream)))
    else:
        if topk_w is not None:
            roww = torch.empty(cap, dtype=torch.float32, device=dev)
        _check("moe_permute_ex", lib().moe_permute_ex(
            _ptr(topk_idx), T, K, E, int(with_shared), _ptr(x), H, out_dtype, _ptr(xp), _ptr(xps), _ptr(cu),
            _ptr(src), _ptr(inv), _ptr(smap), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
            _ptr(dispatch_scale), _fmt(dispatch_format), _ptr(topk_w), _ptr(roww), _stream(stream)))
    return dict(xp=xp, xp_scales=xps, cu_seqlens=cu, src_row=src, inv_map=inv, shared_map=smap, row_weights=roww)


def moe_permute_batched_workspace_bytes(T, K, E, with_shared):
    return lib().moe_permute_batched_workspace_bytes(T, K, E, int(with_shared))


def moe_permute_batched(topk_idx, E, x, max_tokens, with_shared=False, out_dtype=MOE_BF16, ws=None,
                        dev_status=None, stream=None, dispatch_scale=None, topk_w=None, dispatch_format="e4m3"):
    """Batched layout: returns dict(xb [nseg, max_tokens, H], xb_scales, masked_m [nseg], src_row
    [nseg * max_tokens], inv_map, shared_map, row_weights)."""
    _dev(topk_idx)
    _dev(x)
    T, K = topk_idx.shape
    H = x.shape[1]
    dev = x.device
    nseg = E + int(with_shared)
    rows = nseg * max_tokens
    fp8 = out_dtype == MOE_E4M3
    xb = torch.empty(nseg, max_tokens, H, dtype=torch.uint8 if fp8 else torch.bfloat16, device=dev)
    xbs = torch.empty(nseg, max_tokens, H // 128, dtype=torch.float32, device=dev) if fp8 else None
    mm = torch.empty(nseg, dtype=torch.int32, device=dev)
    src = torch.empty(rows, dtype=torch.int32, device=dev)
    inv = torch.empty(T, K, dtype=torch.int32, device=dev)
    smap = torch.empty(T, dtype=torch.int32, device=dev) if with_shared else None
    roww = torch.empty(rows, dtype=torch.float32, device=dev) if topk_w is not None else None
    if ws is None:
        ws = torch.empty(moe_permute_batched_workspace_bytes(T, K, E, with_shared), dtype=torch.uint8, device=dev)
    _check("moe_permute_batched", lib().moe_permute_batched(
        _ptr(topk_idx), T, K, E, int(with_shared), max_tokens, _ptr(x), H, out_dtype, _ptr(xb), _ptr(xbs), _ptr(mm),
        _ptr(src), _ptr(inv), _ptr(smap), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
        _ptr(dispatch_scale), _fmt(dispatch_format), _ptr(topk_w), _ptr(roww), _stream(stream)))
    return dict(xb=xb, xb_scales=xbs, masked_m=mm, src_row=src, inv_map=inv, shared_map=smap, row_weights=roww)


def moe_quantize_act_fp8(x, stream=None):
    _dev(x)
    R, C = x.shape
    q = torch.empty(R, C, dtype=torch.uint8, device=x.device)
    s = torch.empty(R, C // 128, dtype=torch.float32, device=x.device)
    _check("moe_quantize_act_fp8", lib().moe_quantize_act_fp8(_ptr(x), R, C, _ptr(q), _ptr(s), _stream(stream)))
    return q, s


def moe_quantize_weight_fp8(w, stream=None):
    """w BF16 [..., rows, cols] -> (codes uint8 same shape, scales float32 [..., rows/128, cols/128])."""
    _dev(w)
    rows, cols = w.shape[-2:]
    mats = w.numel() // (rows * cols)
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    s = torch.empty(*w.shape[:-2], rows // 128, cols // 128, dtype=torch.float32, device=w.device)
    _check("moe_quantize_weight_fp8", lib().moe_quantize_weight_fp8(_ptr(w), mats, rows, cols, _ptr(q), _ptr(s),
                                                                    _stream(stream)))
    return q, s


def moe_pack_weights(w, out=None, stream=None):
    """w [..., n, k] (bf16, or uint8 E4M3 codes) -> a tensor of the same shape and dtype
    holding the same bytes in the tile layout of moe_pack_weights (pass it with tiled=True
    or to MoeLayer(weight_tiles=True) only: its rows are not w's rows)."""
    _dev(w)
    n, k = w.shape[-2:]
    mats = w.numel() // (n * k)
    if out is None:
        out = torch.empty_like(w)
    _dev(out)
    assert out.numel() * out.element_size() == w.numel() * w.element_size(), "out must hold w's bytes"
    dt = MOE_E4M3 if w.dtype == torch.uint8 else MOE_BF16
    _check("moe_pack_weights", lib().moe_pack_weights(_ptr(w), mats, n, k, dt, _ptr(out), _stream(stream)))
    return out


def moe_grouped_gemm(a, cu_seqlens, w, n_segments=None, a_scales=None, w_scales=None, w_extra=None,
                     w_extra_scales=None, epilogue=MOE_EPI_NONE, out=None, out_scales=None, dev_status=None,
                     stream=None, row_scale=None, pairs=False, tiled=False):
    """a [rows_cap, k] (bf16 or uint8 E4M3 codes); w [num_w, n, k]; returns (out, out_scales).
    pairs=True: the BF16 computation on pairs of SMs (moe_grouped_gemm_pairs); tiled=True: w
    and w_extra from moe_pack_weights (MOE_W_TILED)."""
    _dev(a)
    fp8 = a.dtype == torch.uint8
    rows_cap, k_dim = a.shape
    num_w, n_dim = w.shape[0], w.shape[1]
    if n_segments is None:
        n_segments = cu_seqlens.numel() - 1
    out_cols = n_dim // 2 if epilogue == MOE_EPI_SWIGLU else n_dim
    if out is None:
        odt = torch.uint8 if (fp8 and epilogue == MOE_EPI_SWIGLU) else torch.bfloat16
        out = torch.empty(rows_cap, out_cols, dtype=odt, device=a.device)
    if fp8 and epilogue == MOE_EPI_SWIGLU and out_scales is None:
        out_scales = torch.empty(rows_cap, out_cols // 128, dtype=torch.float32, device=a.device)
    dt = (MOE_E4M3 if fp8 else MOE_BF16) | (MOE_W_TILED if tiled else 0)
    if pairs:
        _check("moe_grouped_gemm_pairs", lib().moe_grouped_gemm_pairs(
            _ptr(a), _ptr(cu_seqlens), n_segments, rows_cap, k_dim, n_dim, _ptr(w), num_w, _ptr(w_extra), epilogue,
            _ptr(out), _ptr(dev_status), _ptr(row_scale), _stream(stream)))
    elif row_scale is None:
        _check("moe_grouped_gemm", lib().moe_grouped_gemm(
            _ptr(a), _ptr(a_scales), _ptr(cu_seqlens), n_segments, rows_cap, k_dim, n_dim, _ptr(w), _ptr(w_scales),
            num_w, _ptr(w_extra), _ptr(w_extra_scales), dt, epilogue, _ptr(out),
            _ptr(out_scales), _ptr(dev_status), _stream(stream)))
    else:
        _check("moe_grouped_gemm_ex", lib().moe_grouped_gemm_ex(
            _ptr(a), _ptr(a_scales), _ptr(cu_seqlens), n_segments, rows_cap, k_dim, n_dim, _ptr(w), _ptr(w_scales),
            num_w, _ptr(w_extra), _ptr(w_extra_scales), dt, epilogue, _ptr(out),
            _ptr(out_scales), _ptr(dev_status), _ptr(row_scale), _stream(stream)))
    return out, out_scales


def moe_grouped_gemm_batched(a, masked_m, w, a_scales=None, w_scales=None, w_extra=None, w_extra_scales=None,
                             epilogue=MOE_EPI_NONE, out=None, out_scales=None, dev_status=None, stream=None,
                             row_scale=None, tiled=False):
    """a [S, max_tokens, k] (bf16 or uint8 E4M3 codes), masked_m int32 [S]; w [num_w, n, k];
    returns (out [S, max_tokens, n_out], out_scales)."""
    _dev(a)
    fp8 = a.dtype == torch.uint8
    S, max_tokens, k_dim = a.shape
    num_w, n_dim = w.shape[0], w.shape[1]
    out_cols = n_dim // 2 if epilogue == MOE_EPI_SWIGLU else n_dim
    if out is None:
        odt = torch.uint8 if (fp8 and epilogue == MOE_EPI_SWIGLU) else torch.bfloat16
        out = torch.empty(S, max_tokens, out_cols, dtype=odt, device=a.device)
    if fp8 and epilogue == MOE_EPI_SWIGLU and out_scales is None:
        out_scales = torch.empty(S, max_tokens, out_cols // 128, dtype=torch.float32, device=a.device)
    _check("moe_grouped_gemm_batched", lib().moe_grouped_gemm_batched(
        _ptr(a), _ptr(a_scales), _ptr(masked_m), S, max_tokens, k_dim, n_dim, _ptr(w), _ptr(w_scales), num_w,
        _ptr(w_extra), _ptr(w_extra_scales), (MOE_E4M3 if fp8 else MOE_BF16) | (MOE_W_TILED if tiled else 0),
        epilogue, _ptr(out), _ptr(out_scales), _ptr(dev_status), _ptr(row_scale), _stream(stream)))
    return out, out_scales


def moe_grouped_gemm_combine(a, seg, w, src_row, inv_map, topk_w, max_tokens=0, shared_map=None, fq_scale=None,
                             a_scales=None, w_scales=None, w_extra=None, w_extra_scales=None, row_scale=None, y=None,
                             out=None, counters=None, dev_status=None, stream=None, tiled=False):
    """Down projection with the combine fused: a [rows, k] (or [S, max_tokens, k] with seg =
    masked_m and max_tokens > 0; else seg = cu_seqlens), w [num_w, H, k]; returns (out [T, H],
    y [rows, H], counters)."""
    _dev(a)
    fp8 = a.dtype == torch.uint8
    k_dim = a.shape[-1]
    rows = a.numel() // k_dim
    num_w, H = w.shape[0], w.shape[1]
    T, K = inv_map.shape
    nseg = seg.numel() if max_tokens else seg.numel() - 1
    if y is None:
        y = torch.empty(rows, H, dtype=torch.bfloat16, device=a.device)
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=a.device)
    if counters is None:
        counters = torch.zeros(T, H // 128, dtype=torch.int32, device=a.device)
    _check("moe_grouped_gemm_combine", lib().moe_grouped_gemm_combine(
        _ptr(a), _ptr(a_scales), _ptr(seg), nseg, max_tokens, rows, k_dim, H, _ptr(w), _ptr(w_scales), num_w,
        _ptr(w_extra), _ptr(w_extra_scales), (MOE_E4M3 if fp8 else MOE_BF16) | (MOE_W_TILED if tiled else 0),
        _ptr(y), _ptr(row_scale), _ptr(src_row), _ptr(inv_map), _ptr(topk_w), T, K, _ptr(shared_map),
        _ptr(fq_scale), _ptr(out), _ptr(counters), _ptr(dev_status), _stream(stream)))
    return out, y, counters


def moe_combine(y, inv_map, topk_w, shared_y=None, shared_map=None, fq_scale=None, out=None, stream=None):
    _dev(y)
    T, K = inv_map.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    _check("moe_combine", lib().moe_combine(_ptr(y), _ptr(inv_map), _ptr(topk_w), T, K, H, _ptr(shared_y),
                                            _ptr(shared_map), _ptr(fq_scale), _ptr(out), _stream(stream)))
    return out


def moe_combine_nvfp4(y, inv_map, topk_w, g_scale, shared_y=None, shared_map=None, out=None, stream=None):
    """Combine with the NVFP4 fake-quant of every routed row (g_scale: the per-tensor
    scale from moe_fq4_scale_from_amax)."""
    _dev(y)
    T, K = inv_map.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    _check("moe_combine_nvfp4", lib().moe_combine_nvfp4(_ptr(y), _ptr(inv_map), _ptr(topk_w), T, K, H,
                                                        _ptr(shared_y), _ptr(shared_map), _ptr(g_scale), _ptr(out),
                                                        _stream(stream)))
    return out


def moe_combine_verify(y, inv_map, topk_w, expected, dev_status, shared_y=None, shared_map=None, fq_scale=None,
                       stream=None):
    T, K = inv_map.shape
    H = y.shape[1]
    _check("moe_combine_verify", lib().moe_combine_verify(
        _ptr(y), _ptr(inv_map), _ptr(topk_w), T, K, H, _ptr(shared_y), _ptr(shared_map), _ptr(fq_scale),
        _ptr(expected), _ptr(dev_status), _stream(stream)))


def moe_combine_amax(y, inv_map, topk_w, amax, stream=None):
    T, K = inv_map.shape
    _check("moe_combine_amax", lib().moe_combine_amax(_ptr(y), _ptr(inv_map), _ptr(topk_w), T, K, y.shape[1],
                                                      _ptr(amax), _stream(stream)))
    return amax


def moe_amax_bf16(x, amax, stream=None):
    _dev(x)
    _check("moe_amax_bf16", lib().moe_amax_bf16(_ptr(x), x.numel(), _ptr(amax), _stream(stream)))
    return amax


def moe_fq_scale_from_amax(amax, scale=None, stream=None):
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=amax.device)
    _check("moe_fq_scale_from_amax", lib().moe_fq_scale_from_amax(_ptr(amax), _ptr(scale), _stream(stream)))
    return scale


def moe_fq4_scale_from_amax(amax, scale=None, stream=None):
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=amax.device)
    _check("moe_fq4_scale_from_amax", lib().moe_fq4_scale_from_amax(_ptr(amax), _ptr(scale), _stream(stream)))
    return scale


class MoeLayer:
    """Holds a layer's descriptor, weight pointers and workspace; forward() is one
    moe_layer_forward call.  Weights: w13 [E, 2I, H], w2 [E, H, I] (+ shared [2I, H],
    [H, I]) in BF16, or E4M3 codes with their 128x128 scales for dtype MOE_E4M3.
    weight_tiles=True: the layer keeps copies of the four weight tensors in the tile layout
    of moe_pack_weights (made once here) and computes from those."""

    def __init__(self, T, H, I, E, K, dtype=MOE_BF16, w13=None, w2=None, shared_w13=None, shared_w2=None,
                 w13_scales=None, w2_scales=None, shared_w13_scales=None, shared_w2_scales=None, device="cuda",
                 weight_in_down=False, max_tokens=0, fuse_combine=False, combine_fq="e4m3", dispatch_fq="e4m3",
                 gemm_pairs=False, weight_tiles=False):
        self.desc = LayerDesc(T, H, I, E, K, dtype, int(shared_w13 is not None), int(weight_in_down),
                              int(max_tokens), int(fuse_combine), _fmt(combine_fq), _fmt(dispatch_fq),
                              int(gemm_pairs), int(weight_tiles))
        if weight_tiles:
            w13, w2, shared_w13, shared_w2 = (None if t is None else moe_pack_weights(t)
                                              for t in (w13, w2, shared_w13, shared_w2))
        self.tensors = (w13, w2, shared_w13, shared_w2, w13_scales, w2_scales, shared_w13_scales, shared_w2_scales)
        self.weights = LayerWeights(_ptr(w13), _ptr(w13_scales), _ptr(w2), _ptr(w2_scales), _ptr(shared_w13),
                                    _ptr(shared_w13_scales), _ptr(shared_w2), _ptr(shared_w2_scales))
        nbytes = lib().moe_layer_workspace_bytes(ctypes.byref(self.desc))
        if nbytes == 0:
            raise MoeError("moe_layer_workspace_bytes", 1)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.views = LayerViews()
        _check("moe_layer_views", lib().moe_layer_views(ctypes.byref(self.desc), _ptr(self.ws),
                                                         ctypes.byref(self.views)))

    def view(self, name, shape, dtype):
        """A torch tensor over one workspace region (see LayerViews)."""
        ptr = getattr(self.views, name)
        n = 1
        for s in shape:
            n *= s
        base = _ptr(self.ws)
        off = ptr - base
        return self.ws[off:off + n * torch.empty(0, dtype=dtype).element_size()].view(dtype).view(*shape)

    def forward(self, x, out, topk_idx, topk_w, logits=None, num_tokens=None, fq_scale=None, dev_status=None,
                stream=None, dispatch_scale=None, x_scales=None):
        """x_scales float32 [T, H/128]: x holds E4M3 codes (moe_layer_forward_e4m3; an E4M3 layer)."""
        if x_scales is not None:
            return self._forward_e4m3(x, x_scales, out, topk_idx, topk_w, logits, num_tokens, fq_scale, dev_status,
                                      stream, dispatch_scale)
        _check("moe_layer_forward", lib().moe_layer_forward(
            ctypes.byref(self.desc), ctypes.byref(self.weights), _ptr(logits), _ptr(num_tokens), _ptr(topk_idx),
            _ptr(topk_w), _ptr(x), _ptr(fq_scale), _ptr(dispatch_scale), _ptr(out), _ptr(self.ws), self.ws.numel(),
            _ptr(dev_status), _stream(stream)))
        return out

    def _forward_e4m3(self, x, x_scales, out, topk_idx, topk_w, logits, num_tokens, fq_scale, dev_status, stream,
                      dispatch_scale):
        d = self.desc
        _need(d.dtype == MOE_E4M3, "x_scales: E4M3 rows go through an E4M3 layer")
        _need(dispatch_scale is None, "E4M3 rows take no dispatch fake-quantisation")
        _need_codes(x, d.T, d.H, "x")
        _need_tensor(x_scales, torch.float32, (d.T, d.H // 128), "x_scales")
        _need_tensor(out, torch.bfloat16, (d.T, d.H), "out")
        _need_tensor(topk_idx, torch.int32, (d.T, d.K), "topk_idx")
        _need_tensor(topk_w, torch.float32, (d.T, d.K), "topk_w")
        _need_tensor(logits, torch.float32, (d.T, d.E), "logits")
        _need_word(num_tokens, "num_tokens")
        _need_word(dev_status, "dev_status")
        _need(fq_scale is None or isinstance(fq_scale, int) or (fq_scale.dtype is torch.float32 and fq_scale.numel() >= 1),
              "fq_scale is a float32 on the GPU")
        dev = _here()
        for t in (x, x_scales, out, topk_idx, topk_w, logits, num_tokens, fq_scale, dev_status, self.ws):
            if isinstance(t, torch.Tensor) and t.get_device() != dev:
                _refuse("MoeLayer.forward")
        _check("moe_layer_forward_e4m3", lib().moe_layer_forward_e4m3(
            ctypes.byref(self.desc), ctypes.byref(self.weights), _ptr(logits), _ptr(num_tokens), _ptr(topk_idx),
            _ptr(topk_w), _ptr(x), _ptr(x_scales), _ptr(fq_scale), _ptr(out), _ptr(self.ws), self.ws.numel(),
            _ptr(dev_status), _stream(stream)))
        return out


# ------------------------------------------------------------------------ a few tokens
# These calls' workspaces have to be zero at first use, so what a call makes itself (a workspace, its outputs)
# is made on the stream it runs on: with stream=s a call is what it is inside torch.cuda.stream(s).
# As with any tensor, what was made on another stream (inputs, weights, a workspace or layer object) has to
# be finished there first.
def _run_on(stream, f, *args, **kw):
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return f(*args, **kw)


# The kernels read what they are given by its address: type, size and layout are compared here.
def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _need_tensor(t, dtype, shape, what):
    """t: a contiguous GPU tensor of dtype and shape (one dimension: that many values), an address, or None."""
    if t is None or isinstance(t, int):
        return
    fits = t.shape == shape if len(shape) > 1 else t.numel() == shape[0]
    if not (fits and t.dtype is dtype and t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{what}: expected a contiguous {dtype} GPU tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _need_rows(t, dtype, rows, cols, what):
    """t: a contiguous GPU tensor of dtype with `rows` rows or more (the rest is left alone), an address, or None."""
    if t is None or isinstance(t, int):
        return
    if not (t.dim() == 2 and t.shape[0] >= rows and t.shape[1] == cols and t.dtype is dtype and t.is_cuda and
            t.is_contiguous()):
        raise ValueError(f"{what}: expected a contiguous {dtype} GPU tensor of {rows} rows of {cols}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _need_matrices(t, dtypes, mats, n, k, what):
    """t: `mats` matrices of n rows and k columns, [mats, n, k] or for one [n, k]; an address, or None."""
    if t is None or isinstance(t, int):
        return
    if not (t.shape[-2:] == (n, k) and t.numel() == mats * n * k and t.dtype in dtypes and t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{what}: expected {mats} x {n} x {k} of {dtypes[0]}, contiguous, on the GPU, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _need_word(t, what):
    """t: an int32 on the GPU, an address, or None."""
    if t is None or isinstance(t, int):
        return
    if not (t.dtype is torch.int32 and t.is_cuda and t.numel() >= 1):
        raise ValueError(f"{what} is an int32 on the GPU")


class W4Packed:
    """4-bit weights in the kernels' order (moe_pack_w4): `mats` matrices of N rows, K columns,
    scales per `group` columns, zero points or not; data uint8 [mats, bytes].  [i] is one
    matrix of a stack."""

    def __init__(self, data, mats, N, K, group, zeros):
        if data is not None:
            nbytes = lib().moe_w4_packed_bytes(N, K, group, int(zeros))
            _need(nbytes > 0, "no such packed matrix: N, K or group")
            _need_tensor(data, torch.uint8, (mats, nbytes), "packed weights")
        self.data, self.mats, self.N, self.K, self.group, self.zeros = data, mats, N, K, group, zeros

    def __getitem__(self, i):
        if not 0 <= i < self.mats:
            raise IndexError(i)
        return W4Packed(None if self.data is None else self.data[i:i + 1], 1, self.N, self.K, self.group, self.zeros)


def moe_quantize_weight_w4(w, group, zeros=False, stream=None):
    """w BF16 [..., rows, cols] -> (codes uint8 [..., rows, cols/2], scales BF16 [..., cols/group,
    rows], zero points uint8 like scales, or None)."""
    if stream is not None:
        return _run_on(stream, moe_quantize_weight_w4, w, group, zeros)
    _dev(w)
    _need(w.dtype is torch.bfloat16, "w is BF16")
    rows, cols = w.shape[-2:]
    _need(rows > 0 and group in (32, 64, 128) and cols > 0 and cols % group == 0,
          "group is 32, 64 or 128 and divides the columns")
    lead = w.shape[:-2]
    mats = w.numel() // (rows * cols)
    q = torch.empty(*lead, rows, cols // 2, dtype=torch.uint8, device=w.device)
    s = torch.empty(*lead, cols // group, rows, dtype=torch.bfloat16, device=w.device)
    z = torch.empty(*lead, cols // group, rows, dtype=torch.uint8, device=w.device) if zeros else None
    _check("moe_quantize_weight_w4", lib().moe_quantize_weight_w4(_ptr(w), mats, rows, cols, group, _ptr(q), _ptr(s),
                                                                  _ptr(z), _stream(None)))
    return q, s, z


def moe_pack_w4(q, scales, zeros=None, stream=None):
    """Codes [..., N, K/2], scales BF16 [..., K/group, N] and zero points (uint8, like scales, or
    None) -> W4Packed."""
    if stream is not None:
        return _run_on(stream, moe_pack_w4, q, scales, zeros)
    _dev(q)
    _dev(scales)
    _need(q.dtype is torch.uint8 and q.numel() > 0, "codes are uint8, two to a byte")
    N, K = q.shape[-2], 2 * q.shape[-1]
    mats = q.numel() // (N * q.shape[-1])
    if scales.dtype != torch.bfloat16 or scales.shape[-1] != N or scales.numel() % (mats * N):
        raise ValueError("scales are BF16 [..., K / group, N]")
    kg = scales.numel() // (mats * N)
    _need(0 < kg <= K, "scales are BF16 [..., K / group, N]")
    group = K // kg
    if zeros is not None and (_dev(zeros).dtype != torch.uint8 or zeros.numel() != scales.numel()):
        raise ValueError("zeros are uint8 with the shape of scales")
    if group * kg != K:
        raise ValueError("the scales' rows do not divide K")
    nbytes = lib().moe_w4_packed_bytes(N, K, group, int(zeros is not None))
    _need(nbytes > 0, "no such packed matrix: N, K or group")
    data = torch.empty(mats, nbytes, dtype=torch.uint8, device=q.device)
    _check("moe_pack_w4", lib().moe_pack_w4(_ptr(q), _ptr(scales), _ptr(zeros), mats, N, K, group, _ptr(data),
                                            _stream(None)))
    return W4Packed(data, mats, N, K, group, zeros is not None)


def _zeroed(nbytes, device):
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def moe_linear_w4_workspace(T, N, K, device="cuda"):
    """A workspace for moe_linear_w4 (zeroed once here; each call leaves its counters zero)."""
    nbytes = lib().moe_linear_w4_workspace_bytes(T, N, K)
    if nbytes == 0:
        raise MoeError("moe_linear_w4_workspace_bytes", 1)
    return _zeroed(nbytes, device)


def moe_linear_w4(x, w, bias=None, out=None, out_dtype=torch.bfloat16, ws=None, dev_status=None, stream=None):
    """x BF16 [T, K] (rows may be strided), w a W4Packed matrix -> out [T, N] = x w^T (+ bias float32
    [N]) in BF16 or float32.  ws: a workspace kept from moe_linear_w4_workspace (made here
    otherwise); calls that may overlap need one each."""
    if stream is not None:
        return _run_on(stream, moe_linear_w4, x, w, bias, out, out_dtype, ws, dev_status)
    T, K = x.shape
    N = w.N
    assert x.is_cuda and x.dtype is torch.bfloat16 and x.stride(1) == 1, "x is BF16 [T, K] on the GPU, rows dense"
    assert w.mats == 1 and w.K == K, "w is one matrix with x's K"
    if bias is not None:
        _need_tensor(bias, torch.float32, (N,), "bias")
    if dev_status is not None:
        _need_word(dev_status, "dev_status")
    if out is None:
        out = torch.empty(T, N, dtype=out_dtype, device=x.device)
        os = N
    else:
        assert out.shape == (T, N) and out.stride(1) == 1
        _need(out.is_cuda, "out is on the GPU")
        os = out.stride(0) if T > 1 else N
        out_dtype = out.dtype
    assert out_dtype is torch.bfloat16 or out_dtype is torch.float32, "out is BF16 or float32"
    if ws is None:
        ws = moe_linear_w4_workspace(T, N, K, x.device)
    elif not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("ws is a contiguous GPU tensor")
    _check("moe_linear_w4", (_lib or lib()).moe_linear_w4(
        x.data_ptr(), T, K, x.stride(0) if T > 1 else K, w.data.data_ptr(), N, w.group, w.zeros,
        None if bias is None else bias.data_ptr(), out.data_ptr(), out_dtype is torch.float32, os, ws.data_ptr(),
        ws.numel(), None if dev_status is None else dev_status.data_ptr(), _stream(None)))
    return out


def moe_route_hidden_workspace(T=None, E=None, device="cuda"):
    """A workspace for moe_route_hidden (zeroed once here); one size serves all, whatever T and E."""
    return _zeroed(lib().moe_route_hidden_workspace_bytes(), device)


def moe_route_hidden(x, w_router, K, bias=None, num_tokens=None, logits=None, topk_idx=None, topk_w=None, ws=None,
                     stream=None):
    """The router from hidden states: x BF16 [T, H], w_router BF16 [E, H] -> (topk_idx int32 [T, K],
    topk_w float32 [T, K], logits float32 [T, E])."""
    if stream is not None:
        return _run_on(stream, moe_route_hidden, x, w_router, K, bias, num_tokens, logits, topk_idx, topk_w, ws)
    assert x.is_cuda and x.is_contiguous() and w_router.is_contiguous(), "expected contiguous CUDA tensors"
    assert x.dtype is torch.bfloat16 and w_router.dtype is torch.bfloat16
    T, H = x.shape
    E, wide = w_router.shape
    if wide != H or not w_router.is_cuda:
        raise ValueError("w_router is [E, H] on the GPU")
    if bias is not None:
        _need_tensor(bias, torch.float32, (E,), "bias")
    if num_tokens is not None:
        _need_word(num_tokens, "num_tokens")
    if logits is None:
        logits = torch.empty(T, E, dtype=torch.float32, device=x.device)
    else:
        _need_rows(logits, torch.float32, T, E, "logits")
    if topk_idx is None:
        topk_idx = torch.empty(T, K, dtype=torch.int32, device=x.device)
    else:
        _need_rows(topk_idx, torch.int32, T, K, "topk_idx")
    if topk_w is None:
        topk_w = torch.empty(T, K, dtype=torch.float32, device=x.device)
    else:
        _need_rows(topk_w, torch.float32, T, K, "topk_w")
    if ws is None:
        ws = moe_route_hidden_workspace(device=x.device)
    elif not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("ws is a contiguous GPU tensor")
    _check("moe_route_hidden", (_lib or lib()).moe_route_hidden(
        x.data_ptr(), T, H, w_router.data_ptr(), _ptr(bias), E, K, _ptr(num_tokens), logits.data_ptr(),
        topk_idx.data_ptr(), topk_w.data_ptr(), ws.data_ptr(), ws.numel(), _stream(None)))
    return topk_idx, topk_w, logits


class MoeLayerFew:
    """The layer for up to T tokens (T <= MOE_FEW_MAX_TOKENS) in one launch: moe_layer_few with the
    weight pointers, descriptor and workspace of one model layer.  Weights as MoeLayer's: BF16
    or E4M3 tensors (weight_tiles=True: already in the layout of moe_pack_weights, as
    MoeLayer.tensors holds them), or W4Packed for MOE_W4.  w_router [E, H] (+ router_bias [E]): forward routes by itself."""

    def __init__(self, T, H, I, E, K, dtype=MOE_BF16, w13=None, w2=None, shared_w13=None, shared_w2=None,
                 w13_scales=None, w2_scales=None, shared_w13_scales=None, shared_w2_scales=None, w_router=None,
                 router_bias=None, weight_tiles=False, device="cuda"):
        w4 = dtype == MOE_W4
        _need((shared_w13 is None) == (shared_w2 is None), "a shared expert has both matrices")
        _need(not w4 or all(isinstance(m, W4Packed) for m in (w13, w2) + (() if shared_w13 is None else (shared_w13, shared_w2))),
              "MOE_W4 takes W4Packed matrices")
        for what, m, sc, e, n, k in (("w13", w13, w13_scales, E, 2 * I, H), ("w2", w2, w2_scales, E, H, I),
                                     ("shared_w13", shared_w13, shared_w13_scales, 1, 2 * I, H),
                                     ("shared_w2", shared_w2, shared_w2_scales, 1, H, I)):
            if w4:
                if m is not None and (m.mats, m.N, m.K, m.group, m.zeros) != (e, n, k, w13.group, w13.zeros):
                    raise ValueError("a packed matrix has another shape, group or zero points than the layer")
            elif dtype == MOE_E4M3:
                _need_matrices(m, (torch.uint8, torch.float8_e4m3fn), e, n, k, what)
                _need_matrices(sc, (torch.float32,), e, n // 128, k // 128, what + "_scales")
            else:
                _need_matrices(m, (torch.bfloat16,), e, n, k, what)
        _need_tensor(w_router, torch.bfloat16, (E, H), "w_router")
        _need_tensor(router_bias, torch.float32, (E,), "router_bias")
        self.desc = FewDesc(T, H, I, E, K, dtype, int(shared_w13 is not None), int(weight_tiles),
                            w13.group if w4 else 0, int(w13.zeros) if w4 else 0)
        parts = []
        for m, s in ((w13, w13_scales), (w2, w2_scales), (shared_w13, shared_w13_scales),
                     (shared_w2, shared_w2_scales)):
            parts += [m.data if isinstance(m, W4Packed) else m, s]
        self.tensors = parts + [w_router, router_bias]
        self.weights = FewWeights(*(_ptr(t) for t in self.tensors))
        nbytes = lib().moe_layer_few_workspace_bytes(ctypes.byref(self.desc))
        if nbytes == 0:
            raise MoeError("moe_layer_few_workspace_bytes", 1)
        self.ws = _zeroed(nbytes, device)
        self.max_tokens = T
        self._descs = {T: self.desc}
        self._w = ctypes.byref(self.weights)
        self._ws = self.ws.data_ptr(), self.ws.numel()

    def forward(self, x, out=None, topk_idx=None, topk_w=None, logits=None, num_tokens=None, dev_status=None,
                stream=None):
        """x BF16 [t, H], t <= T -> (out [t, H], topk_idx, topk_w).  topk_idx / topk_w are inputs
        unless the layer routes (w_router, or logits [t, E])."""
        if stream is not None:
            return _run_on(stream, self.forward, x, out, topk_idx, topk_w, logits, num_tokens, dev_status)
        assert x.is_cuda and x.is_contiguous() and x.dtype is torch.bfloat16, "x is BF16, contiguous, on the GPU"
        t, H = x.shape
        d = self._descs.get(t)
        if d is None:
            if t > self.max_tokens:
                raise ValueError("more tokens than the layer was made for")
            d = self._descs[t] = FewDesc(t, *(getattr(self.desc, f) for f, _ in FewDesc._fields_[1:]))
        assert H == d.H
        if out is None:
            out = torch.empty_like(x)
        else:
            _need_rows(out, torch.bfloat16, t, H, "out")
        if logits is not None:
            _need_rows(logits, torch.float32, t, d.E, "logits")
        if num_tokens is not None:
            _need_word(num_tokens, "num_tokens")
        if dev_status is not None:
            _need_word(dev_status, "dev_status")
        if (topk_idx is None or topk_w is None) and self.weights.w_router is None and logits is None:
            raise ValueError("topk_idx and topk_w are needed: the layer has no router and no logits")
        if topk_idx is None:
            topk_idx = torch.empty(t, d.K, dtype=torch.int32, device=x.device)
        else:
            _need_rows(topk_idx, torch.int32, t, d.K, "topk_idx")
        if topk_w is None:
            topk_w = torch.empty(t, d.K, dtype=torch.float32, device=x.device)
        else:
            _need_rows(topk_w, torch.float32, t, d.K, "topk_w")
        _check("moe_layer_few", (_lib or lib()).moe_layer_few(
            ctypes.byref(d), self._w, x.data_ptr(), _ptr(logits), _ptr(num_tokens), topk_idx.data_ptr(),
            topk_w.data_ptr(), out.data_ptr(), *self._ws, _ptr(dev_status), _stream(None)))
        return out, topk_idx, topk_w


# ---------------------------------------------------------------- the 8-bit activation path
# A call of a few rows takes less time on the GPU than its checks here, so these look at everything in one
# expression and name what does not fit only where something does not.  get_device() is -1 off the GPU.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_CODES = (torch.uint8, torch.float8_e4m3fn)
_here = lambda: torch._C._cuda_getDevice()  # noqa: E731


def _need_codes(t, rows, cols, what):
    """t: E4M3 codes [rows, cols] (uint8 or float8_e4m3fn), contiguous on the GPU, an address, or None."""
    if t is None or isinstance(t, int):
        return
    if not (t.shape == (rows, cols) and t.dtype in _CODES and t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{what}: expected contiguous E4M3 codes (uint8 or float8_e4m3fn) of shape {(rows, cols)} on the "
                         f"GPU, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _refuse(what):
    """Something did not fit and no check of its own named it: tensors of another device than the current one."""
    raise ValueError(f"{what}: expected contiguous tensors on the current device")


def _opt(t, dtype, count, dev, what):
    """The address of an optional contiguous tensor of `count` values on the current device."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.numel() == count and t.get_device() == dev and t.is_contiguous()):
        _need_tensor(t, dtype, (count,), what)
        _refuse(what)
    return t.data_ptr()


def _word(t, dev, what):
    if t is None:
        return None
    if not (t.dtype is _I32 and t.numel() >= 1 and t.get_device() == dev):
        _need_word(t, what)
        _refuse(what)
    return t.data_ptr()


def moe_rmsnorm(x, weight, eps, residual=None, bf16=True, e4m3=False, out=None, q=None, q_scales=None,
                residual_out=None, num_tokens=None, stream=None):
    """x BF16 [T, H] (rows may be strided), weight [H] and residual [T, H] (or None) BF16 or float32 ->
    (out BF16 [T, H], q uint8 [T, H], q_scales float32 [T, H/128], residual_out like residual).
    Without out, q and q_scales, bf16 and e4m3 say which of them are made; with any of them exactly what is
    given is written.  What is not asked for is None.  residual_out=residual adds in place.
    num_tokens: int32 on the GPU; rows from it on are left as they were."""
    if stream is not None:
        return _run_on(stream, moe_rmsnorm, x, weight, eps, residual, bf16, e4m3, out, q, q_scales, residual_out,
                       num_tokens)
    T, H = shape = x.shape
    dev = _here()
    w32 = weight.dtype is _F32
    if not (x.dtype is _BF16 and x.get_device() == dev and (T == 0 or x.stride(1) == 1) and (w32 or weight.dtype is _BF16) and
            weight.numel() == H and weight.get_device() == dev and weight.is_contiguous()):
        _need(x.is_cuda and x.dtype is _BF16 and x.stride(1) == 1, "x is BF16 [T, H] on the GPU, rows dense")
        _need_tensor(weight, _F32 if w32 else _BF16, (H,), "weight")
        _refuse("x, weight")
    _need((q is None) == (q_scales is None), "q and q_scales are given together")
    if out is None and q is None:
        _need(bf16 or e4m3, "one of bf16 and e4m3 is wanted")
        if bf16:
            out = torch.empty(shape, dtype=_BF16, device=x.device)
        if e4m3:
            q = torch.empty(shape, dtype=torch.uint8, device=x.device)
            q_scales = torch.empty((T, H // 128), dtype=_F32, device=x.device)
    else:
        if out is not None and not (out.dtype is _BF16 and out.shape == shape and out.get_device() == dev and out.is_contiguous()):
            _need_tensor(out, _BF16, shape, "out")
            _refuse("out")
        if q is not None and not (q.dtype in _CODES and q.shape == shape and q_scales.dtype is _F32 and
                                  q_scales.shape == (T, H // 128) and q.get_device() == dev and q_scales.get_device() == dev and
                                  q.is_contiguous() and q_scales.is_contiguous()):
            _need_codes(q, T, H, "q")
            _need_tensor(q_scales, _F32, (T, H // 128), "q_scales")
            _refuse("q, q_scales")
    r32 = False
    if residual is not None:
        r32 = residual.dtype is _F32
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        if not ((r32 or residual.dtype is _BF16) and residual.shape == shape and residual.get_device() == dev and
                residual.is_contiguous() and residual_out.dtype is residual.dtype and residual_out.shape == shape and
                residual_out.get_device() == dev and residual_out.is_contiguous()):
            _need_tensor(residual, _F32 if r32 else _BF16, shape, "residual")
            _need_tensor(residual_out, residual.dtype, shape, "residual_out")
            _refuse("residual")
    else:
        _need(residual_out is None, "residual_out without a residual")
    _check("moe_rmsnorm", (_lib or lib()).moe_rmsnorm(
        x.data_ptr(), T, H, x.stride(0) if T > 1 else H, weight.data_ptr(), w32, eps,
        None if residual is None else residual.data_ptr(), r32, None if residual is None else residual_out.data_ptr(),
        None if out is None else out.data_ptr(), None if q is None else q.data_ptr(),
        None if q is None else q_scales.data_ptr(), _word(num_tokens, dev, "num_tokens"), _stream(None)))
    return out, q, q_scales, residual_out


def moe_linear_e4m3_workspace(T, N, K, device="cuda"):
    """A workspace for moe_linear_e4m3 (zeroed once here; each call leaves its counters zero)."""
    nbytes = lib().moe_linear_e4m3_workspace_bytes(T, N, K)
    if nbytes == 0:
        raise MoeError("moe_linear_e4m3_workspace_bytes", 1)
    return _zeroed(nbytes, device)


def moe_linear_e4m3(x, x_scales, w, w_scales, bias=None, out=None, out_dtype=torch.bfloat16, ws=None, dev_status=None,
                    stream=None):
    """x E4M3 codes [T, K] with x_scales float32 [T, K/128], w E4M3 codes [N, K] with w_scales float32
    [ceil(N/128), K/128] -> out [T, N] = x w^T (+ bias float32 [N]) in BF16 or float32 (rows of a given out
    may be strided).  ws: a workspace kept from moe_linear_e4m3_workspace (made and zeroed here otherwise,
    13 us of the call); calls that may overlap need one each."""
    if stream is not None:
        return _run_on(stream, moe_linear_e4m3, x, x_scales, w, w_scales, bias, out, out_dtype, ws, dev_status)
    T, K = x.shape
    N, k = w.shape
    dev = _here()
    if not (k == K and x.dtype in _CODES and w.dtype in _CODES and x_scales.dtype is _F32 and w_scales.dtype is _F32 and
            x_scales.shape == (T, K // 128) and w_scales.shape == ((N + 127) // 128, K // 128) and
            x.get_device() == dev and w.get_device() == dev and x_scales.get_device() == dev and
            w_scales.get_device() == dev and x.is_contiguous() and w.is_contiguous() and x_scales.is_contiguous() and
            w_scales.is_contiguous()):
        _need_codes(x, T, K, "x")
        _need_codes(w, N, K, "w")
        _need_tensor(x_scales, _F32, (T, K // 128), "x_scales")
        _need_tensor(w_scales, _F32, ((N + 127) // 128, K // 128), "w_scales")
        _refuse("x, w")
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=x.device)
        os = N
    else:
        _need(out.get_device() == dev and out.shape == (T, N) and out.stride(1) == 1,
              "out is [T, N] on the current device, rows dense")
        os = out.stride(0) if T > 1 else N
        out_dtype = out.dtype
    f32 = out_dtype is _F32
    _need(f32 or out_dtype is _BF16, "out is BF16 or float32")
    if ws is None:
        ws = moe_linear_e4m3_workspace(T, N, K, x.device)
    elif not (ws.dtype is torch.uint8 and ws.get_device() == dev and ws.is_contiguous()):
        raise ValueError("ws is a workspace of moe_linear_e4m3_workspace on the current device")
    _check("moe_linear_e4m3", (_lib or lib()).moe_linear_e4m3(
        x.data_ptr(), x_scales.data_ptr(), T, K, w.data_ptr(), w_scales.data_ptr(), N, _opt(bias, _F32, N, dev, "bias"),
        out.data_ptr(), f32, os, ws.data_ptr(), ws.numel(), _word(dev_status, dev, "dev_status"), _stream(None)))
    return out


def moe_permute_e4m3(topk_idx, E, x, x_scales, with_shared=False, max_tokens=0, xp=None, xp_scales=None, ws=None,
                     dev_status=None, topk_w=None, stream=None):
    """moe_permute of rows that are E4M3 already: x codes [T, H], x_scales float32 [T, H/128].  Returns
    moe_permute's dict, or with max_tokens > 0 moe_permute_batched's (xb, xb_scales, masked_m).
    xp / xp_scales: buffers to write to ([rows, H], [rows, H/128]; rows past the last one stay as they are)."""
    if stream is not None:
        return _run_on(stream, moe_permute_e4m3, topk_idx, E, x, x_scales, with_shared, max_tokens, xp, xp_scales, ws,
                       dev_status, topk_w)
    T, K = topk_idx.shape
    t, H = x.shape
    dev, nseg = _here(), E + int(with_shared)
    rows = nseg * max_tokens if max_tokens else T * K + (T if with_shared else 0)
    if not (t == T and topk_idx.dtype is _I32 and x.dtype in _CODES and x_scales.dtype is _F32 and
            x_scales.shape == (T, H // 128) and topk_idx.get_device() == dev and x.get_device() == dev and
            x_scales.get_device() == dev and topk_idx.is_contiguous() and x.is_contiguous() and x_scales.is_contiguous()):
        _need_tensor(topk_idx, _I32, (T, K), "topk_idx")
        _need_codes(x, T, H, "x")
        _need_tensor(x_scales, _F32, (T, H // 128), "x_scales")
        _refuse("topk_idx, x")
    if xp is None:
        xp = torch.empty((rows, H), dtype=torch.uint8, device=x.device)
    elif not (xp.dtype in _CODES and xp.shape == (rows, H) and xp.get_device() == dev and xp.is_contiguous()):
        _need_codes(xp, rows, H, "xp")
        _refuse("xp")
    if xp_scales is None:
        xp_scales = torch.empty((rows, H // 128), dtype=_F32, device=x.device)
    elif not (xp_scales.dtype is _F32 and xp_scales.shape == (rows, H // 128) and xp_scales.get_device() == dev and
              xp_scales.is_contiguous()):
        _need_tensor(xp_scales, _F32, (rows, H // 128), "xp_scales")
        _refuse("xp_scales")
    on = x.device
    cu = None if max_tokens else torch.empty(nseg + 1, dtype=_I32, device=on)
    mm = torch.empty(nseg, dtype=_I32, device=on) if max_tokens else None
    src, inv = torch.empty(rows, dtype=_I32, device=on), torch.empty_like(topk_idx)
    smap = torch.empty(T, dtype=_I32, device=on) if with_shared else None
    roww = None
    if topk_w is not None:
        _need_tensor(topk_w, _F32, (T, K), "topk_w")
        roww = torch.empty(rows, dtype=_F32, device=on)
    if ws is None:
        size = moe_permute_batched_workspace_bytes if max_tokens else moe_permute_workspace_bytes
        ws = torch.empty(size(T, K, E, with_shared), dtype=torch.uint8, device=on)
    elif not (ws.get_device() == dev and ws.is_contiguous()):
        raise ValueError("ws is a contiguous tensor on the current device")
    _check("moe_permute_e4m3", (_lib or lib()).moe_permute_e4m3(
        topk_idx.data_ptr(), T, K, E, int(with_shared), max_tokens, x.data_ptr(), x_scales.data_ptr(), H, xp.data_ptr(),
        xp_scales.data_ptr(), _ptr(cu), _ptr(mm), src.data_ptr(), inv.data_ptr(), _ptr(smap), ws.data_ptr(),
        ws.numel() * ws.element_size(), _word(dev_status, dev, "dev_status"), _opt(topk_w, _F32, T * K, dev, "topk_w"),
        _ptr(roww), _stream(None)))
    maps = dict(src_row=src, inv_map=inv, shared_map=smap, row_weights=roww)
    if max_tokens:
        return dict(xb=xp.view(nseg, max_tokens, H), xb_scales=xp_scales.view(nseg, max_tokens, -1), masked_m=mm, **maps)
    return dict(xp=xp, xp_scales=xp_scales, cu_seqlens=cu, **maps)
