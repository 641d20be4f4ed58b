"""Python binding of libsdm.so (ctypes): argument marshalling only.

`sdm_*` are the raw C entry points (pointers and sizes).  The lower-case
helpers take torch CUDA tensors, allocate outputs and the workspace with
torch (device memory is all torch provides here), call the C entry point on
the current stream and return the outputs.  Every computation happens in the
library's CUDA kernels; there is no fallback: if libsdm.so is missing or no
GPU is present the calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsdm.so")

BF16, FP32, E4M3 = 0, 1, 2
GREEDY, SAMPLE = 0, 1
STATIC, COMPACT, CAP_ACCEPT = 0, 1, 2
OP_DRAFT_CHAIN, OP_DRAFT_TREE, OP_SCHEDULE, OP_PACK, OP_VERIFY, OP_VERIFY_TREE, OP_TV_LABEL, OP_DRAFT_CHAIN_RNN = range(8)
OP_ATTEND = 8
DEV_BAD_TOKEN, DEV_TIER_UNCAPTURED, DEV_TIMEOUT, DEV_BAD_WINDOW, DEV_CAPACITY, DEV_BAD_CLASS = 1, 2, 4, 8, 16, 32
DEV_TIER_OVERFLOW, DEV_BAD_PAGE = 64, 128

EXPORTS = ("sdm_workspace_size", "sdm_markov_prepared_size", "sdm_markov_prepare", "sdm_draft_chain",
           "sdm_draft_tree", "sdm_schedule_budget", "sdm_pack_ragged", "sdm_verify", "sdm_verify_tree",
           "sdm_verify_greedy_static", "sdm_schedule_dynamic", "sdm_tv_label", "sdm_observe", "sdm_schedule_threshold",
           "sdm_threshold_sweep", "sdm_draft_chain_rnn", "sdm_status_str", "sdm_status_of_device", "sdm_check_timeout_path",
           "sdm_draft_chain_packed", "sdm_draft_chain_front",
           "sdm_cache_write", "sdm_cache_read", "sdm_cache_commit", "sdm_attend",
           "sdm_version")


class SdmRng(ctypes.Structure):
    _fields_ = [("seed", ctypes.c_uint64), ("cycle", ctypes.c_uint64)]


class SdmCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("table", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("page", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_lib = None
_VP, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_I64 = ctypes.c_int64


def _declare(lib):
    lib.sdm_workspace_size.restype = _SZ
    lib.sdm_workspace_size.argtypes = [_I] * 8
    lib.sdm_status_str.restype = ctypes.c_char_p
    lib.sdm_status_str.argtypes = [_I]
    lib.sdm_version.restype = _I
    lib.sdm_markov_prepared_size.restype = _SZ
    lib.sdm_markov_prepared_size.argtypes = [_I, _I]
    lib.sdm_markov_prepare.restype = _I
    lib.sdm_markov_prepare.argtypes = [_VP, _VP, _I, _I, _VP, _SZ, _VP, _VP]
    lib.sdm_draft_chain.restype = _I
    lib.sdm_draft_chain.argtypes = [_VP, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, SdmRng, _VP, _VP, _VP, _VP,
                                    _SZ, _VP, _VP]
    lib.sdm_draft_tree.restype = _I
    lib.sdm_draft_tree.argtypes = [_VP, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP,
                                   _VP, _VP, _SZ, _VP, _VP]
    lib.sdm_schedule_budget.restype = _I
    lib.sdm_schedule_budget.argtypes = [_VP, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]
    lib.sdm_schedule_dynamic.restype = _I
    lib.sdm_schedule_dynamic.argtypes = [_VP, _VP, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]
    lib.sdm_pack_ragged.restype = _I
    lib.sdm_pack_ragged.argtypes = [_VP, _VP, _VP, _I, _I, _VP, _I, _I, _VP, _VP, _VP, _VP, _I, _VP, _VP, _VP, _VP]
    lib.sdm_draft_chain_front.restype = _I
    lib.sdm_draft_chain_front.argtypes = [_VP, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _I, _VP, _I, _I,
                                          _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _VP, _VP, _VP, _SZ, _VP, _VP]
    lib.sdm_draft_chain_packed.restype = _I
    lib.sdm_draft_chain_packed.argtypes = [_VP, _I, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _I, _VP, _VP, _VP,
                                           _SZ, _VP, _VP]
    lib.sdm_check_timeout_path.restype = _I
    lib.sdm_check_timeout_path.argtypes = [_VP, _I, _VP, _VP, _VP, _I, _I, _I, _I, ctypes.c_ulonglong, _VP, _SZ, _VP,
                                           _VP]
    lib.sdm_status_of_device.restype = _I
    lib.sdm_status_of_device.argtypes = [ctypes.c_int32]
    lib.sdm_verify.restype = _I
    lib.sdm_verify.argtypes = [_I, _I, _F, SdmRng, _VP, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _VP, _VP, _I,
                               _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]
    lib.sdm_verify_greedy_static.restype = _I
    lib.sdm_verify_greedy_static.argtypes = [_I, _VP, _I, _I, _VP, _VP, _VP, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP]
    lib.sdm_draft_chain_rnn.restype = _I
    lib.sdm_draft_chain_rnn.argtypes = [_VP, _I, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, SdmRng, _VP, _VP, _VP,
                                        _VP, _VP, _SZ, _VP, _VP]
    lib.sdm_schedule_threshold.restype = _I
    lib.sdm_schedule_threshold.argtypes = [_VP, _I, _I, _F, _VP, _VP, _VP, _VP]
    lib.sdm_threshold_sweep.restype = _I
    lib.sdm_threshold_sweep.argtypes = [_VP, _VP, _I, _I, _VP, _I, _VP, _VP, _VP, _VP, _VP]
    lib.sdm_tv_label.restype = _I
    lib.sdm_tv_label.argtypes = [_F, _VP, _I, _I, _VP, _VP, _VP, _VP, _VP, _I, _VP, _VP, _I, _I, _I, _I, _VP, _VP,
                                 _SZ, _VP, _VP]
    lib.sdm_observe.restype = _I
    lib.sdm_observe.argtypes = [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]
    cache = ctypes.POINTER(SdmCache)
    lib.sdm_cache_write.restype = _I
    lib.sdm_cache_write.argtypes = [cache, _VP, _VP, _I64, _I64, _VP, _VP, _I, _I, _VP, _VP]
    lib.sdm_cache_read.restype = _I
    lib.sdm_cache_read.argtypes = [cache, _VP, _VP, _I, _I, _VP, _VP, _VP, _VP]
    lib.sdm_cache_commit.restype = _I
    lib.sdm_cache_commit.argtypes = [cache, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _VP, _VP, _VP, _VP]
    lib.sdm_attend.restype = _I
    lib.sdm_attend.argtypes = [cache, _VP, _I64, _VP, _VP, _I, _I, _I, _I, _F, _I, _I, _VP, _I, _VP, _VP, _VP, _SZ,
                               _VP, _VP]
    lib.sdm_verify_tree.restype = _I
    lib.sdm_verify_tree.argtypes = [_VP, _I, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _SZ, _VP, _VP]


def load(path: str = LIB_PATH):
    """Load libsdm.so (built by __graft_entry__.build / build.py); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libsdm.so not built at {path}: run speculative_decoding_markov_gb300.build")
        lib = ctypes.CDLL(path)
        _declare(lib)
        _lib = lib
    return _lib


def lib():
    return _lib or load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(st: int, what: str):
    if st != 0:
        raise RuntimeError(f"{what}: {lib().sdm_status_str(st).decode()} (status {st})")


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("inputs must be contiguous CUDA tensors")


def _need_cost(cost, R, gamma):
    """The step-cost table the schedulers index up to cost[R * (gamma + 1)]:
    fp64 with at least R * (gamma + 1) + 1 entries."""
    if cost.dtype != torch.float64 or cost.numel() < R * (gamma + 1) + 1:
        raise ValueError(f"cost must be fp64 with at least R*(gamma+1)+1 = {R * (gamma + 1) + 1} entries")


def _u16(t):
    """bf16 tensors are passed by pointer; this only checks the dtype."""
    if t.dtype != torch.bfloat16:
        raise TypeError("U and W must be bf16")
    return t


def workspace(op, R, B=0, V=0, r=0, P=0, k=0, N=0, device="cuda"):
    n = lib().sdm_workspace_size(op, R, B, V, r, P, k, N)
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device=device)


def new_status(device="cuda"):
    return torch.zeros(1, dtype=torch.int32, device=device)


# ---------------------------------------------------------------------------
def markov_prepare(U, W, out=None, dev_status=None):
    """Prepared tables of the Markov head (W^T, per-token bounds of the Markov
    term) for greedy drafting."""
    _need_cuda(U, W)
    V, r = U.shape
    n = lib().sdm_markov_prepared_size(V, r)
    if out is None:
        out = torch.empty(int(n), dtype=torch.uint8, device=U.device)
    st = lib().sdm_markov_prepare(_ptr(_u16(U)), _ptr(_u16(W)), V, r, _ptr(out), out.numel(), _ptr(dev_status),
                                  _stream())
    _check(st, "sdm_markov_prepare")
    return out


def draft_chain(L, U, W, anchor, decode=GREEDY, temperature=1.0, seed=0, cycle=0, out=None, ws=None,
                dev_status=None, prepared=None):
    _need_cuda(L, U, W, anchor)
    R, B, V = L.shape
    r = U.shape[1]
    dev = L.device
    if out is None:
        out = dict(tokens=torch.empty((R, B), dtype=torch.int32, device=dev),
                   logq=torch.zeros((R, B), dtype=torch.float32, device=dev),
                   lse=torch.zeros((R, B), dtype=torch.float32, device=dev))
    ws = workspace(OP_DRAFT_CHAIN, R, B, V, r, device=dev) if ws is None else ws
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_draft_chain(_ptr(L), _dt(L), _ptr(_u16(U)), _ptr(_u16(W)), _ptr(prepared), _ptr(anchor), R, B, V,
                               r, decode,
                               float(temperature), SdmRng(seed, cycle), _ptr(out["tokens"]), _ptr(out["logq"]),
                               _ptr(out["lse"]), _ptr(ws), ws.numel(), _ptr(dev_status), _stream())
    _check(st, "sdm_draft_chain")
    out["dev_status"] = dev_status
    return out


def draft_chain_packed(L, U, W, anchor, prepared, cu_seqlens, packed_tok, tokens=None, layout_ready=None, ws=None,
                       dev_status=None):
    """Greedy chain draft (prepared tables) that also fills its drafts into a
    ragged layout made by pack_ragged(draft=None); layout_ready: a
    torch.cuda.Event recorded after that layout's producer (or None)."""
    _need_cuda(L, U, W, anchor, cu_seqlens, packed_tok)
    R, B, V = L.shape
    r = U.shape[1]
    dev = L.device
    tokens = torch.empty((R, B), dtype=torch.int32, device=dev) if tokens is None else tokens
    ws = workspace(OP_DRAFT_CHAIN, R, B, V, r, device=dev) if ws is None else ws
    dev_status = new_status(dev) if dev_status is None else dev_status
    ev = None if layout_ready is None else ctypes.c_void_p(layout_ready.cuda_event)
    st = lib().sdm_draft_chain_packed(_ptr(L), _dt(L), _ptr(_u16(U)), _ptr(_u16(W)), _ptr(prepared), _ptr(anchor), R,
                                      B, V, r, _ptr(cu_seqlens), _ptr(packed_tok), packed_tok.numel(), ev,
                                      _ptr(tokens), _ptr(ws), ws.numel(), _ptr(dev_status), _stream())
    _check(st, "sdm_draft_chain_packed")
    return dict(tokens=tokens, dev_status=dev_status)


def draft_chain_front(L, U, W, anchor, prepared, conf, cost, tiers, use_budget=True, strict=False, tokens=None,
                      sched=None, pk=None, capacity=None, ws=None, dev_status=None):
    """Greedy chain draft (prepared tables) with the budget scheduler and the
    ragged layout in the same launches: the outputs of schedule_budget,
    pack_ragged(draft=None) and draft_chain_packed.  sched / pk: output dicts
    as those calls return (made here when None)."""
    _need_cuda(L, U, W, anchor, conf, cost, tiers)
    R, B, V = L.shape
    _need_cost(cost, R, B)
    r = U.shape[1]
    dev = L.device
    tokens = torch.empty((R, B), dtype=torch.int32, device=dev) if tokens is None else tokens
    if sched is None:
        sched = dict(survival=torch.empty((R, B), dtype=torch.float32, device=dev),
                     budget=torch.empty((R,), dtype=torch.int32, device=dev),
                     expected=torch.empty((1,), dtype=torch.float64, device=dev),
                     total_tokens=torch.empty((1,), dtype=torch.int32, device=dev))
    if pk is None:
        cap = capacity if capacity else pack_capacity(R, B, tiers.tolist())
        pk = dict(cu_seqlens=torch.empty((R + 1,), dtype=torch.int32, device=dev),
                  packed_tok=torch.empty((cap,), dtype=torch.int32, device=dev),
                  packed_req=torch.empty((cap,), dtype=torch.int32, device=dev),
                  packed_pos=torch.empty((cap,), dtype=torch.int32, device=dev),
                  tier=torch.empty((1,), dtype=torch.int32, device=dev))
    ws = workspace(OP_DRAFT_CHAIN, R, B, V, r, device=dev) if ws is None else ws
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_draft_chain_front(
        _ptr(L), _dt(L), _ptr(_u16(U)), _ptr(_u16(W)), _ptr(prepared), _ptr(anchor), R, B, V, r, _ptr(conf),
        _ptr(cost), 1 if use_budget else 0, _ptr(tiers), tiers.numel(), 1 if strict else 0, _ptr(sched["survival"]),
        _ptr(sched["budget"]), _ptr(sched["expected"]), _ptr(sched["total_tokens"]), _ptr(pk["cu_seqlens"]),
        _ptr(pk["packed_tok"]), _ptr(pk["packed_req"]), _ptr(pk["packed_pos"]), pk["packed_tok"].numel(),
        _ptr(pk["tier"]), _ptr(tokens), _ptr(ws), ws.numel(), _ptr(dev_status), _stream())
    _check(st, "sdm_draft_chain_front")
    return dict(tokens=tokens, sched=sched, pk=pk, dev_status=dev_status)


def check_timeout_path(L, U, W, anchor, wait_ns, dev_status=None):
    """One Markov GEMM launch with its loads withheld and every wait limited
    to wait_ns: the kernel records DEV_TIMEOUT and winds down."""
    _need_cuda(L, U, W, anchor)
    R, B, V = L.shape
    r = U.shape[1]
    ws = workspace(OP_DRAFT_CHAIN, R, B, V, r, device=L.device)
    dev_status = new_status(L.device) if dev_status is None else dev_status
    st = lib().sdm_check_timeout_path(_ptr(L), _dt(L), _ptr(_u16(U)), _ptr(_u16(W)), _ptr(anchor), R, B, V, r,
                                      int(wait_ns), _ptr(ws), ws.numel(), _ptr(dev_status), _stream())
    _check(st, "sdm_check_timeout_path")
    return dev_status


def draft_chain_rnn(L, U, W, A, X, anchor, decode=GREEDY, temperature=1.0, seed=0, cycle=0, out=None, ws=None,
                    dev_status=None, memo=False):
    """Chain draft with the RNN head (memo m_d = tanh(A m_{d-1} + U[y_{d-1}]
    + x_d), logits L_d + bf16(m_d) W); memo=True also returns the memo."""
    _need_cuda(L, U, W, A, X, anchor)
    R, B, V = L.shape
    r = U.shape[1]
    dev = L.device
    if out is None:
        out = dict(tokens=torch.empty((R, B), dtype=torch.int32, device=dev),
                   logq=torch.zeros((R, B), dtype=torch.float32, device=dev),
                   lse=torch.zeros((R, B), dtype=torch.float32, device=dev))
        if memo:
            out["memo"] = torch.empty((R, B, r), dtype=torch.float32, device=dev)
    ws = workspace(OP_DRAFT_CHAIN_RNN, R, B, V, r, device=dev) if ws is None else ws
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_draft_chain_rnn(_ptr(L), _dt(L), _ptr(_u16(U)), _ptr(_u16(W)), _ptr(_u16(A)), _ptr(_u16(X)),
                                   _ptr(anchor), R, B, V, r, decode, float(temperature), SdmRng(seed, cycle),
                                   _ptr(out["tokens"]), _ptr(out.get("logq")), _ptr(out.get("lse")),
                                   _ptr(out.get("memo")), _ptr(ws), ws.numel(), _ptr(dev_status), _stream())
    _check(st, "sdm_draft_chain_rnn")
    out["dev_status"] = dev_status
    return out


def draft_tree(L, U, W, anchor, k, P, N, out=None, ws=None, dev_status=None, prepared=None):
    _need_cuda(L, U, W, anchor)
    R, B, V = L.shape
    r = U.shape[1]
    dev = L.device
    S = N + 1
    words = (S + 31) // 32
    if out is None:
        out = dict(tok=torch.empty((R, S), dtype=torch.int32, device=dev),
                   parent=torch.empty((R, S), dtype=torch.int32, device=dev),
                   depth=torch.empty((R, S), dtype=torch.int32, device=dev),
                   score=torch.empty((R, S), dtype=torch.float32, device=dev),
                   mask=torch.empty((R, S, words), dtype=torch.int32, device=dev),
                   n_nodes=torch.empty((R,), dtype=torch.int32, device=dev))
    ws = workspace(OP_DRAFT_TREE, R, B, V, r, P, k, N, device=dev) if ws is None else ws
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_draft_tree(_ptr(L), _dt(L), _ptr(_u16(U)), _ptr(_u16(W)), _ptr(prepared), _ptr(anchor), R, B, V, r,
                              k, P, N,
                              _ptr(out["tok"]), _ptr(out["parent"]), _ptr(out["depth"]), _ptr(out["score"]),
                              _ptr(out["mask"]), _ptr(out["n_nodes"]), _ptr(ws), ws.numel(), _ptr(dev_status),
                              _stream())
    _check(st, "sdm_draft_tree")
    out["dev_status"] = dev_status
    return out


def schedule_budget(conf, cost, out=None, dev_status=None):
    _need_cuda(conf, cost)
    R, g = conf.shape
    _need_cost(cost, R, g)
    dev = conf.device
    if out is None:
        out = dict(survival=torch.empty((R, g), dtype=torch.float32, device=dev),
                   budget=torch.empty((R,), dtype=torch.int32, device=dev),
                   expected=torch.empty((1,), dtype=torch.float64, device=dev),
                   total_tokens=torch.empty((1,), dtype=torch.int32, device=dev))
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_schedule_budget(_ptr(conf), R, g, _ptr(cost), _ptr(out["survival"]), _ptr(out["budget"]),
                                   _ptr(out["expected"]), _ptr(out["total_tokens"]), None, 0, _ptr(dev_status),
                                   _stream())
    _check(st, "sdm_schedule_budget")
    out["dev_status"] = dev_status
    return out


def schedule_dynamic(conf, conf_stale, cost, out=None, dev_status=None):
    """The production scheduler: capacity from conf_stale (the confidences of
    two steps before) by a global search over cost, then the top K of conf's
    survivals."""
    _need_cuda(conf, conf_stale, cost)
    R, g = conf.shape
    _need_cost(cost, R, g)
    assert tuple(conf_stale.shape) == (R, g)
    dev = conf.device
    if out is None:
        out = dict(survival=torch.empty((R, g), dtype=torch.float32, device=dev),
                   budget=torch.empty((R,), dtype=torch.int32, device=dev),
                   expected=torch.empty((1,), dtype=torch.float64, device=dev),
                   total_tokens=torch.empty((1,), dtype=torch.int32, device=dev),
                   capacity=torch.empty((1,), dtype=torch.int32, device=dev))
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_schedule_dynamic(_ptr(conf), _ptr(conf_stale), R, g, _ptr(cost), _ptr(out["survival"]),
                                    _ptr(out["budget"]), _ptr(out["expected"]), _ptr(out["total_tokens"]),
                                    _ptr(out["capacity"]), _ptr(dev_status), _stream())
    _check(st, "sdm_schedule_dynamic")
    out["dev_status"] = dev_status
    return out


def schedule_threshold(conf, tau, out=None, dev_status=None):
    """Fixed-threshold verify length: the longest prefix with every
    confidence >= tau."""
    _need_cuda(conf)
    R, g = conf.shape
    dev = conf.device
    if out is None:
        out = dict(budget=torch.empty((R,), dtype=torch.int32, device=dev),
                   total_tokens=torch.empty((1,), dtype=torch.int32, device=dev))
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_schedule_threshold(_ptr(conf), R, g, float(tau), _ptr(out["budget"]), _ptr(out["total_tokens"]),
                                      _ptr(dev_status), _stream())
    _check(st, "sdm_schedule_threshold")
    return out


def threshold_sweep(conf, taus, ceiling=None, out=None, dev_status=None):
    """Drafts verified, drafts accepted (given whole-block ceilings) and
    expected accepted drafts at every threshold in taus."""
    _need_cuda(conf, taus, ceiling)
    R, g = conf.shape
    K = taus.numel()
    dev = conf.device
    if out is None:
        out = dict(drafts=torch.empty((K,), dtype=torch.int32, device=dev),
                   accepted=torch.empty((K,), dtype=torch.int32, device=dev),
                   expected=torch.empty((K,), dtype=torch.float64, device=dev))
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_threshold_sweep(_ptr(conf), _ptr(ceiling), R, g, _ptr(taus), K, _ptr(out["drafts"]),
                                   _ptr(out["accepted"]), _ptr(out["expected"]), _ptr(dev_status), _stream())
    _check(st, "sdm_threshold_sweep")
    return out


def pack_capacity(R, gamma, tiers) -> int:
    return max(max(tiers) if len(tiers) else 0, R * (gamma + 1))


def pack_ragged(anchor, draft, budget, tiers, capacity=None, out=None, dev_status=None, tier_host=None,
                strict=False, gamma=None):
    """Ragged front-pack; draft=None (give gamma) lays out the windows alone,
    every draft row -1, for draft_chain_packed to fill."""
    _need_cuda(anchor, draft, budget, tiers)
    R = anchor.numel()
    g = draft.shape[1] if draft is not None else int(gamma)
    dev = anchor.device
    if out is None:
        cap = capacity if capacity else pack_capacity(R, g, tiers.tolist())
        out = dict(cu_seqlens=torch.empty((R + 1,), dtype=torch.int32, device=dev),
                   packed_tok=torch.empty((cap,), dtype=torch.int32, device=dev),
                   packed_req=torch.empty((cap,), dtype=torch.int32, device=dev),
                   packed_pos=torch.empty((cap,), dtype=torch.int32, device=dev),
                   tier=torch.empty((1,), dtype=torch.int32, device=dev))
    cap = out["packed_tok"].numel()
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_pack_ragged(_ptr(anchor), _ptr(draft), _ptr(budget), R, g, _ptr(tiers), tiers.numel(),
                               1 if strict else 0, _ptr(out["cu_seqlens"]), _ptr(out["packed_tok"]), _ptr(out["packed_req"]),
                               _ptr(out["packed_pos"]), cap, _ptr(out["tier"]), _ptr(tier_host), _ptr(dev_status),
                               _stream())
    _check(st, "sdm_pack_ragged")
    out["dev_status"] = dev_status
    return out


def verify(mode, decode, target, cu_seqlens, anchor, draft, budget=None, logq=None, lse_q=None, L=None, U=None,
           W=None, temperature=1.0, seed=0, cycle=0, out=None, ws=None, dev_status=None):
    _need_cuda(target, cu_seqlens, anchor, draft, budget, logq, lse_q, L, U, W)
    R, g = draft.shape
    V = target.shape[-1]
    rows = target.numel() // V
    dev = target.device
    r = 0 if U is None else U.shape[1]
    if out is None:
        out = dict(accept=torch.empty((R,), dtype=torch.int32, device=dev),
                   ceiling=torch.empty((R,), dtype=torch.int32, device=dev),
                   out_tok=torch.empty((R, g + 1), dtype=torch.int32, device=dev),
                   n_out=torch.empty((R,), dtype=torch.int32, device=dev))
    ws = workspace(OP_VERIFY, R, g, V, r, rows, device=dev) if ws is None else ws
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_verify(mode, decode, float(temperature), SdmRng(seed, cycle), _ptr(target), _dt(target), rows,
                          _ptr(cu_seqlens), _ptr(anchor), _ptr(draft), _ptr(budget), _ptr(logq), _ptr(lse_q),
                          _ptr(L), _dt(L) if L is not None else BF16, _ptr(U), _ptr(W), r, R, g, V,
                          _ptr(out["accept"]), _ptr(out["ceiling"]), _ptr(out["out_tok"]), _ptr(out["n_out"]),
                          _ptr(ws), ws.numel(), _ptr(dev_status), _stream())
    _check(st, "sdm_verify")
    out["dev_status"] = dev_status
    return out


def tv_label(target, cu_seqlens, anchor, draft, L, U, W, lse_q=None, temperature=1.0, out=None, ws=None,
             dev_status=None):
    """Soft label 1 - TV(q, p) [R, gamma] of every verified window row (-1
    past the window).  target holds the packed verify rows; lse_q (the
    sampling draft's log-sum-exp) may be None."""
    _need_cuda(target, cu_seqlens, anchor, draft, L, U, W, lse_q)
    R, g = draft.shape
    V = target.shape[-1]
    rows = target.numel() // V
    dev = target.device
    r = U.shape[1]
    if out is None:
        out = torch.empty((R, g), dtype=torch.float32, device=dev)
    ws = workspace(OP_TV_LABEL, R, g, V, r, rows, device=dev) if ws is None else ws
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_tv_label(float(temperature), _ptr(target), _dt(target), rows, _ptr(cu_seqlens), _ptr(anchor),
                            _ptr(draft), _ptr(lse_q), _ptr(L), _dt(L), _ptr(_u16(U)), _ptr(_u16(W)), r, R, g, V,
                            _ptr(out), _ptr(ws), ws.numel(), _ptr(dev_status), _stream())
    _check(st, "sdm_tv_label")
    return out


def observe(conf, cu_seqlens, ceiling, cls, n_class, n_bins, out=None, dev_status=None):
    """Verify-cycle statistics: ceiling histograms per class, per-position
    observed / accepted counts, calibration bins and their ECE."""
    _need_cuda(conf, cu_seqlens, ceiling, cls)
    R, g = conf.shape
    dev = conf.device
    i32 = dict(dtype=torch.int32, device=dev)
    if out is None:
        out = dict(hist=torch.empty((n_class, g + 1), **i32), reached=torch.empty((n_class, g), **i32),
                   hits=torch.empty((n_class, g), **i32), bin_n=torch.empty((n_bins,), **i32),
                   bin_hit=torch.empty((n_bins,), **i32),
                   bin_conf=torch.empty((n_bins,), dtype=torch.float64, device=dev),
                   ece=torch.empty((1,), dtype=torch.float64, device=dev))
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_observe(_ptr(conf), _ptr(cu_seqlens), _ptr(ceiling), _ptr(cls), R, g, n_class, n_bins,
                           _ptr(out["hist"]), _ptr(out["reached"]), _ptr(out["hits"]), _ptr(out["bin_n"]),
                           _ptr(out["bin_hit"]), _ptr(out["bin_conf"]), _ptr(out["ece"]), _ptr(dev_status),
                           _stream())
    _check(st, "sdm_observe")
    out["dev_status"] = dev_status
    return out


def verify_tree(target, tok, parent, n_nodes, B, out=None, ws=None, dev_status=None):
    _need_cuda(target, tok, parent, n_nodes)
    R, S, V = target.shape
    dev = target.device
    if out is None:
        out = dict(accept=torch.empty((R,), dtype=torch.int32, device=dev),
                   out_tok=torch.empty((R, B + 1), dtype=torch.int32, device=dev),
                   n_out=torch.empty((R,), dtype=torch.int32, device=dev))
    ws = workspace(OP_VERIFY_TREE, R, B, V, 0, 0, 0, S - 1, device=dev) if ws is None else ws
    dev_status = new_status(dev) if dev_status is None else dev_status
    st = lib().sdm_verify_tree(_ptr(target), _dt(target), _ptr(tok), _ptr(parent), _ptr(n_nodes), R, S - 1, B, V,
                               _ptr(out["accept"]), _ptr(out["out_tok"]), _ptr(out["n_out"]), _ptr(ws), ws.numel(),
                               _ptr(dev_status), _stream())
    _check(st, "sdm_verify_tree")
    out["dev_status"] = dev_status
    return out


# ---------------------------------------------------------------------------
class PagedCache:
    """One layer's paged key/value cache over the caller's tensors: pools k, v
    [pages, kv heads, page, head dim] (bf16, or float8_e4m3fn with the scale
    exponents k_exp, v_exp [pages, kv heads, page] uint8) and the page table
    [requests, columns] int32.  Holds the tensors and their C description."""

    alone = False   # whether its device is the only one, and so the current one

    def __init__(self, k, v, table, k_exp=None, v_exp=None):
        _need_cuda(k, v, table, k_exp, v_exp)
        if any(x is not None and x.get_device() != k.get_device() for x in (v, table, k_exp, v_exp)):
            raise ValueError("a cache's tensors must be on one device")
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must be [pages, kv heads, page, head dim] alike")
        e4m3 = k.dtype == torch.float8_e4m3fn
        if not e4m3 and k.dtype != torch.bfloat16:
            raise TypeError(f"unsupported cache dtype {k.dtype}")
        if e4m3:
            for e in (k_exp, v_exp):
                if e is None or e.dtype != torch.uint8 or e.shape != k.shape[:3]:
                    raise ValueError("an e4m3 cache needs k_exp and v_exp [pages, kv heads, page] uint8")
        elif k_exp is not None or v_exp is not None:
            raise ValueError("only an e4m3 cache has scale exponents")
        if table.dim() != 2 or table.dtype != torch.int32:
            raise ValueError("table must be [requests, columns] int32")
        self.k, self.v, self.table, self.k_exp, self.v_exp = k, v, table, k_exp, v_exp
        self.requests = table.shape[0]
        self.device = k.get_device()
        self.alone = torch.cuda.device_count() == 1
        self.kv_heads, self.page, self.head_dim = k.shape[1:]
        self.c = SdmCache(k.data_ptr(), v.data_ptr(), k_exp.data_ptr() if e4m3 else None,
                          v_exp.data_ptr() if e4m3 else None, table.data_ptr(), E4M3 if e4m3 else BF16, k.shape[0],
                          self.kv_heads, self.page, self.head_dim, table.shape[1])
        self.ref = ctypes.byref(self.c)

    @staticmethod
    def empty(pages, kv_heads, page, head_dim, table, dtype=torch.bfloat16):
        """A cache with pools of its own (dtype bfloat16 or float8_e4m3fn)."""
        dev = table.device
        pool = [torch.zeros((pages, kv_heads, page, head_dim), dtype=torch.uint8 if dtype != torch.bfloat16 else dtype,
                            device=dev) for _ in range(2)]
        if dtype == torch.bfloat16:
            return PagedCache(*pool, table)
        exps = [torch.full((pages, kv_heads, page), 127, dtype=torch.uint8, device=dev) for _ in range(2)]
        return PagedCache(*(x.view(dtype) for x in pool), table, *exps)


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_this_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _stream_of(cache):
    """The current stream of the cache's device, which has to be the current one."""
    if not cache.alone and _this_device() != cache.device:
        raise ValueError(f"the cache is on device {cache.device}, not on the current one")
    return _raw_stream(cache.device)


# The checks of a call's tensors are on the path of the smallest calls (a step's
# write and read: 11 us), so each is one expression without calls of its own.
# `device`: the CUDA device a tensor has to be on (None: any).  What costs is
# reading a tensor's attributes, 50 to 100 ns each: a shape is read once.
_BF16, _I32, _U8 = torch.bfloat16, torch.int32, torch.uint8


def _need_rows(what, x, heads, head_dim, device=None):
    """Packed rows [rows, heads, head dim] bf16, contiguous within a row (a
    slice of a fused projection's output will do); returns the rows and their
    stride."""
    if x.dtype is not _BF16 or (x.get_device() != device and (device is not None or not x.is_cuda)):
        raise TypeError(f"{what} must be a bf16 CUDA tensor on the cache's device")
    shape, st = x.shape, x.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != head_dim:
        raise ValueError(f"{what} must be [rows, {heads}, {head_dim}]")
    if st[2] != 1 or (heads > 1 and st[1] != head_dim):
        raise ValueError(f"{what} must be contiguous within a row")
    return shape[0], st[0] if shape[0] > 1 else heads * head_dim   # one row has no next one


def _need_i32(what, x, n, device=None):
    if (x.dtype is not _I32 or (x.get_device() != device and (device is not None or not x.is_cuda)) or x.numel() < n or
            not x.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous int32 tensor of at least {n} entries on the cache's device")
    return x.data_ptr()


def _need_status(x, device):
    if x.dtype is not _I32 or x.get_device() != device or x.numel() < 1:
        raise ValueError("dev_status must be an int32 on the cache's device")
    return x.data_ptr()


def _need_out(what, x, shape, dtype, device):
    """A buffer the kernels fill: exactly this shape and type, on the cache's device."""
    if x.dtype is not dtype or x.get_device() != device or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {list(shape)} on the cache's device")
    return x.data_ptr()


def _need_ws(ws, device):
    if ws.dtype is not _U8 or ws.get_device() != device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on the cache's device")
    return ws.data_ptr()


def cache_write(cache, k, v, cu_seqlens, ctx_len, dev_status=None):
    """The windows' keys and values [rows, kv heads, head dim] into their slots
    (tokens ctx_len[i], ctx_len[i] + 1, ...), quantised if the cache is e4m3."""
    R, dev = cache.requests, cache.device
    rows, ks = _need_rows("k", k, cache.kv_heads, cache.head_dim, dev)
    v_rows, vs = _need_rows("v", v, cache.kv_heads, cache.head_dim, dev)
    if v_rows != rows:
        raise ValueError("k and v must have the same rows")
    dev_status = new_status(k.device) if dev_status is None else dev_status
    st = lib().sdm_cache_write(cache.ref, k.data_ptr(), v.data_ptr(), ks, vs,
                               _need_i32("cu_seqlens", cu_seqlens, R + 1, dev), _need_i32("ctx_len", ctx_len, R, dev),
                               R, rows, _need_status(dev_status, dev), _stream_of(cache))
    if st:
        _check(st, "sdm_cache_write")
    return dev_status


def _new_status_in(out, device):
    """A status word of the call's own, returned with its outputs."""
    out["dev_status"] = new_status(device)
    return out["dev_status"]


def cache_read(cache, cu_rows, rows, first=None, out=None, dev_status=None):
    """Tokens first[i], first[i] + 1, ... (first None: from 0) of every request
    back as bf16 rows cu_rows[i] .. cu_rows[i+1] - 1 of out["k"], out["v"].
    Without a dev_status, out["dev_status"] is the call's own (as in
    cache_commit and attend)."""
    R, dev = cache.requests, cache.device
    shape = (rows, cache.kv_heads, cache.head_dim)
    if out is None:
        out = {n: torch.empty(shape, dtype=torch.bfloat16, device=cache.k.device) for n in ("k", "v")}
    ko, vo = _need_out("out['k']", out["k"], shape, _BF16, dev), _need_out("out['v']", out["v"], shape, _BF16, dev)
    dev_status = _new_status_in(out, cache.k.device) if dev_status is None else dev_status
    st = lib().sdm_cache_read(cache.ref, _need_i32("cu_rows", cu_rows, R + 1, dev),
                              None if first is None else _need_i32("first", first, R, dev), R, rows, ko, vo,
                              _need_status(dev_status, dev), _stream_of(cache))
    if st:
        _check(st, "sdm_cache_read")
    return out


def cache_commit(cache, tok, parent, n_nodes, out_tok, accept, ctx_len, out=None, dev_status=None):
    """Moves a verified tree's accepted path (verify_tree's out_tok, accept) to
    follow the committed tokens; returns the path's slots and the new lengths."""
    R, S = tok.shape
    B, dev = out_tok.shape[1] - 1, cache.device
    if R != cache.requests:
        raise ValueError("tok must have one row per request of the cache")
    if out is None:
        out = dict(path=torch.empty((R, B + 1), dtype=torch.int32, device=tok.device),
                   length=torch.empty((R,), dtype=torch.int32, device=tok.device))
    dev_status = _new_status_in(out, tok.device) if dev_status is None else dev_status
    st = lib().sdm_cache_commit(cache.ref, _need_i32("tok", tok, R * S, dev), _need_i32("parent", parent, R * S, dev),
                                _need_i32("n_nodes", n_nodes, R, dev), _need_i32("out_tok", out_tok, R * (B + 1), dev),
                                _need_i32("accept", accept, R, dev), _need_i32("ctx_len", ctx_len, R, dev), R, S - 1, B,
                                _need_i32("path", out["path"], R * (B + 1), dev),
                                _need_i32("length", out["length"], R, dev),
                                _need_status(dev_status, dev), _stream_of(cache))
    if st:
        _check(st, "sdm_cache_commit")
    return out


def attend_workspace(cache, rows, max_window, H):
    return workspace(OP_ATTEND, cache.requests, max_window, H, cache.head_dim, rows, cache.kv_heads,
                     device=cache.k.device)


def attend(cache, q, cu_seqlens, ctx_len, max_window, scale=None, window=0, sinks=0, tree_mask=None, lse=False,
           out=None, ws=None, dev_status=None):
    """Attention of every window row q [rows, H, head dim] over its request's
    cached tokens: causal, or by a draft tree's ancestor mask (draft_tree's
    mask); window > 0 limits it to that many last tokens and the first
    `sinks`.  Returns out (and the log-sum-exp if lse)."""
    R, D, dev = cache.requests, cache.head_dim, cache.device
    shape = q.shape
    H = shape[1]
    rows, qs = _need_rows("q", q, H, D, dev)
    if H % cache.kv_heads:
        raise ValueError("q's heads must be a multiple of the cache's")
    if out is None:
        out = dict(out=torch.empty((rows, H, D), dtype=torch.bfloat16, device=q.device))
        if lse:
            out["lse"] = torch.empty((rows, H), dtype=torch.float32, device=q.device)
    o, z = _need_out("out", out["out"], shape, _BF16, dev), out.get("lse")
    if z is not None:
        z = _need_out("lse", z, (rows, H), torch.float32, dev)
    elif lse:
        raise ValueError("lse was asked for, but out has no \"lse\" to hold it")
    nodes, mask = 0, None
    if tree_mask is not None:
        nodes = tree_mask.shape[1]
        mask = _need_i32("tree_mask", tree_mask, R * nodes * ((nodes + 31) // 32), dev)
        if tree_mask.shape != (R, nodes, (nodes + 31) // 32):
            raise ValueError("tree_mask must be [requests, nodes, ceil(nodes / 32)]")
    ws = attend_workspace(cache, rows, max_window, H) if ws is None else ws
    dev_status = _new_status_in(out, q.device) if dev_status is None else dev_status
    st = lib().sdm_attend(cache.ref, q.data_ptr(), qs, _need_i32("cu_seqlens", cu_seqlens, R + 1, dev),
                          _need_i32("ctx_len", ctx_len, R, dev), R, rows, max_window, H,
                          D ** -0.5 if scale is None else scale, window, sinks, mask, nodes, o, z, _need_ws(ws, dev),
                          ws.numel(), _need_status(dev_status, dev), _stream_of(cache))
    if st:
        _check(st, "sdm_attend")
    return out
