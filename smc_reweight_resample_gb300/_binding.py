"""ctypes binding of the C ABI in ``include/smcsd.h``.

Argument marshalling only: every step of the path runs in the CUDA library. Tensors must
already live on the CUDA device; outputs are allocated with torch when not supplied. The
library is loaded from this package directory and its absence is an error: there is no
fallback.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsmcsd.so")

OK, ERR_INVALID_ARG, ERR_DTYPE, ERR_WORKSPACE, ERR_CUDA, ERR_NONFINITE, ERR_RANGE, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5, -6, -7
ERR_PAGES = -8
F32, BF16 = 0, 1
TARGET_TOKEN, TARGET_SEQUENCE = 0, 1
(OP_SD_VERIFY, OP_SMC_REWEIGHT, OP_SMC_STEP, OP_ESS_RESAMPLE, OP_PAGETABLE_REMAP, OP_PACER_BLOCK_STOP,
 OP_DRAFT_SAMPLE, OP_KV_SLOT_MAP, OP_KV_APPEND, OP_TREE_MASK, OP_LOGITS_PROCESS, OP_BEAM_SELECT, OP_STATE_REORDER,
 OP_KV_FORK, OP_KV_COMPACT, OP_DISTILL_LOSS) = range(16)

_lib = None


class SMCSDError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_string(code)} (status {code})")
        self.code = code


def load(path: str = LIB_PATH):
    """Load the CUDA library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} is missing "
                           "(run smc_reweight_resample_gb300.build.build())")
    lib = ctypes.CDLL(path)
    P, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.smcsd_workspace_size.argtypes = [i, i, i, i]
    lib.smcsd_workspace_size.restype = sz
    lib.smcsd_workspace_init.argtypes = [P, sz, P]
    lib.smcsd_check_status.argtypes = [P, P]
    lib.smcsd_status_string.argtypes = [i]
    lib.smcsd_status_string.restype = ctypes.c_char_p
    lib.sd_verify.argtypes = [P, P, i, P, P, P, i, i, i, f, P, P, P, P, P, P, sz, P]
    lib.smc_reweight.argtypes = [P, P, i, P, i, i, i, f, f, P, P, P, P, P, P, sz, P]
    lib.smc_ess_resample.argtypes = [P, i, i, f, P, P, P, P, P, sz, P]
    lib.kv_pagetable_remap.argtypes = [P, P, i, i, P, P, i, P, i, P, sz, P]
    lib.pacer_block_stop.argtypes = [P, P, f, i, i, i, i, f, f, P, P, P, P, P, sz, P]
    lib.smc_step.argtypes = [P, P, i, P, i, i, i, i, f, f, P, P, P, f, P, P, P, P, P, P, i, P, i,
                             P, sz, P]
    lib.smc_step_static.argtypes = [P, P, i, P, i, i, i, i, f, f, P, P, P, f, P, P, P, P, P, P, i,
                                    P, i, P, P]
    lib.smc_step_logq.argtypes = [P, i, P, P, i, i, i, i, f, f, P, P, P, f, P, P, P, P, P, P, i, P,
                                  i, P, sz, P]
    lib.smc_reweight_tilted.argtypes = [P, P, i, P, i, i, i, f, f, i, P, f, P, P, P, P, P, P, sz, P]
    lib.smc_step_tilted.argtypes = [P, P, i, P, i, i, i, i, f, f, i, P, f, P, P, P, f, P, P, P, P,
                                    P, P, i, P, i, P, sz, P]
    lib.pacer_block_stop_pos.argtypes = [P, P, P, f, i, i, i, i, f, f, P, P, P, P, P, sz, P]
    lib.draft_sample.argtypes = [P, i, i, i, f, P, P, P, P, P, sz, P]
    lib.smcsd_selftest_wait.argtypes = [ctypes.c_uint, P, sz, P]
    ll = ctypes.c_longlong
    lib.kv_slot_map.argtypes = [P, P, i, i, i, P, P, i, i, P, P, i, P, P, P, P, sz, P]
    lib.kv_append.argtypes = [P, P, i, i, i, i, ll, P, P, P, P, i, P, P, i, i, P, sz, P]
    lib.tree_mask.argtypes = [P, P, i, i, i, P, P, sz, P]
    lib.tree_attention_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.tree_attention_workspace_size.restype = sz
    lib.tree_attention.argtypes = [P, ll, P, P, i, i, i, P, i, P, P, i, i, i, i, P, i, i, i, f, P, P,
                                   P, sz, P]
    pp, llp = ctypes.POINTER(P), ctypes.POINTER(ll)
    lib.beam_select.argtypes = [P, ll, i, i, i, i, i, f, P, P, i, i, P, P, P, P, P, sz, P]
    lib.state_reorder.argtypes = [pp, pp, llp, i, P, i, i, i, P, sz, P]
    lib.kv_fork.argtypes = [P, P, i, P, P, i, i, P, P, i, P, sz, P]
    lib.kv_free.argtypes = [P, i, P, P, i, i, P, P, i, P, sz, P]
    lib.kv_compact.argtypes = [i, P, P, i, P, P, i, P, P, P, P, sz, P]
    lib.kv_copy_pages.argtypes = [pp, i, ll, i, P, P, i, P, P, sz, P]
    lib.distill_loss.argtypes = [P, ll, i, i, i, P, P, i, f, i, P, P, P, ll, P, sz, P]
    lib.logits_process.argtypes = [P, P, i, i, i, i, i, P, P, P, P, P, i, P, P, P, P, P, P, i, P, P, sz, P]
    for fn in ("smcsd_workspace_init", "smcsd_check_status", "sd_verify", "smc_reweight",
               "smc_ess_resample", "kv_pagetable_remap", "pacer_block_stop", "smc_step",
               "smc_step_static", "smc_step_logq", "smc_reweight_tilted", "smc_step_tilted",
               "pacer_block_stop_pos", "draft_sample", "smcsd_selftest_wait", "kv_slot_map",
               "kv_append", "tree_mask", "tree_attention", "logits_process", "beam_select",
               "state_reorder", "kv_fork", "kv_free", "kv_compact", "kv_copy_pages", "distill_loss"):
        getattr(lib, fn).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().smcsd_status_string(int(code)).decode()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"logits must be float32 or bfloat16, not {t.dtype}")


def _check(rc: int, where: str):
    if rc != OK:
        raise SMCSDError(rc, where)


def workspace_size(op: int, S: int, K: int = 0, V: int = 1) -> int:
    return int(load().smcsd_workspace_size(op, S, K, V))


class Workspace:
    """Scratch buffer for one stream of calls (zero-filled at creation, as the ABI requires)."""

    def __init__(self, op: int, S: int, K: int = 0, V: int = 1, device=None):
        self._allocate(workspace_size(op, S, K, V), device)

    def _allocate(self, n, device):
        if n == 0:
            raise ValueError("invalid workspace request")
        self.buf = torch.zeros(n + 256, dtype=torch.uint8, device=device or "cuda")
        self.filled_on = torch.cuda.current_stream(self.buf.device)  # until a call on another stream has waited for it
        off = (-self.buf.data_ptr()) % 256
        self.ptr = self.buf.data_ptr() + off
        self.nbytes = n

    @property
    def args(self):
        return ctypes.c_void_p(self.ptr), ctypes.c_size_t(self.nbytes)


def selftest_wait(ws: Workspace, limit_us: int, stream=None):
    """Runs the bounded waits against nothing; check_status(ws) then reports ERR_TIMEOUT."""
    w, n = ws.args
    _check(load().smcsd_selftest_wait(int(limit_us), w, n, _stream(stream)), "smcsd_selftest_wait")


def check_status(ws: Workspace, stream=None) -> int:
    """Wait for the stream; return (and clear) the first device-side error recorded in ws."""
    return int(load().smcsd_check_status(ctypes.c_void_p(ws.ptr), _stream(stream)))


def _on(stream, call, given):
    """call(**given) with `stream` as the current one, so that what it allocates (workspace, outputs) is that stream's memory
    and is filled in its order. The caching allocator hands memory out again in the order of the stream that it belongs to:
    what crosses between `stream` and the caller's own is marked as in use on both."""
    del given["stream"]
    current = torch.cuda.current_stream(stream.device)
    if stream == current:
        return call(**given)
    ws = given.get("ws")
    with torch.cuda.stream(stream):
        # a new workspace may not be zero yet (a captured stream cannot wait for what lies outside the capture)
        if getattr(ws, "filled_on", stream) not in (None, stream) and not torch.cuda.is_current_stream_capturing():
            stream.wait_stream(ws.filled_on)
            ws.filled_on = None
        got = call(**given)
    for t in _tensors(given.values()):
        t.record_stream(stream)
    for t in _tensors(got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)):
        t.record_stream(current)
    return got


def _tensors(values):
    """The CUDA tensors among arguments or results: themselves, a workspace's buffer, those of a list or tuple."""
    for t in values:
        if isinstance(t, (list, tuple)):
            yield from _tensors(t)
            continue
        t = getattr(t, "buf", t)
        if isinstance(t, torch.Tensor) and t.is_cuda:
            yield t


def _out(t, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if t is None else t


def sd_verify(tgt_logits, drf_logits, draft_tokens, S, K, V, temperature, uniforms,
              tgt_offsets=None, drf_offsets=None, ws=None, accept_len=None, out_token=None,
              lse_tgt=None, lse_drf=None, stream=None):
    """Returns (accept_len, out_token) int32 tensors [S]."""
    if stream is not None:
        return _on(stream, sd_verify, locals())
    dev = tgt_logits.device
    ws = ws or Workspace(OP_SD_VERIFY, S, K, V, dev)
    accept_len = _out(accept_len, (S,), torch.int32, dev)
    out_token = _out(out_token, (S,), torch.int32, dev)
    w, n = ws.args
    rc = load().sd_verify(_ptr(tgt_logits), _ptr(drf_logits), _dtype_code(tgt_logits),
                          _ptr(draft_tokens), _ptr(tgt_offsets), _ptr(drf_offsets), S, K, V,
                          float(temperature), _ptr(uniforms), _ptr(accept_len), _ptr(out_token),
                          _ptr(lse_tgt), _ptr(lse_drf), w, n, _stream())
    _check(rc, "sd_verify")
    return accept_len, out_token


def smc_reweight(tgt_logits, drf_logits, draft_tokens, S, K, V, temperature, alpha, uniforms,
                 logw, ws=None, bonus_token=None, lse_tgt=None, lse_drf=None, stream=None):
    """Updates logw in place; returns bonus_token int32 [S]."""
    if stream is not None:
        return _on(stream, smc_reweight, locals())
    dev = tgt_logits.device
    ws = ws or Workspace(OP_SMC_REWEIGHT, S, K, V, dev)
    bonus_token = _out(bonus_token, (S,), torch.int32, dev)
    w, n = ws.args
    rc = load().smc_reweight(_ptr(tgt_logits), _ptr(drf_logits), _dtype_code(tgt_logits),
                             _ptr(draft_tokens), S, K, V, float(temperature), float(alpha),
                             _ptr(uniforms), _ptr(logw), _ptr(bonus_token), _ptr(lse_tgt),
                             _ptr(lse_drf), w, n, _stream())
    _check(rc, "smc_reweight")
    return bonus_token


def smc_reweight_tilted(tgt_logits, drf_logits, draft_tokens, S, K, V, temperature, alpha,
                        uniforms, logw, target=TARGET_SEQUENCE, log_reward=None,
                        reward_scale=0.0, ws=None, bonus_token=None, lse_tgt=None, lse_drf=None,
                        stream=None):
    """smc_reweight toward the per-position (TARGET_TOKEN) or whole-sequence (TARGET_SEQUENCE)
    power target, with an optional additive log-reward float32 [S]. Updates logw in place;
    returns bonus_token int32 [S]."""
    if stream is not None:
        return _on(stream, smc_reweight_tilted, locals())
    dev = tgt_logits.device
    ws = ws or Workspace(OP_SMC_REWEIGHT, S, K, V, dev)
    bonus_token = _out(bonus_token, (S,), torch.int32, dev)
    w, n = ws.args
    rc = load().smc_reweight_tilted(_ptr(tgt_logits), _ptr(drf_logits), _dtype_code(tgt_logits),
                                    _ptr(draft_tokens), S, K, V, float(temperature), float(alpha),
                                    int(target), _ptr(log_reward), float(reward_scale),
                                    _ptr(uniforms), _ptr(logw), _ptr(bonus_token), _ptr(lse_tgt),
                                    _ptr(lse_drf), w, n, _stream())
    _check(rc, "smc_reweight_tilted")
    return bonus_token


def draft_sample(logits, R, V, temperature, uniforms, ws=None, tokens=None, logq=None, lse=None,
                 stream=None):
    """One token per row of logits [R, V] from softmax(z/T). Returns (tokens int32 [R], logq
    float [R] or None); pass logq=False to skip it, lse (float [R]) to get the normalisers."""
    if stream is not None:
        return _on(stream, draft_sample, locals())
    dev = logits.device
    ws = ws or Workspace(OP_DRAFT_SAMPLE, R, 0, V, dev)
    tokens = _out(tokens, (R,), torch.int32, dev)
    if logq is None:
        logq = torch.empty(R, dtype=torch.float32, device=dev)
    elif logq is False:
        logq = None
    w, n = ws.args
    rc = load().draft_sample(_ptr(logits), _dtype_code(logits), R, V, float(temperature),
                             _ptr(uniforms), _ptr(tokens), _ptr(logq), _ptr(lse), w, n,
                             _stream())
    _check(rc, "draft_sample")
    return tokens, logq


def smc_ess_resample(logw, G, N, ess_threshold, uniforms, ws=None, ancestors=None, ess=None,
                     resampled=None, stream=None):
    """Updates logw in place; returns (ancestors [G*N], ess [G], resampled [G])."""
    if stream is not None:
        return _on(stream, smc_ess_resample, locals())
    dev = logw.device
    ws = ws or Workspace(OP_ESS_RESAMPLE, G, 0, 1, dev)
    ancestors = _out(ancestors, (G * N,), torch.int32, dev)
    ess = _out(ess, (G,), torch.float32, dev)
    resampled = _out(resampled, (G,), torch.int32, dev)
    w, n = ws.args
    rc = load().smc_ess_resample(_ptr(logw), G, N, float(ess_threshold), _ptr(uniforms),
                                 _ptr(ancestors), _ptr(ess), _ptr(resampled), w, n, _stream())
    _check(rc, "smc_ess_resample")
    return ancestors, ess, resampled


def kv_pagetable_remap(ancestors, resampled, G, N, table_in, pages_per_seq, num_pages=0,
                       table_out=None, refcount=None, with_refcount=True, ws=None, stream=None):
    """Returns (table_out, refcount or None)."""
    if stream is not None:
        return _on(stream, kv_pagetable_remap, locals())
    ws = ws or Workspace(OP_PAGETABLE_REMAP, G, 0, 1, table_in.device)
    calls = _calls or _native(needed=False) or _Remap
    return calls.kv_pagetable_remap(ancestors, resampled, G, N, table_in, pages_per_seq, num_pages, table_out, refcount,
                                    bool(with_refcount), ws.ptr, ws.nbytes)


class _Remap:
    """kv_pagetable_remap where the call module was not built: it belongs to the step, which needs the library alone."""

    @staticmethod
    def kv_pagetable_remap(ancestors, resampled, G, N, table_in, pages_per_seq, num_pages, table_out, refcount, with_refcount, ws, nbytes):
        given = [t for t in (ancestors, resampled, table_in, table_out, refcount) if t is not None]
        for t in given:
            if t.dtype != torch.int32:
                raise TypeError(f"tensor must be Int, not {t.dtype}")
        if min(G, N, pages_per_seq) > 0:  # others are refused by the call
            for t, n, what in ((ancestors, G * N, "ancestors"), (resampled, G, "resampled"), (table_in, G * N * pages_per_seq, "a table"),
                               (table_out, G * N * pages_per_seq, "a table")):
                if t is not None and t.numel() < n:
                    raise ValueError(f"{what} is too small")
            for t in (table_in, table_out):
                # one row behind the other, whichever dimensions make up a row
                if t is not None and G * N > 1 and t.dim() > 1 and t.numel() != pages_per_seq and \
                        pages_per_seq not in [math.prod(t.shape[k:]) for k in range(1, t.dim())]:
                    raise ValueError("a table has rows of another size")
        if refcount is not None and refcount.numel() < num_pages:
            raise ValueError("refcount is too small")
        dev = table_in.device
        if dev.type != "cuda":
            raise ValueError("tensor must be on the CUDA device")
        if any(t.device != dev for t in given):
            raise ValueError("tensors must be on one device")
        with torch.cuda.device(dev):
            table_out = _out(table_out, table_in.shape, torch.int32, dev)
            if with_refcount and refcount is None:
                refcount = torch.empty(num_pages, dtype=torch.int32, device=dev)
            rc = load().kv_pagetable_remap(_ptr(ancestors), _ptr(resampled), G, N, _ptr(table_in), _ptr(table_out), pages_per_seq,
                                           _ptr(refcount), num_pages, ctypes.c_void_p(ws), ctypes.c_size_t(nbytes), _stream())
        _check(rc, "kv_pagetable_remap")
        return table_out, refcount


def pacer_block_stop(hidden, w, c, S, b, max_blocks, d, t0, rho, ws=None, lengths=None,
                     block_scores=None, offsets=True, stream=None):
    """hidden bf16 [S, max_blocks*b, d], w bf16 [d]. Returns (lengths, block_scores,
    tgt_offsets, drf_offsets); the offsets are None when offsets=False."""
    if stream is not None:
        return _on(stream, pacer_block_stop, locals())
    return pacer_block_stop_pos(hidden, w, None, c, S, b, max_blocks, d, t0, rho, ws, lengths,
                                block_scores, offsets, stream)


def pacer_block_stop_pos(hidden, w, pos_emb, c, S, b, max_blocks, d, t0, rho, ws=None,
                         lengths=None, block_scores=None, offsets=True, stream=None):
    """pacer_block_stop with position embeddings pos_emb bf16 [max_blocks*b, d] (None: none)."""
    if stream is not None:
        return _on(stream, pacer_block_stop_pos, locals())
    dev = hidden.device
    ws = ws or Workspace(OP_PACER_BLOCK_STOP, S, 0, 1, dev)
    lengths = _out(lengths, (S,), torch.int32, dev)
    block_scores = _out(block_scores, (S * max_blocks,), torch.float32, dev)
    to = torch.empty(S + 1, dtype=torch.int32, device=dev) if offsets else None
    do = torch.empty(S + 1, dtype=torch.int32, device=dev) if offsets else None
    wp, n = ws.args
    if pos_emb is None:
        rc = load().pacer_block_stop(_ptr(hidden), _ptr(w), float(c), S, b, max_blocks, d,
                                     float(t0), float(rho), _ptr(lengths), _ptr(block_scores),
                                     _ptr(to), _ptr(do), wp, n, _stream())
    else:
        rc = load().pacer_block_stop_pos(_ptr(hidden), _ptr(w), _ptr(pos_emb), float(c), S, b,
                                         max_blocks, d, float(t0), float(rho), _ptr(lengths),
                                         _ptr(block_scores), _ptr(to), _ptr(do), wp, n,
                                         _stream())
    _check(rc, "pacer_block_stop")
    return lengths, block_scores, to, do


def _step_outputs(dev, G, N, table_in, num_pages, bonus_token, ancestors, ess, resampled,
                  table_out, refcount, with_refcount):
    S = G * N
    bonus_token = _out(bonus_token, (S,), torch.int32, dev)
    ancestors = _out(ancestors, (S,), torch.int32, dev)
    ess = _out(ess, (G,), torch.float32, dev)
    resampled = _out(resampled, (G,), torch.int32, dev)
    if table_in is not None:
        table_out = _out(table_out, table_in.shape, torch.int32, dev)
        if with_refcount and refcount is None:
            refcount = torch.empty(num_pages, dtype=torch.int32, device=dev)
    else:
        table_out = refcount = None
    return dict(bonus_token=bonus_token, ancestors=ancestors, ess=ess, resampled=resampled,
                table_out=table_out, refcount=refcount)


def smc_step_tilted(tgt_logits, drf_logits, draft_tokens, G, N, K, V, temperature, alpha,
                    bonus_uniforms, logw, ess_threshold, resample_uniforms, target=TARGET_SEQUENCE,
                    log_reward=None, reward_scale=0.0, table_in=None, pages_per_seq=0,
                    num_pages=0, ws=None, bonus_token=None, ancestors=None, ess=None,
                    resampled=None, table_out=None, refcount=None, with_refcount=True,
                    stream=None):
    """smc_step toward a tilted target (see smc_reweight_tilted). Updates logw in place.
    Returns a dict of output tensors."""
    if stream is not None:
        return _on(stream, smc_step_tilted, locals())
    dev = tgt_logits.device
    ws = ws or Workspace(OP_SMC_STEP, G * N, K, V, dev)
    o = _step_outputs(dev, G, N, table_in, num_pages, bonus_token, ancestors, ess, resampled,
                      table_out, refcount, with_refcount)
    w, n = ws.args
    rc = load().smc_step_tilted(_ptr(tgt_logits), _ptr(drf_logits), _dtype_code(tgt_logits),
                                _ptr(draft_tokens), G, N, K, V, float(temperature), float(alpha),
                                int(target), _ptr(log_reward), float(reward_scale),
                                _ptr(bonus_uniforms), _ptr(logw), _ptr(o["bonus_token"]),
                                float(ess_threshold), _ptr(resample_uniforms),
                                _ptr(o["ancestors"]), _ptr(o["ess"]), _ptr(o["resampled"]),
                                _ptr(table_in), _ptr(o["table_out"]), pages_per_seq,
                                _ptr(o["refcount"]), num_pages, w, n, _stream())
    _check(rc, "smc_step_tilted")
    return o


def smc_step(tgt_logits, drf_logits, draft_tokens, G, N, K, V, temperature, alpha,
             bonus_uniforms, logw, ess_threshold, resample_uniforms, table_in=None,
             pages_per_seq=0, num_pages=0, ws=None, bonus_token=None, ancestors=None, ess=None,
             resampled=None, table_out=None, refcount=None, with_refcount=True, stream=None):
    """Fused SMC-SD step. Updates logw in place. Returns a dict of output tensors."""
    if stream is not None:
        return _on(stream, smc_step, locals())
    dev = tgt_logits.device
    S = G * N
    ws = ws or Workspace(OP_SMC_STEP, S, K, V, dev)
    bonus_token = _out(bonus_token, (S,), torch.int32, dev)
    ancestors = _out(ancestors, (S,), torch.int32, dev)
    ess = _out(ess, (G,), torch.float32, dev)
    resampled = _out(resampled, (G,), torch.int32, dev)
    if table_in is not None:
        table_out = _out(table_out, table_in.shape, torch.int32, dev)
        if with_refcount and refcount is None:
            refcount = torch.empty(num_pages, dtype=torch.int32, device=dev)
    else:
        table_out = refcount = None
    w, n = ws.args
    rc = load().smc_step(_ptr(tgt_logits), _ptr(drf_logits), _dtype_code(tgt_logits),
                         _ptr(draft_tokens), G, N, K, V, float(temperature), float(alpha),
                         _ptr(bonus_uniforms), _ptr(logw), _ptr(bonus_token), float(ess_threshold),
                         _ptr(resample_uniforms), _ptr(ancestors), _ptr(ess), _ptr(resampled),
                         _ptr(table_in), _ptr(table_out), pages_per_seq, _ptr(refcount), num_pages,
                         w, n, _stream())
    _check(rc, "smc_step")
    return dict(bonus_token=bonus_token, ancestors=ancestors, ess=ess, resampled=resampled,
                table_out=table_out, refcount=refcount)


def smc_step_logq(tgt_logits, draft_tokens, drf_logq, G, N, K, V, temperature, alpha,
                  bonus_uniforms, logw, ess_threshold, resample_uniforms, table_in=None,
                  pages_per_seq=0, num_pages=0, ws=None, bonus_token=None, ancestors=None,
                  ess=None, resampled=None, table_out=None, refcount=None, with_refcount=True,
                  stream=None):
    """smc_step with the draft's log q(x_k) (float32 [G*N*K]) in place of the draft logits."""
    if stream is not None:
        return _on(stream, smc_step_logq, locals())
    dev = tgt_logits.device
    S = G * N
    ws = ws or Workspace(OP_SMC_STEP, S, K, V, dev)
    bonus_token = _out(bonus_token, (S,), torch.int32, dev)
    ancestors = _out(ancestors, (S,), torch.int32, dev)
    ess = _out(ess, (G,), torch.float32, dev)
    resampled = _out(resampled, (G,), torch.int32, dev)
    if table_in is not None:
        table_out = _out(table_out, table_in.shape, torch.int32, dev)
        if with_refcount and refcount is None:
            refcount = torch.empty(num_pages, dtype=torch.int32, device=dev)
    else:
        table_out = refcount = None
    w, n = ws.args
    rc = load().smc_step_logq(_ptr(tgt_logits), _dtype_code(tgt_logits), _ptr(draft_tokens),
                              _ptr(drf_logq), G, N, K, V, float(temperature), float(alpha),
                              _ptr(bonus_uniforms), _ptr(logw), _ptr(bonus_token),
                              float(ess_threshold), _ptr(resample_uniforms), _ptr(ancestors),
                              _ptr(ess), _ptr(resampled), _ptr(table_in), _ptr(table_out),
                              pages_per_seq, _ptr(refcount), num_pages, w, n, _stream())
    _check(rc, "smc_step_logq")
    return dict(bonus_token=bonus_token, ancestors=ancestors, ess=ess, resampled=resampled,
                table_out=table_out, refcount=refcount)


STATIC_SCRATCH_BYTES = (32 << 20) + (32 << 10)


def smc_step_static(tgt_logits, drf_logits, draft_tokens, G, N, K, V, temperature, alpha,
                    bonus_uniforms, logw, ess_threshold, resample_uniforms, table_in=None,
                    pages_per_seq=0, num_pages=0, bonus_token=None, ancestors=None, ess=None,
                    resampled=None, table_out=None, refcount=None, with_refcount=True,
                    status=None, stream=None):
    """smc_step on the library's own scratch area (no workspace argument). Output tensors must
    be passed in by a caller that cannot allocate; missing ones are allocated here for
    convenience. `status` (int32 [1] on the device) receives the call's device-side status."""
    if stream is not None:
        return _on(stream, smc_step_static, locals())
    dev = tgt_logits.device
    S = G * N
    bonus_token = _out(bonus_token, (S,), torch.int32, dev)
    ancestors = _out(ancestors, (S,), torch.int32, dev)
    ess = _out(ess, (G,), torch.float32, dev)
    resampled = _out(resampled, (G,), torch.int32, dev)
    if table_in is not None:
        table_out = _out(table_out, table_in.shape, torch.int32, dev)
        if with_refcount and refcount is None:
            refcount = torch.empty(num_pages, dtype=torch.int32, device=dev)
    else:
        table_out = refcount = None
    rc = load().smc_step_static(_ptr(tgt_logits), _ptr(drf_logits), _dtype_code(tgt_logits),
                                _ptr(draft_tokens), G, N, K, V, float(temperature), float(alpha),
                                _ptr(bonus_uniforms), _ptr(logw), _ptr(bonus_token),
                                float(ess_threshold), _ptr(resample_uniforms), _ptr(ancestors),
                                _ptr(ess), _ptr(resampled), _ptr(table_in), _ptr(table_out),
                                pages_per_seq, _ptr(refcount), num_pages, _ptr(status),
                                _stream())
    _check(rc, "smc_step_static")
    return dict(bonus_token=bonus_token, ancestors=ancestors, ess=ess, resampled=resampled,
                table_out=table_out, refcount=refcount)


# ----------------------------------------------------------------------------------------------
# the step around the verify: page tables and slots, cache writes, attention of the drafted tokens,
# logits. Tensor shapes give the sizes that are not named; the marshalling is native (_native).
# ----------------------------------------------------------------------------------------------

class TreeAttentionWorkspace(Workspace):
    """Scratch of tree_attention for S sequences in groups of N, at most T nodes each."""

    def __init__(self, S: int, N: int, T: int, Hq: int, Hkv: int, D: int, device=None):
        n = int(load().tree_attention_workspace_size(S, N, T, Hq, Hkv, D))
        self._allocate(n, device)


_calls = None


def _native(needed=True):
    """The call module (csrc/py_calls.cpp), loaded and given the library's entry points on first use. None, where it was not built and is
    not `needed`."""
    global _calls
    if _calls is None:
        lib = load()
        path = os.path.join(_HERE, "_calls.so")
        if not os.path.exists(path):
            if not needed:
                return None
            raise RuntimeError(f"call module not built: {path} is missing "
                               "(run smc_reweight_resample_gb300.build.build())")
        spec = importlib.util.spec_from_file_location("smc_reweight_resample_gb300._calls", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in
                      ("kv_slot_map", "kv_append", "tree_mask", "tree_attention", "logits_process", "kv_pagetable_remap",
                       "beam_select", "state_reorder", "kv_fork", "kv_free", "kv_compact", "kv_copy_pages", "distill_loss")), _check)
        _calls = module
    return _calls


def kv_slot_map(ctx_len, table_in, refcount_in, S, T, page_size, new_offsets=None, rows=None, ws=None,
                table_out=None, refcount_out=None, slots=None, copy_src=None, copy_dst=None,
                stream=None):
    """Page tables, slots and copies of the step's new tokens. table_in int32 [S, pages_per_seq],
    refcount_in int32 [num_pages]; T new tokens for each sequence, or given by new_offsets (int32 [S+1],
    `rows` tokens in all). Returns dict(table_out, refcount_out, slots, copy_src, copy_dst)."""
    if stream is not None:
        return _on(stream, kv_slot_map, locals())
    ws = ws or Workspace(OP_KV_SLOT_MAP, S, 0, refcount_in.numel(), table_in.device)
    o = (_calls or _native()).kv_slot_map(ctx_len, table_in, refcount_in, S, T, page_size, new_offsets, rows,
                                          table_out, refcount_out, slots, copy_src, copy_dst, ws.ptr,
                                          ws.nbytes)
    return {"table_out": o[0], "refcount_out": o[1], "slots": o[2], "copy_src": o[3], "copy_dst": o[4]}


def kv_append(k_new, v_new, slots, k_cache, v_cache, ctx_len=None, copy_src=None, copy_dst=None, ws=None,
              stream=None):
    """Writes k_new, v_new [R, Hkv, D] (rows may be strided) to their slots (int64 [R]) of the caches
    [num_pages, Hkv, page_size, D], and the page copies that kv_slot_map asked for. Returns the caches,
    which are changed in place."""
    if stream is not None:
        return _on(stream, kv_append, locals())
    ws = ws or Workspace(OP_KV_APPEND, 1, device=k_cache.device)
    (_calls or _native()).kv_append(k_new, v_new, slots, k_cache, v_cache, ctx_len, copy_src, copy_dst, ws.ptr,
                                    ws.nbytes)
    return k_cache, v_cache


def tree_mask(parents, S, T, node_offsets=None, mask=None, ws=None, stream=None):
    """Node mask int32 [R, ceil(T/32)] (bits) of the trees that parents (int32 [R]) describes."""
    if stream is not None:
        return _on(stream, tree_mask, locals())
    ws = ws or Workspace(OP_TREE_MASK, 1, device=parents.device)
    return (_calls or _native()).tree_mask(parents, S, T, node_offsets, mask, ws.ptr, ws.nbytes)


def tree_attention(q, k_cache, v_cache, table, ctx_len, S, T, scale, N=1, node_offsets=None, mask=None,
                   ws=None, out=None, lse=None, with_lse=True, stream=None):
    """q [R, Hq, D] (rows may be strided) over the paged caches [num_pages, Hkv, page_size, D] of
    sequences with tables int32 [S, pages_per_seq] and ctx_len cached tokens, and over the nodes that
    each row sees (mask int32 [R, ceil(T/32)]; None: a chain). Returns (out [R, Hq, D], lse float
    [R, Hq], or None without it)."""
    if stream is not None:
        return _on(stream, tree_attention, locals())
    ws = ws or TreeAttentionWorkspace(S, N, T, q.shape[1], k_cache.shape[1], q.shape[2], q.device)
    return (_calls or _native()).tree_attention(q, k_cache, v_cache, table, ctx_len, S, T, scale, N, node_offsets,
                                                mask, out, lse, with_lse, ws.ptr, ws.nbytes)


def logits_process(logits, S, T, V, node_offsets=None, node_tokens=None, mask=None, hist_tokens=None,
                   hist_offsets=None, repetition=None, presence=None, frequency=None, bias_tokens=None,
                   bias_values=None, bias_offsets=None, allowed=None, out=None, ws=None, stream=None):
    """Penalties, biases and a grammar mask (bits, int32 [R, ceil(V/32)]) on logits [R, V]; pass
    out=logits to change them in place. Returns out."""
    if stream is not None:
        return _on(stream, logits_process, locals())
    ws = ws or Workspace(OP_LOGITS_PROCESS, 1, device=logits.device)
    return (_calls or _native()).logits_process(logits, S, T, V, node_offsets, node_tokens, mask, hist_tokens,
                                                hist_offsets, repetition, presence, frequency, bias_tokens,
                                                bias_values, bias_offsets, allowed, out, ws.ptr, ws.nbytes)


# ----------------------------------------------------------------------------------------------
# beam search, the pages' housekeeping, distillation
# ----------------------------------------------------------------------------------------------

def beam_select(logits, G, N, V, M, temperature=1.0, scores=None, finished=None, pad_token=0, eos_token=-1, ws=None, tokens=None,
                ancestors=None, out_scores=None, out_finished=None, stream=None):
    """The M best continuations of each of G groups of N beams: logits [G*N, >= V] (rows may be strided), scores float [G*N] of the
    beams so far, finished int32 [G*N] (such a beam stays as it is, with pad_token). Returns dict(tokens, ancestors (group-local),
    scores, finished), each [G*M], in falling order of score. N=1 without scores: the M largest log-probabilities of each row."""
    if stream is not None:
        return _on(stream, beam_select, locals())
    ws = ws or Workspace(OP_BEAM_SELECT, G * N, 0, V, logits.device)
    o = (_calls or _native()).beam_select(logits, G, N, V, M, temperature, scores, finished, pad_token, eos_token, tokens, ancestors,
                                          out_scores, out_finished, ws.ptr, ws.nbytes)
    return {"tokens": o[0], "ancestors": o[1], "scores": o[2], "finished": o[3]}


def state_reorder(states, ancestors, G, N, M=None, out=None, ws=None, stream=None):
    """Rows of each of the tensors `states` [G*N, ...] by ancestors (int32 [G*M], group-local; M=None: N). Returns the list of
    tensors [G*M, ...] (`out`, if given: memory of none of the states, in whichever order)."""
    if stream is not None:
        return _on(stream, state_reorder, locals())
    ws = ws or Workspace(OP_STATE_REORDER, 1, device=ancestors.device)
    return (_calls or _native()).state_reorder(states, ancestors, G, N, N if M is None else M, out, ws.ptr, ws.nbytes)


def kv_fork(table_in, refcount_in, parents, page_size, lengths=None, table_out=None, refcount_out=None, ws=None, stream=None):
    """Every sequence becomes a copy of its parent's first ceil(length / page_size) pages (parents int32 [S]: itself to stay, -1 for
    none; lengths int32 [S], None: all pages), shared by reference counts. Returns (table_out, refcount_out)."""
    if stream is not None:
        return _on(stream, kv_fork, locals())
    ws = ws or Workspace(OP_KV_FORK, 1, device=table_in.device)
    return (_calls or _native()).kv_fork(table_in, refcount_in, parents, page_size, lengths, table_out, refcount_out, ws.ptr, ws.nbytes)


def kv_free(table_in, refcount_in, lengths, page_size, table_out=None, refcount_out=None, ws=None, stream=None):
    """Lets go of every sequence's pages past its length (int32 [S]; 0: all of them). Returns (table_out, refcount_out)."""
    if stream is not None:
        return _on(stream, kv_free, locals())
    ws = ws or Workspace(OP_KV_FORK, 1, device=table_in.device)
    return (_calls or _native()).kv_free(table_in, refcount_in, lengths, page_size, table_out, refcount_out, ws.ptr, ws.nbytes)


def kv_compact(table_in, refcount_in, table_out=None, refcount_out=None, src=None, dst=None, counts=None, ws=None, stream=None):
    """New ids for the pages in use, so that they fill the front of the cache: dict(table_out, refcount_out, src, dst (int32
    [num_pages // 2], -1 behind the moves), counts (int32 [2]: moves, pages in use)); kv_copy_pages then moves the pages."""
    if stream is not None:
        return _on(stream, kv_compact, locals())
    ws = ws or Workspace(OP_KV_COMPACT, 1, 0, refcount_in.numel(), table_in.device)
    o = (_calls or _native()).kv_compact(table_in, refcount_in, table_out, refcount_out, src, dst, counts, ws.ptr, ws.nbytes)
    return {"table_out": o[0], "refcount_out": o[1], "src": o[2], "dst": o[3], "counts": o[4]}


def kv_copy_pages(caches, src, dst, count=None, ws=None, stream=None):
    """Copies page src[i] to page dst[i] (int32) in each of the tensors `caches` [num_pages, ...], for all i or the first count[0]
    (int32). Returns the caches, which are changed in place."""
    if stream is not None:
        return _on(stream, kv_copy_pages, locals())
    ws = ws or Workspace(OP_KV_FORK, 1, device=src.device)
    (_calls or _native()).kv_copy_pages(caches, src, dst, count, ws.ptr, ws.nbytes)
    return caches


def distill_loss(logits, top_tokens, top_values, V, temperature=1.0, rest=False, weight=None, loss=None, dlogits=None, grad=True,
                 with_loss=True, ws=None, stream=None):
    """Loss of the draft's logits [R, >= V] (rows may be strided) against a teacher's top tokens (int32 [R, K], -1: none) with their
    values (float [R, K]), and the gradient weight[r] * dloss[r]/dlogits (pass dlogits=logits for it to take their place). rest: the
    values are log-probabilities over the whole vocabulary, and what they leave goes to all other tokens. Returns (loss float [R] or
    None, dlogits [R, V] or None). The loss has no graph, also where the logits require a gradient: logits.backward(dlogits) sends the
    gradient on (of loss.sum(), or with `weight` of (weight * loss).sum())."""
    if stream is not None:
        return _on(stream, distill_loss, locals())
    ws = ws or Workspace(OP_DISTILL_LOSS, 1, device=logits.device)
    return (_calls or _native()).distill_loss(logits, top_tokens, top_values, V, temperature, bool(rest), weight, loss, dlogits, bool(grad),
                                              bool(with_loss), ws.ptr, ws.nbytes)
